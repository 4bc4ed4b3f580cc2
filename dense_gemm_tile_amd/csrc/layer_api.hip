// Host side of the layer operators (gemm_layer.h): argument checks, kernel
// choice and launches. A call either enqueues its work or returns a code and
// launches nothing.
#include <cstdio>
#include <cstring>
#include <new>
#include <string>

#include "gemm_layer.h"
#include "api_state.h"
#include "layer.h"
#include "layer_checks.h"
#include "layer_rows.h"

namespace dgt {
namespace {

// Widest staging load, in 16-bit elements, that an operand's base and row
// pitch allow.
int vector_width16(const void* ptr, int64_t ld) {
  int vw = 8;
  while (vw > 1 && ((uintptr_t)ptr % (2 * vw) != 0 || ld % vw != 0)) vw /= 2;
  return vw;
}
bool wide16(const Mat& m) {
  return m.ptr && (uintptr_t)m.ptr % 16 == 0 && m.ld * m.elem % 16 == 0 &&
         (m.count <= 1 || m.stride * m.elem % 16 == 0);
}

// ----------------------------------------------------------------- products --
enum LayerKernel : int {
  LK_GENERAL128 = 0, LK_GENERAL64, LK_PP256, LK_PP128, LK_PP128_DEEP,
  LK_SKINNY16, LK_SKINNY16N16, LK_SKINNY32, LK_SKINNY48, LK_SKINNY64, LK_SKINNY64N64,
  LK_ANY16, LK_ANY32, LK_ANY64, LK_ROWS16, LK_GENERAL64K4, LK_RING128,
  NUM_LAYER_KERNELS
};
struct LayerKernelInfo {
  const char* name;
  int bm, bn, threads;
};
const LayerKernelInfo kLayerKernels[NUM_LAYER_KERNELS] = {
    {"g128x128", 128, 128, 256}, {"g64x64", 64, 64, 256}, {"pp256x256", 256, 256, 512},
    {"pp128x128", 128, 128, 512}, {"pp128x128deep", 128, 128, 512},
    {"s16x32", 16, 32, 512}, {"s16x16", 16, 16, 512}, {"s32x32", 32, 32, 512},
    {"s48x32", 48, 32, 512}, {"s64x32", 64, 32, 256},
    {"s64x64", 64, 64, 256}, {"u16x32", 16, 32, 512}, {"u32x32", 32, 32, 512},
    {"u64x32", 64, 32, 512}, {"r16x32", 16, 32, 512},
    {"g64x64k4", 64, 64, 1024}, {"r128x128", 128, 128, 256},
};

struct LayerPlan {
  LayerArgs a{};
  int dtype = 0;
  bool ta = false, tb = false;
  bool reach = false;   // 32-bit offsets reach a tile's rows of both operands
  bool direct = false;  // and both load in whole 16-byte pieces
  int kernel = LK_GENERAL128;
  int ntiles = 0;  // workgroups that cover every tile (by rows: at least)
};

thread_local struct {
  const char* op;
  const char* ops;
  int kernel, act;
  bool bias, residual, z, out32;
} g_layer_path;
const char* const kActNames[] = {"none", "relu", "gelu", "gelu_erf", "silu"};

void write_layer_path(std::string& to) {
  const auto& m = g_layer_path;
  to = std::string(m.op) + " mfma " + kLayerKernels[m.kernel].name + " " + m.ops;
  if (m.act) to += std::string(" act=") + kActNames[m.act];
  if (m.bias) to += " bias";
  if (m.residual) to += " residual";
  if (m.z) to += " z";
  if (m.out32) to += " f32-out";
}

// Row tiles that hold M rows in G groups, whatever the groups' sizes: each
// group's last tile may be cut short.
int64_t row_tiles(const LayerArgs& a, int bm) {
  if (a.mode != LAYER_ROWS) return ((int64_t)a.M + bm - 1) / bm;
  const int64_t g = a.G < a.M ? a.G : a.M;
  return ((int64_t)a.M + g * (bm - 1)) / bm;
}
int64_t count_tiles(const LayerArgs& a, const LayerKernelInfo& k) {
  return row_tiles(a, k.bm) * (((int64_t)a.N + k.bn - 1) / k.bn) *
         (a.mode == LAYER_SUM ? a.G : 1);
}

// Whether 32-bit offsets reach the 257 rows that a tile of any kernel spans, and
// whether an operand loads in whole 16-byte pieces as well. `along` is its
// contiguous dimension.
bool layer_reach(const Mat& m) { return m.ptr && m.ld < (int64_t{1} << 31) / (2 * 257) - 4096; }
bool layer_direct(const Mat& m, int64_t along) {
  return layer_reach(m) && wide16(m) && along % 8 == 0;
}

// Whether kernel k can run the call at all.
bool kernel_runs(const LayerPlan& pl, int k) {
  if (k == LK_GENERAL128 || k == LK_GENERAL64 || k == LK_GENERAL64K4) return true;
  if (pl.a.K == 0) return false;
  // Operands stored along K are not staged there.
  if (k == LK_RING128)
    return pl.reach && (pl.ta || !pl.tb) && (pl.a.a_direct || pl.ta) && (pl.a.b_direct || !pl.tb);
  if (k == LK_ROWS16) return pl.direct && pl.tb && pl.a.mode == LAYER_ROWS;
  if (k >= LK_ANY16) return pl.reach && !pl.ta && pl.tb && pl.a.mode != LAYER_SUM;
  if (!pl.direct) return false;
  if (k < LK_SKINNY16) return true;
  // Operands not stored along K come in rows of 32 or 64 elements.
  if (pl.ta) return k == LK_SKINNY32 || k == LK_SKINNY64 || k == LK_SKINNY64N64;
  return pl.tb || k != LK_SKINNY16N16;
}

// By rows, the groups' sizes are only known on average. Measured on weights of
// 2048 x 2048, 64 groups, us by average rows a group:
//            2    8    16   32   64   128  (1024)
//   r16x32   81  110  156  247
//   s64x64  100  118  121  133  166  257
//   pp128   109  127  129  131  164  163   742
//   pp256   122  137  139  141  149  207   515
// and with B stored [K][N], where pieces of 32 or 64 columns cost the small tiles
// as much as whole lines: s16x32 119 at 2 rows, pp128 89.
int choose_grouped(const LayerPlan& pl) {
  const LayerArgs& a = pl.a;
  const int64_t used = a.G < a.M ? a.G : a.M, rows = (a.M + a.G - 1) / a.G;
  // Tiles to expect: whole ones, and one cut short for every other group.
  auto tiles = [&](int k) {
    const LayerKernelInfo& i = kLayerKernels[k];
    int64_t m = a.M / i.bm + (used + 1) / 2;
    m = (m > used ? m : used) + used / 20;
    return m * ((a.N + i.bn - 1) / i.bn);
  };
  // One wave of workgroups takes 1.4 times as long on 256 x 256 tiles (one to a
  // CU) as on 128 x 128 ones (two to a CU).
  const int64_t rounds256 = (tiles(LK_PP256) + 255) / 256, rounds128 = (tiles(LK_PP128) + 511) / 512;
  if (rows >= 96 && tiles(LK_PP256) >= 192 && 14 * rounds256 < 10 * rounds128) return LK_PP256;
  if (!pl.tb && rows <= 16 && tiles(LK_SKINNY16) <= 512) return LK_SKINNY16;
  if (pl.tb) {
    if (rows <= 32 && tiles(LK_SKINNY32) <= 256) return LK_SKINNY32;
    if (tiles(LK_SKINNY64N64) <= 512) return LK_SKINNY64N64;
    // (A K that leaves a wave less than two slices is too short to split.)
    if (a.K >= 1024 && rows <= 48) return rows <= 8 ? LK_ROWS16 : LK_SKINNY64N64;
  }
  return tiles(LK_PP128) > 256 ? LK_PP128 : LK_PP128_DEEP;
}

// own: a product that is a step of another operator.
int choose_kernel(const LayerPlan& pl, bool own) {
  const LayerArgs& a = pl.a;
  auto tiles = [&](int k) { return count_tiles(a, kLayerKernels[k]); };
  if (!kernel_runs(pl, LK_PP256)) {
    // Few rows a group: one row of tiles each, so 64 x 64 tiles. The count above is of
    // the most tiles that the groups' sizes could make, not of those to expect. An odd
    // pitch of A, B stored [N][K], 2 rows a group, us:
    //                            tiles   u16x32   g64x64k4   g64x64   g128x128
    //   256 groups of 1024x512    4096     136       135        60        67
    //   64 groups of 2048x2048    2048     147       140       127       130
    //   8 groups of 2048x2048      256      21        17        28        36
    //   8 groups of 1024x1024      128       9        10        13        20
    // (16 rows of 64 groups: 171, 145, 128, 131; 64 rows: g64x64 145, g128x128 141; B
    // stored [K][N] with an odd pitch, 16 rows: g64x64 114, g128x128 121, r128x128 131.)
    // With an odd pitch of B, up to 4 rows a group, u16x32 is ahead to 512 tiles:
    //   24 groups of 1024x1024     384      15        21        18        24
    //   8 groups of 4096x2048      512      30        35        32        42
    //   16 groups of 4096x1024    1024      35        43        24        27
    const int64_t used = a.G < a.M ? a.G : a.M, rows = a.G ? (a.M + (int64_t)a.G - 1) / a.G : 0;
    if (a.mode == LAYER_ROWS && rows <= 32) {
      const int64_t n = used * (((int64_t)a.N + 63) / 64);
      if (kernel_runs(pl, LK_ANY16) && rows <= 16 && n <= (rows <= 4 && !a.b_direct ? 512 : 128))
        return LK_ANY16;
      return n <= 256 && a.K >= 512 ? LK_GENERAL64K4 : LK_GENERAL64;
    }
    if (kernel_runs(pl, LK_ANY16) && a.mode == LAYER_DENSE && (a.M <= 64 || tiles(LK_ANY64) <= 256)) {
      // The most rows a tile that still give every CU one (64x4096x4095:
      // 128 tiles of 64 rows 43 us, 256 of 32 rows 29).
      for (int k : {LK_ANY64, LK_ANY32})
        if (a.M > kLayerKernels[k].bm / 2 && tiles(k) >= 224) return k;
      return a.M <= 32 ? LK_ANY16 : LK_ANY32;
    }
    // The sum split over wave groups where 64 x 64 tiles leave CUs idle, or a long
    // sum dominates (300x5001x3001: 87 us on 64 x 64 tiles, 65 split).
    const int64_t n64 = tiles(LK_GENERAL64);
    if ((n64 <= 256 && a.K >= 512) || (n64 <= 512 && a.K >= 2048)) return LK_GENERAL64K4;
    // 64 x 64 tiles where 128 x 128 ones would leave CUs without work.
    if (tiles(LK_GENERAL128) < 256) return LK_GENERAL64;
    // The general kernel transposes operands not stored along K in registers; the
    // ring reads them transposed from LDS, and pays for staging the others (4096^3,
    // us: one of the former 336-357 against 246-282, one of the latter 185 against
    // 209, one of each 104 against 112 at 4000x4001x1023).
    return kernel_runs(pl, LK_RING128) ? LK_RING128 : LK_GENERAL128;
  }
  if (a.mode == LAYER_ROWS) return choose_grouped(pl);
  const bool split = kernel_runs(pl, LK_SKINNY64N64);
  // Few rows: the weights' bytes count.
  if (split && !pl.ta && a.M <= 64) {
    // Many columns, one tile of 64 to a CU or more (us, bf16, float32 out, K of 2048; of
    // 1024 and 4096 the same way):
    //                     16384   32001   65536   128000 columns
    //   61 rows, s64x32    21.4    41.6    78.4    152
    //            s64x64    17.1    32.9    64.6    131
    //   24 rows, s32x32    16.7    32.4    62.5    121
    //            s64x64    15.5    30.3    58.4    115
    // and at 8192, 128 tiles, s64x32 9.3, s64x64 11.1. (gemm_linear's own calls keep the
    // order of their sums.)
    if (own && a.M > 16 && tiles(LK_SKINNY64N64) >= 256) return LK_SKINNY64N64;
    // (16 columns of B stored [K][N] would be a quarter of a line.)
    if (a.M <= 16) return pl.tb && a.N <= 16 * 256 ? LK_SKINNY16N16 : LK_SKINNY16;
    if (a.M <= 32 || tiles(LK_SKINNY32) <= 256) return LK_SKINNY32;
    return a.M <= 48 ? LK_SKINNY48 : LK_SKINNY64;
  }
  const int64_t n256 = tiles(LK_PP256);
  if (n256 >= 256 || (n256 >= 192 && a.K >= 1024) || (n256 >= 128 && a.K >= 2048)) return LK_PP256;
  // Small grids: tiles with the sum split over waves, the smallest that fit the
  // CUs in one round, or two rounds of 64 x 64 ones (512x4096x4096 41 us against
  // 52 on 128 x 128 tiles, 1024x2048x2048 26 against 30; four rounds, 2048^3, 49
  // against 32).
  if (split) {
    for (int k : {LK_SKINNY32, LK_SKINNY64})
      if (tiles(k) <= 256) return k;
    if (tiles(LK_SKINNY64N64) <= 512) return LK_SKINNY64N64;
  }
  return tiles(LK_PP128) > 256 ? LK_PP128 : LK_PP128_DEEP;
}

// forced: GEMM_LAYER_TILE counts; without it the product is a step of another operator.
int plan_tiles(LayerPlan& pl, const char* op, bool forced = true) {
  LayerArgs& a = pl.a;
  pl.kernel = choose_kernel(pl, !forced);
  if (const char* want = forced ? forced_layer_tile() : nullptr) {
    int found = -1;
    for (int k = 0; k < NUM_LAYER_KERNELS; ++k)
      if (std::strcmp(want, kLayerKernels[k].name) == 0) found = k;
    if (found < 0)
      return fail(GEMM_ERR_INVALID_ARG, std::string("GEMM_LAYER_TILE names no kernel: ") + want);
    if (!kernel_runs(pl, found))
      return fail(GEMM_ERR_UNSUPPORTED, std::string("GEMM_LAYER_TILE cannot run this call: ") + want);
    pl.kernel = found;
  }
  const LayerKernelInfo& k = kLayerKernels[pl.kernel];
  const int64_t n = count_tiles(a, k);
  // (A launch holds less than 2^32 threads.)
  if (n > ((int64_t{1} << 32) - 1) / k.threads)
    return fail(GEMM_ERR_UNSUPPORTED, "too many output tiles for one launch");
  a.tiles_m = (a.M + k.bm - 1) / k.bm;
  a.tiles_n = (a.N + k.bn - 1) / k.bn;
  a.group_m = 8;
  pl.ntiles = (int)n;
  static const char* const ops[4] = {"NN", "NT", "TN", "TT"};
  a.whole8 = a.N % 8 == 0;
  g_layer_path = {op, ops[pl.ta * 2 + pl.tb], pl.kernel, a.act, a.bias != nullptr,
                  a.R != nullptr, a.Z != nullptr, a.out32 != 0};
  set_path_writer(write_layer_path);
  return GEMM_OK;
}

hipError_t launch_product(const LayerPlan& pl, hipStream_t s) {
  switch (pl.kernel) {
    case LK_PP256: return launch_layer_pp256(pl.dtype, pl.ta, pl.tb, pl.a, pl.ntiles, s);
    case LK_PP128:
    case LK_PP128_DEEP:
      return launch_layer_pp128(pl.dtype, pl.ta, pl.tb, pl.kernel == LK_PP128_DEEP, pl.a, pl.ntiles, s);
    case LK_RING128: return launch_layer_ring(pl.dtype, pl.ta, pl.tb, pl.a, pl.ntiles, s);
    case LK_GENERAL128:
    case LK_GENERAL64:
    case LK_GENERAL64K4:
      return launch_layer_general(pl.dtype, pl.ta, pl.tb,
                                  pl.kernel == LK_GENERAL128 ? 0 : pl.kernel == LK_GENERAL64 ? 1 : 2,
                                  pl.a, pl.ntiles, s);
    default: {
      const LayerKernelInfo& k = kLayerKernels[pl.kernel];
      if (pl.kernel >= LK_ANY16)
        return launch_layer_skinny(pl.dtype, pl.kernel != LK_ROWS16, k.bm / 16, pl.a, pl.ntiles, s);
      return launch_layer_split(pl.dtype, pl.ta, pl.tb, k.bm / 16, k.bn / 16, pl.a, pl.ntiles, s);
    }
  }
}

// Dense and by-rows products (G < 0: dense).
int plan_product(int64_t G, int64_t M, int64_t N, int64_t K, int dtype, int transA, int transB,
                 const int32_t* offsets, const void* A, int64_t lda, const void* B, int64_t ldb,
                 int64_t stride_b, const void* bias, int act, const void* R, int64_t ldr,
                 const void* Y, int64_t ldy, int out_dtype, const void* Z, int64_t ldz,
                 LayerPlan& pl, bool& noop, bool forced = true) {
  const bool dense = G < 0;
  noop = false;
  CHECK(check_dim("M", M));
  CHECK(check_dim("N", N));
  CHECK(check_dim("K", K));
  CHECK(check_dtype16(dtype));
  CHECK(check_out_dtype(dtype, out_dtype));
  CHECK(check_act(act));
  const bool ta = transA != 0, tb = transB != 0;
  const int osz = out_dtype == GEMM_DTYPE_F32 ? 4 : 2;
  const int64_t g = dense ? 1 : G;
  const Mat ma{"A", A, ta ? K : M, ta ? M : K, lda, 2};
  const Mat mb{"B", B, tb ? N : K, tb ? K : N, ldb, 2, g, stride_b};
  const Mat mbias{"bias", bias, 1, N, N, 2, g, N};
  const Mat mr{"R", R, M, N, ldr, osz}, my{"Y", Y, M, N, ldy, osz}, mz{"Z", Z, M, N, ldz, 2};
  const Mat moff{"offsets", offsets, 1, g + 1, g + 1, 4};
  CHECK(check_ld(ma));
  CHECK(check_ld(mb));
  CHECK(check_ld(my));
  if (R) CHECK(check_ld(mr));
  if (Z) CHECK(check_ld(mz));
  if (!dense && g > 1 && stride_b < 0) return bad("%s is negative: %lld", "stride_b", stride_b);
  if (M == 0 || N == 0 || g == 0) {
    noop = true;
    set_path("noop: empty output");
    return GEMM_OK;
  }
  CHECK(check_ptr(my));
  if (K > 0) {
    CHECK(check_ptr(ma));
    CHECK(check_ptr(mb));
    CHECK(check_apart(my, ma));
    CHECK(check_apart(my, mb));
    CHECK(check_apart(mz, ma));
    CHECK(check_apart(mz, mb));
  }
  if (bias) CHECK(check_ptr(mbias));
  if (R) CHECK(check_ptr(mr));
  if (Z) CHECK(check_ptr(mz));
  CHECK(check_apart(my, mbias));
  CHECK(check_apart(mz, mbias));
  CHECK(check_apart_or_same(my, mr));
  CHECK(check_apart(mz, mr));
  CHECK(check_apart(my, mz));
  if (!dense) {
    CHECK(check_ptr(moff));
    CHECK(check_apart(my, moff));
    CHECK(check_apart(mz, moff));
  }
  LayerArgs& a = pl.a;
  a.A = A;
  a.B = B;
  a.bias = bias;
  a.R = R;
  a.Y = const_cast<void*>(Y);
  a.Z = const_cast<void*>(Z);
  a.offsets = offsets;
  a.lda = lda;
  a.ldb = ldb;
  a.ldr = ldr;
  a.ldy = ldy;
  a.ldz = ldz;
  a.stride_b = stride_b;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.G = (int)g;
  a.mode = dense ? LAYER_DENSE : LAYER_ROWS;
  a.act = act;
  a.out32 = osz == 4;
  a.a_vw = vector_width16(A, lda);
  a.b_vw = vector_width16(B, ldb);
  if (g > 1)
    while (a.b_vw > 1 && stride_b % a.b_vw != 0) a.b_vw /= 2;
  pl.dtype = dtype;
  pl.ta = ta;
  pl.tb = tb;
  pl.reach = layer_reach(ma) && layer_reach(mb);
  a.a_direct = layer_direct(ma, ta ? M : K);
  a.b_direct = layer_direct(mb, tb ? K : N);
  pl.direct = a.a_direct && a.b_direct;
  return plan_tiles(pl, dense ? "linear" : "grouped", forced);
}

int plan_grad_weight(int64_t G, int64_t M, int64_t N, int64_t K, int dtype, const int32_t* offsets,
                     const void* A, int64_t lda, const void* B, int64_t ldb, const void* D,
                     int64_t ldd, int64_t stride_d, int out_dtype, int accumulate, LayerPlan& pl,
                     bool& noop, bool forced = true) {
  noop = false;
  CHECK(check_dim("M", M));
  CHECK(check_dim("N", N));
  CHECK(check_dim("K", K));
  CHECK(check_dtype16(dtype));
  CHECK(check_out_dtype(dtype, out_dtype));
  const int osz = out_dtype == GEMM_DTYPE_F32 ? 4 : 2;
  const Mat ma{"A", A, M, N, lda, 2}, mb{"B", B, M, K, ldb, 2};
  const Mat md{"D", D, N, K, ldd, osz, G, stride_d};
  const Mat moff{"offsets", offsets, 1, G + 1, G + 1, 4};
  CHECK(check_ld(ma));
  CHECK(check_ld(mb));
  CHECK(check_ld(md));
  if (N == 0 || K == 0 || G == 0) {
    noop = true;
    set_path("noop: empty output");
    return GEMM_OK;
  }
  // (128 bits: a matrix of N - 1 long pitches may be past 64.)
  const __int128 one = (__int128)(N - 1) * ldd + K;
  if (G > 1 && stride_d < one)
    return bad("%s=%lld is smaller than one matrix of %lld elements", "stride_d", stride_d,
               one > INT64_MAX ? INT64_MAX : (int64_t)one);
  CHECK(check_ptr(md));
  CHECK(check_ptr(moff));
  CHECK(check_apart(md, moff));
  if (M > 0) {
    CHECK(check_ptr(ma));
    CHECK(check_ptr(mb));
    CHECK(check_apart(md, ma));
    CHECK(check_apart(md, mb));
  }
  LayerArgs& a = pl.a;
  a.A = A;
  a.B = B;
  a.Y = const_cast<void*>(D);
  a.R = accumulate ? D : nullptr;
  a.offsets = offsets;
  a.lda = lda;
  a.ldb = ldb;
  a.ldr = a.ldy = ldd;
  a.stride_y = stride_d;
  a.M = (int)N;
  a.N = (int)K;
  a.K = (int)M;
  a.G = (int)G;
  a.mode = LAYER_SUM;
  a.out32 = osz == 4;
  a.a_vw = vector_width16(A, lda);
  a.b_vw = vector_width16(B, ldb);
  pl.dtype = dtype;
  pl.ta = true;
  pl.tb = false;
  pl.reach = M > 0 && layer_reach(ma) && layer_reach(mb);
  a.a_direct = M > 0 && layer_direct(ma, N);
  a.b_direct = M > 0 && layer_direct(mb, K);
  pl.direct = a.a_direct && a.b_direct;
  return plan_tiles(pl, "grad_weight", forced);
}

// ------------------------------------------------------------- rows and ids --
int64_t act_grad_bytes(int64_t G, int64_t M, int64_t N) {
  if (G < 0 || M < 0 || N < 0 || G > kMaxGroups || M > kMaxDim || N > kMaxDim) return 0;
  const int64_t rows = act_grad_rows(M, N);
  const unsigned __int128 b =
      (unsigned __int128)((M + rows - 1) / rows + G) * (unsigned __int128)N * 4;
  return b > (unsigned __int128)INT64_MAX ? 0 : (int64_t)b;
}

int64_t route_bytes(int64_t T, int64_t top, int64_t E) {
  if (T < 0 || top < 0 || E < 0 || E > kRouteMaxExperts || T > kMaxDim || top > kMaxDim ||
      T * top > kMaxDim)
    return 0;
  int blocks, chunk;
  route_blocks(T * top, blocks, chunk);
  return blocks > 1 ? (int64_t)blocks * (E + 1) * 4 : 0;
}

// Elements per access that H and every matrix's base and pitch allow, at most
// 16 bytes.
template <size_t n>
int common_piece(int64_t H, int elem, const Mat* const (&mats)[n]) {
  int piece = 16 / elem;
  auto fits = [&](int q) {
    if (H % q) return false;
    for (const Mat* m : mats)
      if (m->ptr && ((uintptr_t)m->ptr % (q * elem) || (m->ld % q && m->rows > 1))) return false;
    return true;
  };
  while (piece > 1 && !fits(piece)) piece /= 2;
  return piece;
}
int check_span(int64_t blocks) {
  return blocks > 65535 ? fail(GEMM_ERR_UNSUPPORTED, "rows are too long for one launch") : GEMM_OK;
}

}  // namespace

static void scale_product(LayerPlan& pl, const float* scale) {
  if (!scale) return;
  pl.a.act = ACT_SCALE;
  pl.a.scale = scale;
}

int run_dense(const DenseCall& c, bool launch, hipStream_t s) {
  LayerPlan pl;
  bool noop;
  CHECK(plan_product(-1, c.M, c.N, c.K, c.dtype, c.ta, c.tb, nullptr, c.A, c.lda, c.B, c.ldb, 0,
                     nullptr, GEMM_ACT_NONE, c.R, c.ldr, c.Y, c.ldy, c.out_dtype, nullptr, 0, pl, noop,
                     false));
  scale_product(pl, c.scale);
  return noop || !launch ? GEMM_OK : launched(launch_product(pl, s));
}

int run_sums(const SumsCall& c, bool launch, hipStream_t s) {
  LayerPlan pl;
  bool noop;
  CHECK(plan_grad_weight(c.G, c.M, c.N, c.K, c.dtype, c.offsets, c.A, c.lda, c.B, c.ldb, c.D, c.ldd, c.stride_d,
                         c.out_dtype, c.accumulate, pl, noop, false));
  scale_product(pl, c.scale);
  return noop || !launch ? GEMM_OK : launched(launch_product(pl, s));
}

}  // namespace dgt

using namespace dgt;

extern "C" {

int gemm_linear(int64_t M, int64_t N, int64_t K, int dtype, int transA, int transB, const void* A,
                int64_t lda, const void* B, int64_t ldb, const void* bias, int act, const void* R,
                int64_t ldr, void* Y, int64_t ldy, int out_dtype, void* Z, int64_t ldz,
                void* stream) {
  return entry("linear", M, N, K, [&] {
    LayerPlan pl;
    bool noop;
    CHECK(plan_product(-1, M, N, K, dtype, transA, transB, nullptr, A, lda, B, ldb, 0, bias, act, R,
                       ldr, Y, ldy, out_dtype, Z, ldz, pl, noop));
    return noop ? GEMM_OK : launched(launch_product(pl, static_cast<hipStream_t>(stream)));
  });
}

int gemm_linear_validate(int64_t M, int64_t N, int64_t K, int dtype, int transA, int transB,
                         const void* A, int64_t lda, const void* B, int64_t ldb, const void* bias,
                         int act, const void* R, int64_t ldr, const void* Y, int64_t ldy,
                         int out_dtype, const void* Z, int64_t ldz) {
  return entry("linear", M, N, K, [&] {
    LayerPlan pl;
    bool noop;
    return plan_product(-1, M, N, K, dtype, transA, transB, nullptr, A, lda, B, ldb, 0, bias, act,
                        R, ldr, Y, ldy, out_dtype, Z, ldz, pl, noop);
  });
}

int gemm_grouped(int64_t G, int64_t M, int64_t N, int64_t K, int dtype, int transB,
                 const int32_t* offsets, const void* A, int64_t lda, const void* B, int64_t ldb,
                 int64_t stride_b, const void* bias, int act, const void* R, int64_t ldr, void* Y,
                 int64_t ldy, int out_dtype, void* Z, int64_t ldz, void* stream) {
  return entry("grouped", M, N, K, [&] {
    LayerPlan pl;
    bool noop;
    CHECK(check_groups(G));
    CHECK(plan_product(G, M, N, K, dtype, 0, transB, offsets, A, lda, B, ldb, stride_b, bias, act,
                       R, ldr, Y, ldy, out_dtype, Z, ldz, pl, noop));
    return noop ? GEMM_OK : launched(launch_product(pl, static_cast<hipStream_t>(stream)));
  });
}

int gemm_grouped_validate(int64_t G, int64_t M, int64_t N, int64_t K, int dtype, int transB,
                          const int32_t* offsets, const void* A, int64_t lda, const void* B,
                          int64_t ldb, int64_t stride_b, const void* bias, int act, const void* R,
                          int64_t ldr, const void* Y, int64_t ldy, int out_dtype, const void* Z,
                          int64_t ldz) {
  return entry("grouped", M, N, K, [&] {
    LayerPlan pl;
    bool noop;
    CHECK(check_groups(G));
    return plan_product(G, M, N, K, dtype, 0, transB, offsets, A, lda, B, ldb, stride_b, bias, act,
                        R, ldr, Y, ldy, out_dtype, Z, ldz, pl, noop);
  });
}

int gemm_grouped_grad_weight(int64_t G, int64_t M, int64_t N, int64_t K, int dtype,
                             const int32_t* offsets, const void* A, int64_t lda, const void* B,
                             int64_t ldb, void* D, int64_t ldd, int64_t stride_d, int out_dtype,
                             int accumulate, void* stream) {
  return entry("grad_weight", M, N, K, [&] {
    LayerPlan pl;
    bool noop;
    CHECK(check_groups(G));
    CHECK(plan_grad_weight(G, M, N, K, dtype, offsets, A, lda, B, ldb, D, ldd, stride_d, out_dtype,
                           accumulate, pl, noop));
    return noop ? GEMM_OK : launched(launch_product(pl, static_cast<hipStream_t>(stream)));
  });
}

int gemm_grouped_grad_weight_validate(int64_t G, int64_t M, int64_t N, int64_t K, int dtype,
                                      const int32_t* offsets, const void* A, int64_t lda,
                                      const void* B, int64_t ldb, const void* D, int64_t ldd,
                                      int64_t stride_d, int out_dtype, int accumulate) {
  return entry("grad_weight", M, N, K, [&] {
    LayerPlan pl;
    bool noop;
    CHECK(check_groups(G));
    return plan_grad_weight(G, M, N, K, dtype, offsets, A, lda, B, ldb, D, ldd, stride_d, out_dtype,
                            accumulate, pl, noop);
  });
}

int64_t gemm_act_grad_workspace(int64_t G, int64_t M, int64_t N) { return act_grad_bytes(G, M, N); }

int gemm_act_grad(int64_t G, int64_t M, int64_t N, int dtype, int act, const int32_t* offsets,
                  const void* dY, int64_t lddy, const void* Z, int64_t ldz, void* dZ, int64_t lddz,
                  float* db, void* workspace, int64_t workspace_bytes, void* stream) {
  return entry("act_grad", M, N, 0, [&]() -> int {
    CHECK(check_groups(G));
    CHECK(check_dim("M", M));
    CHECK(check_dim("N", N));
    CHECK(check_dtype16(dtype));
    CHECK(check_act(act));
    if (!offsets && G != 1)
      return bad("%s is NULL with %lld groups", "offsets", G);
    if (act == GEMM_ACT_NONE) Z = nullptr;
    const Mat my{"dY", dY, M, N, lddy, 2}, mz{"Z", Z, M, N, ldz, 2}, md{"dZ", dZ, M, N, lddz, 2};
    const Mat mb{"db", db, G, N, N, 4}, moff{"offsets", offsets, 1, G + 1, G + 1, 4};
    const int64_t need = db ? act_grad_bytes(G, M, N) : 0;
    const Mat mw{"workspace", db ? workspace : nullptr, 1, need, need, 1};
    CHECK(check_ld(my));
    if (act != GEMM_ACT_NONE) CHECK(check_ld(mz));
    if (dZ) CHECK(check_ld(md));
    if (N == 0 || G == 0 || (M == 0 && !db) || (!dZ && !db)) {
      set_path("noop: empty output");
      return GEMM_OK;
    }
    if (M > 0) {
      CHECK(check_ptr(my));
      if (act != GEMM_ACT_NONE) CHECK(check_ptr(mz));
      if (dZ) CHECK(check_ptr(md));
    }
    if (db) {
      CHECK(check_ptr(mb));
      if (need == 0 && M > 0) return fail(GEMM_ERR_UNSUPPORTED, "the workspace would be too large");
      CHECK(check_workspace(workspace, workspace_bytes, need));
    }
    if (offsets) CHECK(check_ptr(moff));
    const Mat* reads[] = {&my, &mz, &moff};
    const Mat* writes[] = {&md, &mb, &mw};
    for (const Mat* w : writes)
      for (const Mat* r : reads)
        CHECK(w == &md && r != &moff ? check_apart_or_same(*w, *r) : check_apart(*w, *r));
    CHECK(check_apart(md, mb));
    CHECK(check_apart(md, mw));
    CHECK(check_apart(mb, mw));
    if (act_grad_waves(M, N) > 0x7ffffff0)
      return fail(GEMM_ERR_UNSUPPORTED, "too many pieces of rows for one launch");
    ActGradArgs a{};
    a.offsets = offsets;
    a.dY = dY;
    a.Z = Z;
    a.dZ = dZ;
    a.db = db;
    a.part = static_cast<float*>(workspace);
    a.lddy = lddy;
    a.ldz = ldz;
    a.lddz = lddz;
    a.G = (int)G;
    a.M = (int)M;
    a.N = (int)N;
    a.act = act;
    a.rows = act_grad_rows(M, N);
    set_path(std::string("act_grad act=") + kActNames[act] + (dZ ? " dz" : "") + (db ? " db" : ""));
    return launched(launch_act_grad(dtype, a, static_cast<hipStream_t>(stream)));
  });
}

int64_t gemm_route_workspace(int64_t T, int64_t top, int64_t E) { return route_bytes(T, top, E); }

int gemm_route(int64_t T, int64_t top, int64_t E, const int32_t* ids, int32_t* offsets,
               int32_t* order, int32_t* slot, void* workspace, int64_t workspace_bytes,
               void* stream) {
  return entry("route", T, top, E, [&]() -> int {
    CHECK(check_choices(T, top));
    if (E < 0) return bad("negative number of experts: %s=%lld", "E", E);
    if (E > kRouteMaxExperts) return fail(GEMM_ERR_UNSUPPORTED, "more than 1024 experts");
    const int64_t n = T * top, need = route_bytes(T, top, E);
    const Mat mi{"ids", ids, 1, n, n, 4}, mo{"offsets", offsets, 1, E + 1, E + 1, 4};
    const Mat mr{"order", order, 1, n, n, 4}, ms{"slot", slot, 1, n, n, 4};
    const Mat mw{"workspace", need ? workspace : nullptr, 1, need, need, 1};
    CHECK(check_ptr(mo));
    if (n > 0) {
      CHECK(check_ptr(mi));
      CHECK(check_ptr(mr));
      CHECK(check_ptr(ms));
    }
    CHECK(check_workspace(workspace, workspace_bytes, need));
    const Mat* all[] = {&mi, &mo, &mr, &ms, &mw};
    for (int i = 0; i < 5; ++i)
      for (int j = i + 1; j < 5; ++j) CHECK(check_apart(*all[j], *all[i]));
    RouteArgs a{};
    a.ids = ids;
    a.offsets = offsets;
    a.order = order;
    a.slot = slot;
    a.counts = static_cast<int*>(workspace);
    a.n = (int)n;
    a.E = (int)E;
    route_blocks(n, a.blocks, a.chunk);
    set_path(a.blocks > 1 ? "route counted and placed by blocks" : "route in one block");
    return launched(launch_route(a, static_cast<hipStream_t>(stream)));
  });
}

int gemm_dispatch(int64_t T, int64_t top, int64_t H, int dtype, const void* X, int64_t ldx,
                  const int32_t* slot, void* Xs, int64_t ldxs, void* stream) {
  return entry("dispatch", T, top, H, [&]() -> int {
    int rowtype, elem;
    CHECK(check_choices(T, top));
    CHECK(check_dim("H", H));
    CHECK(check_rowtype(dtype, rowtype, elem));
    const int64_t n = T * top;
    const Mat mx{"X", X, T, H, ldx, elem}, ms{"slot", slot, 1, n, n, 4},
        mo{"Xs", Xs, n, H, ldxs, elem};
    CHECK(check_ld(mx));
    CHECK(check_ld(mo));
    if (n == 0 || H == 0) {
      set_path("noop: empty output");
      return GEMM_OK;
    }
    CHECK(check_ptr(mx));
    CHECK(check_ptr(ms));
    CHECK(check_ptr(mo));
    CHECK(check_apart(mo, mx));
    CHECK(check_apart(mo, ms));
    DispatchArgs a{};
    a.X = static_cast<const char*>(X);
    a.Xs = static_cast<char*>(Xs);
    a.slot = slot;
    a.ldx = ldx * elem;
    a.ldxs = ldxs * elem;
    a.T = (int)T;
    a.top = (int)top;
    a.bytes = H * elem;
    const Mat* mats[] = {&mx, &mo};
    a.piece = common_piece(H, elem, mats) * elem;
    CHECK(check_span(dispatch_column_blocks(a)));
    set_path("dispatch in pieces of " + std::to_string(a.piece) + " bytes");
    return launched(launch_dispatch(a, static_cast<hipStream_t>(stream)));
  });
}

int gemm_combine(int64_t T, int64_t top, int64_t H, int dtype, const void* Ys, int64_t ldys,
                 const int32_t* slot, const float* weights, const void* R, int64_t ldr, void* Y,
                 int64_t ldy, void* stream) {
  return entry("combine", T, top, H, [&]() -> int {
    int rowtype, elem;
    CHECK(check_choices(T, top));
    CHECK(check_dim("H", H));
    CHECK(check_rowtype(dtype, rowtype, elem));
    const int64_t n = T * top;
    const Mat mi{"Ys", Ys, n, H, ldys, elem}, ms{"slot", slot, 1, n, n, 4},
        mw{"weights", weights, 1, n, n, 4};
    const Mat mr{"R", R, T, H, ldr, elem}, my{"Y", Y, T, H, ldy, elem};
    CHECK(check_ld(mi));
    if (R) CHECK(check_ld(mr));
    CHECK(check_ld(my));
    if (T == 0 || H == 0) {
      set_path("noop: empty output");
      return GEMM_OK;
    }
    CHECK(check_ptr(my));
    if (n > 0) {
      CHECK(check_ptr(mi));
      CHECK(check_ptr(ms));
      if (weights) CHECK(check_ptr(mw));
    }
    if (R) CHECK(check_ptr(mr));
    CHECK(check_apart(my, mi));
    CHECK(check_apart(my, ms));
    CHECK(check_apart(my, mw));
    CHECK(check_apart_or_same(my, mr));
    CombineArgs a{};
    a.Ys = Ys;
    a.slot = slot;
    a.weights = weights;
    a.R = R;
    a.Y = Y;
    a.ldys = ldys;
    a.ldr = ldr;
    a.ldy = ldy;
    a.T = (int)T;
    a.top = (int)top;
    a.H = (int)H;
    const Mat* mats[] = {&mi, &mr, &my};
    a.piece = common_piece(H, elem, mats);
    a.once = n * H * elem >= (int64_t{128} << 20);
    if (combine_waves(a) > 0x7ffffff0)
      return fail(GEMM_ERR_UNSUPPORTED, "too many pieces of rows for one launch");
    set_path("combine in pieces of " + std::to_string(a.piece * elem) + " bytes");
    return launched(launch_combine(rowtype, a, static_cast<hipStream_t>(stream)));
  });
}

int gemm_combine_grad(int64_t T, int64_t top, int64_t H, int dtype, const void* dY, int64_t lddy,
                      const void* Ys, int64_t ldys, const int32_t* slot, const float* weights,
                      void* dYs, int64_t lddys, float* dweights, void* stream) {
  return entry("combine_grad", T, top, H, [&]() -> int {
    int rowtype, elem;
    CHECK(check_choices(T, top));
    CHECK(check_dim("H", H));
    CHECK(check_rowtype(dtype, rowtype, elem));
    const int64_t n = T * top;
    if (!dweights) Ys = nullptr;
    const Mat mdy{"dY", dY, T, H, lddy, elem}, mi{"Ys", Ys, n, H, ldys, elem};
    const Mat ms{"slot", slot, 1, n, n, 4}, mw{"weights", weights, 1, n, n, 4};
    const Mat mo{"dYs", dYs, n, H, lddys, elem}, mdw{"dweights", dweights, 1, n, n, 4};
    CHECK(check_ld(mdy));
    if (dweights) CHECK(check_ld(mi));
    if (dYs) CHECK(check_ld(mo));
    if (n == 0 || (H == 0 && !dweights) || (!dYs && !dweights)) {
      set_path("noop: empty output");
      return GEMM_OK;
    }
    if (H > 0) {
      CHECK(check_ptr(mdy));
      if (dweights) CHECK(check_ptr(mi));
      if (dYs) CHECK(check_ptr(mo));
    }
    CHECK(check_ptr(ms));
    if (weights) CHECK(check_ptr(mw));
    if (dweights) CHECK(check_ptr(mdw));
    CHECK(check_apart_or_same(mo, mi));
    CHECK(check_apart(mo, mdy));
    CHECK(check_apart(mo, ms));
    CHECK(check_apart(mo, mw));
    CHECK(check_apart(mdw, mdy));
    CHECK(check_apart(mdw, mi));
    CHECK(check_apart(mdw, ms));
    CHECK(check_apart(mdw, mw));
    CHECK(check_apart(mo, mdw));
    CombineGradArgs a{};
    a.dY = dY;
    a.Ys = Ys;
    a.slot = slot;
    a.weights = weights;
    a.dYs = dYs;
    a.dw = dweights;
    a.lddy = lddy;
    a.ldys = ldys;
    a.lddys = lddys;
    a.T = (int)T;
    a.top = (int)top;
    a.H = (int)H;
    const Mat* mats[] = {&mdy, &mi, &mo};
    a.piece = common_piece(H, elem, mats);
    set_path("combine_grad in pieces of " + std::to_string(a.piece * elem) + " bytes");
    return launched(launch_combine_grad(rowtype, a, static_cast<hipStream_t>(stream)));
  });
}

}  // extern "C"
