// Products with 4-bit weights: Y = act(A @ W^T + bias) + R, where
//   W[n][k] = s[n][j] (code[n][k] - z[n][j]),  j = k / group.
//
// The matrix cores take 16-bit operands, and a code becomes one without an
// arithmetic operation: its four bits, placed below the leading bit of 16.0, are the
// number 16 + code, exactly, in both types. So for every group
//   sum over k of A[m][k] (code - z) = P - (16 + z) S,  P = sum A (16 + code),  S = sum A,
// P and S from matrix instructions (S against ones), the rest in float32: no weight
// is rounded to 16 bits. 16 and not the type's larger powers of two, since P and
// (16 + z) S cancel by that factor.
//
// A pair of codes k and k + 4 of a 32-bit word goes to one register with one shift
// and one and-or; A's values are brought into that order instead.
#include "layer_split.h"
#include "layer_checks.h"

namespace dgt {

namespace {

struct W4Args {
  LayerArgs a;  // B: codes; ldb, stride_b: bytes
  const void* scales;
  const void* zeros;   // null: 8
  int64_t lds, stride_s;
  int group;
};

typedef u32x4 u32x4_at1 __attribute__((aligned(1)));
typedef unsigned u32_at1 __attribute__((aligned(1)));

template <class Tag>
struct W4Type;
template <>
struct W4Type<TagBF16> {
  static constexpr unsigned BASE = 0x41804180u, MASK = 0x00780078u, ONES = 0x3F803F80u;
  static constexpr int AT = 3;  // the place of a code's lowest bit
};
template <>
struct W4Type<TagF16> {
  static constexpr unsigned BASE = 0x4C004C00u, MASK = 0x03C003C0u, ONES = 0x3C003C00u;
  static constexpr int AT = 6;
};

// Eight codes as the 16-bit numbers 16 + code, in the order 0 4 1 5 2 6 3 7.
template <class Tag>
__device__ __forceinline__ u32x4 w4_codes(unsigned q) {
  using T = W4Type<Tag>;
  u32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int right = 4 * j - T::AT;
    v[j] = ((right > 0 ? q >> (right > 0 ? right : 0) : q << (right > 0 ? 0 : -right)) & T::MASK) | T::BASE;
  }
  return v;
}
// Eight 16-bit values in that order.
__device__ __forceinline__ u32x4 w4_order(u32x4 x) {
  return u32x4{__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
               __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
}

// A workgroup's tile: its group's rows, weights and outputs. g: the group.
template <int MODE, int BM, int BN>
__device__ __forceinline__ LayerTile w4_tile(const LayerArgs& p, int t, int total, int lane, int& g) {
  LayerTile q;
  const int osz = p.out32 ? 4 : 2, lid = xcd_remap(t, total);
  int tm, tn, first = 0, count = p.M, tiles_m = p.tiles_m, in = lid;
  g = 0;
  if constexpr (MODE == LAYER_ROWS) {
    g = LayerRows<BM>::find(p, lid, p.tiles_n, lane, first, count, in);
    tiles_m = (count + BM - 1) / BM;
    if (in < 0 || in >= (int64_t)tiles_m * p.tiles_n) {  // whatever the offsets hold
      in = count = 0;
      tiles_m = 1;
    }
  }
  grouped_tile(in, tiles_m, p.tiles_n, p.group_m, tm, tn);
  q.A = static_cast<const char*>(p.A) + (int64_t)first * p.lda * 2;
  q.B = static_cast<const char*>(p.B) + (int64_t)g * p.stride_b;
  q.bias = static_cast<const char*>(p.bias);
  if (q.bias) q.bias += (int64_t)g * p.N * 2;
  q.R = static_cast<const char*>(p.R);
  if (q.R) q.R += (int64_t)first * p.ldr * osz;
  q.Y = static_cast<char*>(p.Y) + (int64_t)first * p.ldy * osz;
  q.Z = nullptr;
  q.M = count;
  q.N = p.N;
  q.K = p.K;
  q.m0 = tm * BM;
  q.n0 = tn * BN;
  return q;
}

// Eight values of a row from element k on, zeros past K.
__device__ __forceinline__ u32x4 w4_values(const char* row, int k, int K) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (k + 8 <= K) return *reinterpret_cast<const u32x4_at2*>(row + (int64_t)k * 2);
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (k + e < K) v[e / 2] |= (unsigned)*reinterpret_cast<const unsigned short*>(row + (int64_t)(k + e) * 2) << (16 * (e % 2));
  return v;
}
// Eight codes of a row from code k (a multiple of 8) on, any value past K.
__device__ __forceinline__ unsigned w4_word(const char* row, int k, int K) {
  if (k + 8 <= K) return *reinterpret_cast<const u32_at1*>(row + k / 2);
  unsigned q = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (k + 2 * e < K) q |= (unsigned)(unsigned char)row[k / 2 + e] << (8 * e);
  return q;
}

template <class Tag, int MODE, int MT, int NT, int KW>
__global__ void __launch_bounds__(KW * 64) layer_w4_kernel(const W4Args p) {
  using At = SplitAtom;
  using Sum = SplitSum<MT, NT, KW>;
  __shared__ __attribute__((aligned(1024))) char smem[Sum::LDS_BYTES];
  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int total = layer_tiles<MODE, Sum::BM>(p.a, lane);
  if ((int)blockIdx.x >= total) return;  // by rows the grid is an upper bound
  int g;
  const LayerTile q = w4_tile<MODE, Sum::BM, Sum::BN>(p.a, blockIdx.x, total, lane, g);

  At::acc_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][n][v] = 0.0f;
  const int r16 = lane & 15, oct = lane >> 4;
  const char* scale[NT];
  const char* zero[NT];
  const char* codes[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    // (Columns past N repeat the last one; nothing of theirs is stored.)
    int col = q.n0 + 16 * n + r16;
    if (col >= q.N) col = q.N - 1;
    codes[n] = q.B + (int64_t)col * p.a.ldb;
    const int64_t at = ((int64_t)g * p.stride_s + (int64_t)col * p.lds) * 2;
    scale[n] = static_cast<const char*>(p.scales) + at;
    zero[n] = static_cast<const char*>(p.zeros) + at;
  }
  const u32x4 ones = {W4Type<Tag>::ONES, W4Type<Tag>::ONES, W4Type<Tag>::ONES, W4Type<Tag>::ONES};
  const At::acc_t none = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = 32 * w; k0 < q.K; k0 += 32 * KW) {
    u32x4 x[MT];
    At::acc_t sx[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      const int row = q.m0 + 16 * i + r16;
      x[i] = u32x4{0u, 0u, 0u, 0u};
      if (row < q.M) x[i] = w4_order(w4_values(q.A + (int64_t)row * p.a.lda * 2, k0 + 8 * oct, q.K));
      sx[i] = At::mma(Tag{}, x[i], ones, none);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const u32x4 c = w4_codes<Tag>(w4_word(codes[n], k0 + 8 * oct, q.K));
      const int j = k0 / p.group;
      const float s = layer_f32(Tag{}, reinterpret_cast<const unsigned short*>(scale[n])[j]);
      const float z = 16.0f + (p.zeros ? layer_f32(Tag{}, reinterpret_cast<const unsigned short*>(zero[n])[j]) : 8.0f);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const At::acc_t d = At::mma(Tag{}, x[i], c, none);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][n][v] = __builtin_fmaf(s, __builtin_fmaf(-z, sx[i][v], d[v]), acc[i][n][v]);
      }
    }
  }
  Sum::template finish<Tag>(acc, p.a, q, smem, tid, w);
}

template <class Tag, int MODE, int MT, int NT, int KW>
hipError_t launch(W4Args p, hipStream_t s) {
  using Sum = SplitSum<MT, NT, KW>;
  LayerArgs& a = p.a;
  a.tiles_m = (a.M + Sum::BM - 1) / Sum::BM;
  a.tiles_n = (a.N + Sum::BN - 1) / Sum::BN;
  a.group_m = 8;
  int64_t rows = a.tiles_m;
  if (MODE == LAYER_ROWS) {  // whatever the groups' sizes: each group's last tile may be cut short
    const int64_t g = a.G < a.M ? a.G : a.M;
    rows = ((int64_t)a.M + g * (Sum::BM - 1)) / Sum::BM;
  }
  const int64_t n = rows * a.tiles_n;
  return launch_kernel(layer_w4_kernel<Tag, MODE, MT, NT, KW>, dim3((unsigned)n), dim3(KW * 64), s, p);
}
template <class Tag, int MODE>
hipError_t launch_rows(const W4Args& p, hipStream_t s) {
  const int64_t rows = MODE == LAYER_ROWS ? ((int64_t)p.a.M + p.a.G - 1) / p.a.G : p.a.M;
  if (rows <= 16) return launch<Tag, MODE, 1, 1, 8>(p, s);
  if (rows <= 32) return launch<Tag, MODE, 2, 1, 8>(p, s);
  return launch<Tag, MODE, 4, 2, 8>(p, s);
}
hipError_t launch_w4(int dtype, const W4Args& p, hipStream_t s) {
  if (p.a.mode == LAYER_ROWS)
    return dtype == GEMM_DTYPE_F16 ? launch_rows<TagF16, LAYER_ROWS>(p, s) : launch_rows<TagBF16, LAYER_ROWS>(p, s);
  return dtype == GEMM_DTYPE_F16 ? launch_rows<TagF16, LAYER_DENSE>(p, s) : launch_rows<TagBF16, LAYER_DENSE>(p, s);
}

// Both entry points (G < 0: dense).
int run_w4(int64_t G, int64_t M, int64_t N, int64_t K, int dtype, const int32_t* offsets, const void* A, int64_t lda,
           const void* B, int64_t ldb, int64_t stride_b, const void* scales, const void* zeros, int64_t lds,
           int64_t stride_s, int64_t group, const void* bias, int act, const void* R, int64_t ldr, void* Y, int64_t ldy,
           int out_dtype, void* stream) {
  const bool dense = G < 0;
  CHECK(check_dim("M", M));
  CHECK(check_dim("N", N));
  CHECK(check_dim("K", K));
  CHECK(check_dtype16(dtype));
  CHECK(check_out_dtype(dtype, out_dtype));
  CHECK(check_act(act));
  if (group < 32 || group % 32) return bad("%s=%lld is not a multiple of 32", "group", group);
  const int osz = out_dtype == GEMM_DTYPE_F32 ? 4 : 2;
  const int64_t g = dense ? 1 : G, runs = (K + group - 1) / group;
  if (ldb % 2) return bad("%s=%lld is odd: a row of codes starts in a byte's lower half", "ldb", ldb);
  if (!dense && g > 1) {
    if (stride_b < 0 || stride_b % 2) return bad("%s=%lld is negative or odd", "stride_b", stride_b);
    if (stride_s < 0) return bad("%s is negative: %lld", "stride_s", stride_s);
  }
  const Mat ma{"A", A, M, K, lda, 2}, mb{"B", B, N, (K + 1) / 2, ldb / 2, 1, g, stride_b / 2};
  const Mat ms{"scales", scales, N, runs, lds, 2, g, stride_s}, mz{"zeros", zeros, N, runs, lds, 2, g, stride_s};
  const Mat mbias{"bias", bias, 1, N, N, 2, g, N};
  const Mat mr{"R", R, M, N, ldr, osz}, my{"Y", Y, M, N, ldy, osz};
  const Mat moff{"offsets", offsets, 1, g + 1, g + 1, 4};
  CHECK(check_ld(ma));
  if (ldb < (K > 1 ? K : 1)) return bad("leading dimension of %s is %lld, smaller than %lld", "B", ldb, K > 1 ? K : 1);
  CHECK(check_ld(ms));
  CHECK(check_ld(my));
  if (R) CHECK(check_ld(mr));
  if (M == 0 || N == 0 || g == 0) {
    set_path("noop: empty output");
    return GEMM_OK;
  }
  CHECK(check_ptr(my));
  if (K > 0) {
    for (const Mat* m : {&ma, &mb, &ms}) CHECK(check_ptr(*m));
    if (zeros) CHECK(check_ptr(mz));
    for (const Mat* m : {&ma, &mb, &ms, &mz}) CHECK(check_apart(my, *m));
  }
  if (bias) CHECK(check_ptr(mbias));
  if (R) CHECK(check_ptr(mr));
  CHECK(check_apart(my, mbias));
  CHECK(check_apart_or_same(my, mr));
  if (!dense) {
    CHECK(check_ptr(moff));
    CHECK(check_apart(my, moff));
  }
  // (A launch holds less than 2^32 threads; tiles are at least 16 x 16, and groups' last ones cut short.)
  const __int128 tiles = ((__int128)M / 16 + (g < M ? g : M) + 1) * ((N + 15) / 16);
  if (tiles > ((int64_t{1} << 32) - 1) / 512) return fail(GEMM_ERR_UNSUPPORTED, "too many output tiles for one launch");
  W4Args p{};
  LayerArgs& a = p.a;
  a.A = A;
  a.B = B;
  a.bias = bias;
  a.R = R;
  a.Y = Y;
  a.offsets = offsets;
  a.lda = lda;
  a.ldb = ldb / 2;
  a.ldr = ldr;
  a.ldy = ldy;
  a.stride_b = stride_b / 2;
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.G = (int)g;
  a.mode = dense ? LAYER_DENSE : LAYER_ROWS;
  a.act = act;
  a.out32 = osz == 4;
  p.scales = scales;
  p.zeros = zeros;
  p.lds = lds;
  p.stride_s = stride_s;
  p.group = (int)(group < kMaxDim ? group : kMaxDim / 32 * 32);
  set_path(dense ? "linear_w4" : "grouped_w4");
  return launched(launch_w4(dtype, p, static_cast<hipStream_t>(stream)));
}

}  // namespace
}  // namespace dgt

using namespace dgt;

extern "C" {

int gemm_linear_w4(int64_t M, int64_t N, int64_t K, int dtype, const void* A, int64_t lda, const void* B, int64_t ldb,
                   const void* scales, const void* zeros, int64_t lds, int64_t group, const void* bias, int act,
                   const void* R, int64_t ldr, void* Y, int64_t ldy, int out_dtype, void* stream) {
  return entry("linear_w4", M, N, K, [&] {
    return run_w4(-1, M, N, K, dtype, nullptr, A, lda, B, ldb, 0, scales, zeros, lds, 0, group, bias, act, R, ldr, Y,
                  ldy, out_dtype, stream);
  });
}

int gemm_grouped_w4(int64_t G, int64_t M, int64_t N, int64_t K, int dtype, const int32_t* offsets, const void* A,
                    int64_t lda, const void* B, int64_t ldb, int64_t stride_b, const void* scales, const void* zeros,
                    int64_t lds, int64_t stride_s, int64_t group, const void* bias, int act, const void* R, int64_t ldr,
                    void* Y, int64_t ldy, int out_dtype, void* stream) {
  return entry("grouped_w4", M, N, K, [&] {
    CHECK(check_groups(G));
    return run_w4(G, M, N, K, dtype, offsets, A, lda, B, ldb, stride_b, scales, zeros, lds, stride_s, group, bias, act,
                  R, ldr, Y, ldy, out_dtype, stream);
  });
}

}  // extern "C"
