// The layer operators' product for few rows (A stored [M][K]): decoding
// batches, and the handful of rows that each of many experts gets. Bound by
// the weights' bytes, so the point is to have enough of them in flight.
//
// A workgroup owns 16*MT rows and 16*NT columns; its KW waves split K: wave w
// takes slices w, w + KW, ... of 64 (whole 128-byte lines of a row stored
// along K), so the workgroup walks consecutive memory and no two waves share
// an operand byte. There is no barrier in the loop and no LDS round trip for
// operands stored along K: fragments are loaded into registers, D slices
// ahead, with buffer loads whose offsets are out of range (read as zeros, not
// fetched) past M, N and K. B stored [K][N] is loaded straight into this
// wave's own LDS, D slices ahead as well, and read transposed.
//
// The waves' sums meet in LDS and are added in wave order.
#include "gemm_mfma_pingpong.h"
#include "layer.h"

namespace dgt {

namespace {

using At16 = Atom<16>;

// No memory operation crosses, neither in the compiler's view nor in its
// schedule: loads that a wait counts have to be issued in the order written.
__device__ __forceinline__ void layer_fixed_order() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

template <int MT_, int NT_, int D_, int KW_, bool BMN>
struct SkinnyCfg {
  static constexpr int MT = MT_, NT = NT_, KW = KW_;
  static constexpr int BM = 16 * MT, BN = 16 * NT, BK = 64, THREADS = KW * 64;
  static constexpr int D = D_;                  // slices in flight
  static constexpr int PITCH = BN + 4;          // floats of an output row
  static constexpr int B_SLICE = BK * BN * 2;   // LDS bytes of a slice of B stored [K][N]
  static constexpr int B_BYTES = BMN ? KW * D * B_SLICE : 0;
  static constexpr int SUM_BYTES = KW * MT * NT * 1024;  // every wave's accumulators
  static constexpr int OUT_BYTES = BM * PITCH * 4;
  static constexpr int LDS_BYTES = (B_BYTES > SUM_BYTES ? B_BYTES : SUM_BYTES) + OUT_BYTES;
  static_assert(LDS_BYTES <= 160 * 1024, "gfx950 has 160 KiB of LDS per workgroup");
  static_assert(!BMN || NT == 2 || NT == 4, "B stored [K][N] is laid out in 64- or 128-byte rows");
};

// A resource's record count: `rows` rows of a matrix, the last one cut after
// `cols` elements.
__device__ __forceinline__ unsigned skinny_records(int64_t rows, int64_t ld, int64_t cols) {
  const int64_t n = 2 * ((rows - 1) * ld + cols);
  return n > 0x7FFFFFFC ? 0x7FFFFFFCu : (rows <= 0 || n <= 0 ? 0u : (unsigned)n);
}

// s_waitcnt vmcnt(n * LOADS) for a run-time n (0..3 are told apart).
template <int LOADS>
__device__ __forceinline__ void skinny_wait(int n) {
  layer_fixed_order();
  if (n >= 3) pp_wait_vm<3 * LOADS>();
  else if (n == 2) pp_wait_vm<2 * LOADS>();
  else if (n == 1) pp_wait_vm<LOADS>();
  else pp_wait_vm<0>();
  layer_fixed_order();
}

// A slice of B stored [K][N]: 64 K rows of 16 NT columns (32 NT bytes) in LDS.
// Chunk c (8 columns) of row r sits at chunk c ^ swz(r), so that the rows 0-3
// and 8-11 that 32 lanes of a transposed read name lie in different banks.
template <int NT>
struct SkinnyRows {
  static constexpr int RB = 32 * NT;             // bytes of a row
  static constexpr int CPR = 2 * NT;             // chunks of a row
  static constexpr int RPI = 64 / CPR;           // rows an instruction fills
  static constexpr int LOADS = 64 / RPI;
  __device__ static __forceinline__ int swz(int r) {
    return NT == 2 ? 2 * ((r >> 3) & 1) : 2 * (((r >> 1) & 1) | ((r >> 2) & 2));
  }
  // Columns left from X (the tile's first), K rows left from the slice's.
  __device__ static __forceinline__ void request(const char* X, int64_t ld, int rows, int cols,
                                                 int slice, char* lds, int lane) {
    // The slice's first row goes into the resource base: 32-bit offsets within
    // 64 rows.
    const char* base = X + (int64_t)slice * 64 * ld * 2;
    const auto rs = make_rsrc_n(base, skinny_records(rows, ld, cols));
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int r = RPI * i + lane / CPR, c = (lane % CPR) ^ swz(r);
      const int off = r < rows && 8 * c < cols ? (int)(r * ld * 2) + c * 16 : kOutOfRange;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (pp_lds_ptr_t)(lds + i * 1024), 16, off, 0, 0, 0);
    }
  }
  // The fragment of columns 16 n .. +15, K rows 32 h .. +31. The second read is
  // 4 rows down, which swz() does not see.
  __device__ static __forceinline__ u32x4 read(const char* lds, int n, int h, int lane) {
    typedef __attribute__((address_space(3))) pp_i16x4 lds_i16x4;
    const int r = 8 * (lane >> 4) + ((lane & 15) >> 2);
    const int c = (2 * n + ((lane & 3) >> 1)) ^ swz(r);
    const char* x = lds + (r + 32 * h) * RB + c * 16 + (lane & 1) * 8;
    const pp_i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(x));
    const pp_i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(x + 4 * RB));
    const u32x2 l2 = __builtin_bit_cast(u32x2, lo), h2 = __builtin_bit_cast(u32x2, hi);
    return u32x4{l2.x, l2.y, h2.x, h2.y};
  }
};

template <class Tag, int MODE, bool BMN, int MT, int NT, int D, int KW>
__global__ void __launch_bounds__(KW * 64) layer_skinny_kernel(const LayerArgs p) {
  using C = SkinnyCfg<MT, NT, D, KW, BMN>;
  using Rows = SkinnyRows<NT == 1 ? 2 : NT>;
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS_BYTES];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int total = layer_tiles<MODE, C::BM>(p, lane);
  if ((int)blockIdx.x >= total) return;  // by rows the grid is an upper bound
  const LayerTile q = layer_tile<MODE, C::BM, C::BN>(p, blockIdx.x, total, lane);

  // Resources end at the last byte of the operand's last row here, so no offset
  // below 2^31 reads past it.
  const char* Ab = q.A + (int64_t)q.m0 * p.lda * 2;
  const auto ra = make_rsrc_n(Ab, skinny_records(q.M - q.m0, p.lda, q.K));
  // This lane's piece of a slice stored along K: row l%16 of an atom, K values
  // 8 (l/16) .. +7 of each half of 32.
  const int r16 = lane & 15, kl = 8 * (lane >> 4);
  int arow[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = 16 * i + r16;
    arow[i] = q.m0 + r < q.M ? (int)(r * p.lda * 2) : kOutOfRange;
  }
  auto along_k = [&](const __amdgpu_buffer_rsrc_t& rs, int row, int k) {
    const int off = row != kOutOfRange && k < q.K ? row + k * 2 : kOutOfRange;
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
  };

  const char* Bb = BMN ? q.B + (int64_t)q.n0 * 2 : q.B + (int64_t)q.n0 * p.ldb * 2;
  const auto rb = make_rsrc_n(Bb, BMN ? skinny_records(q.K, p.ldb, q.N - q.n0)
                                      : skinny_records(q.N - q.n0, p.ldb, q.K));
  int brow[NT];
  if constexpr (!BMN) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int n = 16 * j + r16;
      brow[j] = q.n0 + n < q.N ? (int)(n * p.ldb * 2) : kOutOfRange;
    }
  }
  char* const bl = smem + w * D * C::B_SLICE;
  // Column tiles start at different slices and walk around: workgroups that
  // all read the same part of rows a power of two apart would meet in few
  // memory channels. Row tiles of one column tile walk alike and share B.
  const int KT = (q.K + 63) / 64;
  const int rot =
      (int)(((uint64_t)((unsigned)(q.n0 / C::BN) * 0x9E3779B1u) * (unsigned)KT) >> 32);
  auto place = [&](int s) { return s + rot >= KT ? s + rot - KT : s + rot; };
  auto request_b = [&](int s, int d) {
    const int slice = place(s);
    if constexpr (BMN)
      Rows::request(Bb, p.ldb, q.K - slice * 64, q.N - q.n0, slice, bl + d * C::B_SLICE, lane);
  };

  At16::acc_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][j][v] = 0.0f;

  u32x4 fa[D][MT][2], fb[D][NT][2];
  const int NJ = KT > w ? (KT - w + KW - 1) / KW : 0;  // this wave's slices
  auto load = [&](int d, int j) {
    const int slice = place(j * KW + w);
    if constexpr (!BMN) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) fb[d][n][h] = along_k(rb, brow[n], slice * 64 + 32 * h + kl);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) fa[d][i][h] = along_k(ra, arow[i], slice * 64 + 32 * h + kl);
  };
  auto multiply = [&](int d) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
          acc[i][n] = At16::mma(Tag{}, fa[d][i][h], fb[d][n][h], acc[i][n]);
  };
  // Slices beyond NJ are not asked for: even loads that fetch nothing take
  // their time in the address units (64 bytes a clock and CU).
  auto request = [&](int d, int j) {
    request_b(j * KW + w, d);
    if constexpr (BMN) layer_fixed_order();
    load(d, j);
    if constexpr (BMN) layer_fixed_order();
  };
  // Slice j (in place d), while `younger` slices asked for after it may stay in
  // flight.
  auto step = [&](int d, int younger) {
    if constexpr (BMN) {
      skinny_wait<Rows::LOADS + 2 * MT>(younger);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) fb[d][n][h] = Rows::read(bl + d * C::B_SLICE, n, h, lane);
      pp_wait_lgkm0();  // read before the slot is filled again
      layer_fixed_order();
    }
    multiply(d);
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < NJ) request(d, d);
  int j = 0;
  for (; j + 2 * D <= NJ; j += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      step(d, D - 1);
      request(d, j + d + D);
    }
  }
  // At most 2 D - 1 slices are left, D of them in flight.
#pragma unroll
  for (int d = 0; d < D; ++d) {
    const int left = NJ - 1 - (j + d);  // slices after this one
    if (left >= 0) step(d, left < D - 1 ? left : D - 1);
    if (left >= D) request(d, j + d + D);
  }
  j += D;
#pragma unroll
  for (int d = 0; d < D - 1; ++d) {
    const int left = NJ - 1 - (j + d);
    if (left >= 0) step(d, left);
  }

  // Sums of the waves, in wave order; one output a thread and round.
  if constexpr (BMN) __syncthreads();  // the sums overlay the slices
  float* sums = reinterpret_cast<float*>(smem);
  float* outs = reinterpret_cast<float*>(smem + C::LDS_BYTES - C::OUT_BYTES);
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        sums[((w * MT + i) * NT + n) * 256 + v * 64 + lane] = acc[i][n][v];
  __syncthreads();
  constexpr int VALUES = MT * NT * 256;
  for (int x = tid; x < VALUES; x += C::THREADS) {
    float s = sums[x];
#pragma unroll
    for (int u = 1; u < KW; ++u) s += sums[u * VALUES + x];
    const int ln = x & 63, v = (x >> 6) & 3, at = x >> 8;
    outs[(16 * (at / NT) + At16::acc_row(ln, v)) * C::PITCH + 16 * (at % NT) + At16::acc_col(ln)] = s;
  }
  __syncthreads();
  for (int x = tid; x < C::BM * (C::BN / 8); x += C::THREADS) {
    const int rr = x / (C::BN / 8), cl = 8 * (x % (C::BN / 8));
    const int r = q.m0 + rr, c = q.n0 + cl, nv = q.N - c >= 8 ? 8 : q.N - c;
    if (r < q.M && nv > 0) {
      float bias[8], v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        bias[e] = 0.0f;
        v[e] = outs[rr * C::PITCH + cl + e];
      }
      if (q.bias) layer_load8_16<Tag>(q.bias + (int64_t)c * 2, p.vec & VEC_BIAS, nv, bias);
      layer_finish8<Tag>(p, q, r, c, nv, bias, v);
    }
  }
}

template <class Tag, int MODE, bool BMN, int MT, int NT, int D>
hipError_t launch(const LayerArgs& a, int ntiles, hipStream_t s) {
  constexpr int KW = 8;
  return launch_kernel(layer_skinny_kernel<Tag, MODE, BMN, MT, NT, D, KW>, dim3(ntiles), dim3(KW * 64), s, a);
}
template <class Tag, int MODE>
hipError_t launch_form(bool tb, int mt, int nt, const LayerArgs& a, int ntiles, hipStream_t s) {
  if (!tb) {
    if (mt == 1) return launch<Tag, MODE, true, 1, 2, 4>(a, ntiles, s);
    if (mt == 2) return launch<Tag, MODE, true, 2, 2, 4>(a, ntiles, s);
    if (nt == 2) return launch<Tag, MODE, true, 4, 2, 4>(a, ntiles, s);
    return launch<Tag, MODE, true, 4, 4, 2>(a, ntiles, s);
  }
  if (nt == 1) return launch<Tag, MODE, false, 1, 1, 8>(a, ntiles, s);
  if (mt == 1) return launch<Tag, MODE, false, 1, 2, 4>(a, ntiles, s);
  if (mt == 2) return launch<Tag, MODE, false, 2, 2, 4>(a, ntiles, s);
  if (mt == 3) return launch<Tag, MODE, false, 3, 2, 4>(a, ntiles, s);
  if (nt == 2) return launch<Tag, MODE, false, 4, 2, 4>(a, ntiles, s);
  return launch<Tag, MODE, false, 4, 4, 2>(a, ntiles, s);
}
template <class Tag>
hipError_t launch_mode(bool tb, int mt, int nt, const LayerArgs& a, int ntiles, hipStream_t s) {
  return a.mode == LAYER_ROWS ? launch_form<Tag, LAYER_ROWS>(tb, mt, nt, a, ntiles, s)
                              : launch_form<Tag, LAYER_DENSE>(tb, mt, nt, a, ntiles, s);
}

}  // namespace

hipError_t launch_layer_skinny(int dtype, bool tb, int mt, int nt, const LayerArgs& a, int ntiles,
                               hipStream_t s) {
  if (dtype == 0) return launch_mode<TagF16>(tb, mt, nt, a, ntiles, s);
  return launch_mode<TagBF16>(tb, mt, nt, a, ntiles, s);
}

}  // namespace dgt
