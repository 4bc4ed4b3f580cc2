// The layer operators' product on tiles of up to 64 rows, the sum split over the
// workgroup's waves: decoding batches, and grids too small for larger tiles.
//
// A workgroup owns 16 MT rows and 16 NT columns; wave w takes slices w, w + KW,
// ... of 64 and loads their pieces of both operands straight into LDS of its
// own, D slices ahead: no barrier in the loop, and no two waves share an operand
// byte. Consecutive lanes load consecutive bytes (8 rows of 128 bytes of an
// operand stored along K, whole rows of the tile of B stored [K][N]); loading
// fragments into registers as layer_skinny.hip does puts neighbouring lanes into
// different rows, which takes the address units four times as long (48x8192x8192
// 44 us, 30 here).
#include "layer_split.h"

namespace dgt {

namespace {

// s_waitcnt vmcnt(n * LOADS) for a run-time n (0..3 are told apart).
template <int LOADS>
__device__ __forceinline__ void split_wait(int n) {
  layer_fixed_order();
  if (n >= 3) pp_wait_vm<3 * LOADS>();
  else if (n == 2) pp_wait_vm<2 * LOADS>();
  else if (n == 1) pp_wait_vm<LOADS>();
  else pp_wait_vm<0>();
  layer_fixed_order();
}

// A slice of an operand stored along K: 16 T rows of 64 K values, 128 bytes each
// in LDS. Chunk c (8 values) of row r sits at chunk c ^ swz(r), the conflict-free
// swizzle of gemm_mfma_pingpong.h's 16-wide atom.
template <int T>
struct SplitAlong {
  static constexpr int LOADS = 2 * T;
  using Op = PpOperand<false, T, 16>;
  // rs starts at the tile's first row; `rows` and `K` are left of the operand.
  __device__ static __forceinline__ void request(const __amdgpu_buffer_rsrc_t& rs, int ld2,
                                                 int rows, int K, int slice, char* lds, int lane) {
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int r = 8 * i + (lane >> 3), k = slice * 64 + 8 * ((lane & 7) ^ Op::swz(r));
      const int off = r < rows && k < K ? r * ld2 + k * 2 : kOutOfRange;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (pp_lds_ptr_t)(lds + i * 1024), 16, off, 0, 0, 0);
    }
  }
  // The fragment of rows 16 t .. +15, K values 32 h .. +31 of the slice.
  __device__ static __forceinline__ u32x4 read(const char* lds, int t, int h, int lane) {
    return *reinterpret_cast<const u32x4*>(
        lds + Op::lds_off(16 * t + SplitAtom::frag_row(lane), 4 * h + SplitAtom::frag_koct(lane)));
  }
};

// A slice of B stored [K][N]: 64 K rows of 16 NT columns (32 NT bytes) in LDS.
// Chunk c (8 columns) of row r sits at chunk c ^ swz(r), so that the rows 0-3
// and 8-11 that 32 lanes of a transposed read name lie in different banks.
template <int NT>
struct SplitRows {
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
    const auto rs = make_rsrc_n(base, split_records(rows, ld, cols));
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

template <class Tag, int MODE, bool AMN, bool BMN, int MT, int NT, int D, int KW>
__global__ void __launch_bounds__(KW * 64) layer_split_kernel(const LayerArgs p) {
  using At = SplitAtom;
  using Sum = SplitSum<MT, NT, KW>;
  using SA = SplitAlong<MT>;
  using SB = SplitAlong<NT>;
  using RA = SplitRows<MT == 2 ? 2 : 4>;  // (A stored [K][M]: 32 or 64 rows)
  using RB = SplitRows<NT == 1 ? 2 : NT>;  // (B stored [K][N]: not 16 columns)
  constexpr int A_SLICE = 2048 * MT, SLICE = A_SLICE + 2048 * NT;
  constexpr int LOADS = 2 * MT + 2 * NT;
  constexpr int BYTES = KW * D * SLICE > Sum::LDS_BYTES ? KW * D * SLICE : Sum::LDS_BYTES;
  static_assert(BYTES <= 160 * 1024, "gfx950 has 160 KiB of LDS per workgroup");
  static_assert(!BMN || (NT > 1 && RB::LOADS == SB::LOADS), "both forms of B take as many loads");
  static_assert(!AMN || MT == 2 || MT == 4, "A stored [K][M] is laid out in 64- or 128-byte rows");
  static_assert(D <= 4, "split_wait tells at most three slices apart");
  __shared__ __attribute__((aligned(1024))) char smem[BYTES];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int total = layer_tiles<MODE, Sum::BM>(p, lane);
  if ((int)blockIdx.x >= total) return;  // by rows the grid is an upper bound
  const LayerTile q = layer_tile<MODE, Sum::BM, Sum::BN>(p, blockIdx.x, total, lane);

  // Resources end at the last byte of the operand's last row here, so no offset
  // below 2^31 reads past it.
  const char* const Ab = AMN ? q.A + (int64_t)q.m0 * 2 : q.A + (int64_t)q.m0 * p.lda * 2;
  const auto ra = make_rsrc_n(Ab, split_records(q.M - q.m0, p.lda, q.K));  // (not AMN)
  const char* const Bb = BMN ? q.B + (int64_t)q.n0 * 2 : q.B + (int64_t)q.n0 * p.ldb * 2;
  const auto rb = make_rsrc_n(Bb, split_records(q.N - q.n0, p.ldb, q.K));  // (not BMN)

  At::acc_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][n][v] = 0.0f;

  const int KT = (q.K + 63) / 64;
  // (B stored [K][N]: neighbouring column tiles share lines, so all walk alike.)
  const int start = AMN || BMN ? 0 : split_start(q.n0 / Sum::BN, KT);
  const int NJ = KT > w ? (KT - w + KW - 1) / KW : 0;  // this wave's slices
  char* const mine = smem + w * D * SLICE;
  auto request = [&](int d, int j) {
    const int s = j * KW + w + start, slice = s >= KT ? s - KT : s;
    char* const lds = mine + d * SLICE;
    if constexpr (AMN)
      RA::request(Ab, p.lda, q.K - slice * 64, q.M - q.m0, slice, lds, lane);
    else
      SA::request(ra, (int)(p.lda * 2), q.M - q.m0, q.K, slice, lds, lane);
    if constexpr (BMN)
      RB::request(Bb, p.ldb, q.K - slice * 64, q.N - q.n0, slice, lds + A_SLICE, lane);
    else
      SB::request(rb, (int)(p.ldb * 2), q.N - q.n0, q.K, slice, lds + A_SLICE, lane);
  };
  // Slice j, `younger` slices asked for after it; then slice j + D into its
  // place where there is one.
  auto step = [&](int d, int j, int younger, bool more) {
    split_wait<LOADS>(younger);
    u32x4 a[MT][2], b[NT][2];
    const char* const lds = mine + d * SLICE;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
        a[i][h] = AMN ? RA::read(lds, i, h, lane) : SA::read(lds, i, h, lane);
#pragma unroll
      for (int n = 0; n < NT; ++n)
        b[n][h] = BMN ? RB::read(lds + A_SLICE, n, h, lane) : SB::read(lds + A_SLICE, n, h, lane);
    }
    pp_wait_lgkm0();  // read before the place is filled again
    layer_fixed_order();
    if (more) request(d, j + D);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[i][n] = At::mma(Tag{}, a[i][h], b[n][h], acc[i][n]);
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < NJ) request(d, d);
  for (int j = 0; j < NJ; j += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      const int left = NJ - 1 - (j + d);  // slices after this one
      if (left >= 0) step(d, j + d, left < D - 1 ? left : D - 1, left >= D);
    }
  }
  // Every request was waited for; the sums overlay the slices.
  __syncthreads();
  Sum::template finish<Tag>(acc, p, q, smem, tid, w);
}

template <class Tag, int MODE, bool AMN, bool BMN, int MT, int NT, int D, int KW>
hipError_t launch(const LayerArgs& a, int ntiles, hipStream_t s) {
  return launch_kernel(layer_split_kernel<Tag, MODE, AMN, BMN, MT, NT, D, KW>, dim3(ntiles),
                       dim3(KW * 64), s, a);
}
// D and KW: as many slices as the LDS holds, for eight waves while two fit.
template <class Tag, int MODE, bool AMN, bool BMN>
hipError_t launch_form(int mt, int nt, const LayerArgs& a, int ntiles, hipStream_t s) {
  if constexpr (!AMN) {
    if constexpr (!BMN)
      if (mt == 1 && nt == 1) return launch<Tag, MODE, AMN, BMN, 1, 1, 4, 8>(a, ntiles, s);
    if (mt == 1) return launch<Tag, MODE, AMN, BMN, 1, 2, 3, 8>(a, ntiles, s);
    if (mt == 3) return launch<Tag, MODE, AMN, BMN, 3, 2, 2, 8>(a, ntiles, s);
  }
  if (mt == 2) return launch<Tag, MODE, AMN, BMN, 2, 2, 2, 8>(a, ntiles, s);
  if (nt == 2) return launch<Tag, MODE, AMN, BMN, 4, 2, 3, 4>(a, ntiles, s);
  return launch<Tag, MODE, AMN, BMN, 4, 4, 2, 4>(a, ntiles, s);
}
template <class Tag>
hipError_t launch_layout(bool ta, bool tb, int mt, int nt, const LayerArgs& a, int ntiles,
                         hipStream_t s) {
  return layer_for_layout(a, ta, tb, [&](auto mode, auto la, auto lb) {
    return launch_form<Tag, mode.value, la.value != 0, lb.value == 0>(mt, nt, a, ntiles, s);
  });
}

}  // namespace

hipError_t launch_layer_split(int dtype, bool ta, bool tb, int mt, int nt, const LayerArgs& a,
                              int ntiles, hipStream_t s) {
  if (dtype == 0) return launch_layout<TagF16>(ta, tb, mt, nt, a, ntiles, s);
  return launch_layout<TagBF16>(ta, tb, mt, nt, a, ntiles, s);
}

}  // namespace dgt
