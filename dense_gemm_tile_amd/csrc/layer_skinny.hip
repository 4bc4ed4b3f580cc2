// The layer operators' product for at most 16 rows a tile, A stored [M][K], B
// stored [N][K]: decoding batches, and the handful of rows that each of many
// experts gets. Bound by the weights' bytes, so the point is to have enough of
// them in flight.
//
// A workgroup owns 16 rows and 16 NT columns; its KW waves split K: wave w
// takes slices w, w + KW, ... of 64 (whole 128-byte lines), so the workgroup
// walks consecutive memory and no two waves share an operand byte. There is no
// barrier and no LDS in the loop: fragments are loaded into registers, D slices
// ahead, with buffer loads whose offsets are out of range (read as zeros, not
// fetched) past M, N and K. Four lanes of such a load lie in four rows, which
// the address units serve at 16 bytes a clock and CU, a quarter of their rate
// for consecutive lanes: enough for weights that come from memory, not for more
// rows (layer_split.hip).
#include "layer_split.h"

namespace dgt {

namespace {

template <class Tag, int MODE, int NT, int D, int KW>
__global__ void __launch_bounds__(KW * 64) layer_skinny_kernel(const LayerArgs p) {
  using At = SplitAtom;
  using Sum = SplitSum<1, NT, KW>;
  __shared__ __attribute__((aligned(1024))) char smem[Sum::LDS_BYTES];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int total = layer_tiles<MODE, Sum::BM>(p, lane);
  if ((int)blockIdx.x >= total) return;  // by rows the grid is an upper bound
  const LayerTile q = layer_tile<MODE, Sum::BM, Sum::BN>(p, blockIdx.x, total, lane);

  // Resources end at the last byte of the operand's last row here, so no offset
  // below 2^31 reads past it.
  const auto ra = make_rsrc_n(q.A + (int64_t)q.m0 * p.lda * 2, split_records(q.M - q.m0, p.lda, q.K));
  const auto rb = make_rsrc_n(q.B + (int64_t)q.n0 * p.ldb * 2, split_records(q.N - q.n0, p.ldb, q.K));
  // This lane's piece of a slice: row l%16 of an atom, K values 8 (l/16) .. +7
  // of each half of 32.
  const int r16 = lane & 15, kl = 8 * (lane >> 4);
  const int arow = q.m0 + r16 < q.M ? (int)(r16 * p.lda * 2) : kOutOfRange;
  int brow[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    brow[n] = q.n0 + 16 * n + r16 < q.N ? (int)((16 * n + r16) * p.ldb * 2) : kOutOfRange;
  auto along_k = [&](const __amdgpu_buffer_rsrc_t& rs, int row, int k) {
    const int off = row != kOutOfRange && k < q.K ? row + k * 2 : kOutOfRange;
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
  };

  At::acc_t acc[1][NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[0][n][v] = 0.0f;

  const int KT = (q.K + 63) / 64;
  const int start = split_start(q.n0 / Sum::BN, KT);
  const int NJ = KT > w ? (KT - w + KW - 1) / KW : 0;  // this wave's slices
  u32x4 fa[D][2], fb[D][NT][2];
  // Slices beyond NJ are not asked for: even loads that fetch nothing take
  // their time in the address units.
  auto request = [&](int d, int j) {
    const int s = j * KW + w + start, k0 = 64 * (s >= KT ? s - KT : s);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) fb[d][n][h] = along_k(rb, brow[n], k0 + 32 * h + kl);
#pragma unroll
    for (int h = 0; h < 2; ++h) fa[d][h] = along_k(ra, arow, k0 + 32 * h + kl);
  };
  auto multiply = [&](int d) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[0][n] = At::mma(Tag{}, fa[d][h], fb[d][n][h], acc[0][n]);
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < NJ) request(d, d);
  int j = 0;
  for (; j + 2 * D <= NJ; j += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      multiply(d);
      request(d, j + d + D);
    }
  }
  // At most 2 D - 1 slices are left, D of them in flight.
#pragma unroll
  for (int d = 0; d < D; ++d) {
    const int left = NJ - 1 - (j + d);  // slices after this one
    if (left >= 0) multiply(d);
    if (left >= D) request(d, j + d + D);
  }
  j += D;
#pragma unroll
  for (int d = 0; d < D - 1; ++d)
    if (j + d < NJ) multiply(d);

  Sum::template finish<Tag>(acc, p, q, smem, tid, w);
}

template <class Tag, int MODE>
hipError_t launch(int nt, const LayerArgs& a, int ntiles, hipStream_t s) {
  constexpr int KW = 8;
  const dim3 grid(ntiles), block(KW * 64);
  if (nt == 1) return launch_kernel(layer_skinny_kernel<Tag, MODE, 1, 8, KW>, grid, block, s, a);
  return launch_kernel(layer_skinny_kernel<Tag, MODE, 2, 4, KW>, grid, block, s, a);
}

}  // namespace

hipError_t launch_layer_skinny(int dtype, int nt, const LayerArgs& a, int ntiles, hipStream_t s) {
  if (dtype == 0)
    return a.mode == LAYER_ROWS ? launch<TagF16, LAYER_ROWS>(nt, a, ntiles, s)
                                : launch<TagF16, LAYER_DENSE>(nt, a, ntiles, s);
  return a.mode == LAYER_ROWS ? launch<TagBF16, LAYER_ROWS>(nt, a, ntiles, s)
                              : launch<TagBF16, LAYER_DENSE>(nt, a, ntiles, s);
}

}  // namespace dgt
