// The layer operators' product for few rows, A stored [M][K], B stored [N][K],
// fragments straight from memory into registers. Bound by the weights' bytes, so
// the point is to have enough of them in flight.
//
// A workgroup owns 16 MT rows and 16 NT columns; its KW waves split K: wave w
// takes slices w, w + KW, ... of 64 (whole 128-byte lines), so the workgroup
// walks consecutive memory and no two waves share an operand byte. There is no
// barrier and no LDS in the loop: fragments are loaded into registers, D slices
// ahead, with buffer loads whose offsets are out of range (read as zeros, not
// fetched) past M, N and K. Four lanes of such a load lie in four rows, which
// the address units serve at 16 bytes a clock and CU, a quarter of their rate
// for consecutive lanes. For the few rows that each of many experts gets that
// is enough, and two workgroups of these fit a CU, which hides the start and the
// end of their short walks (64 experts of 2 rows, 2048x2048: 81 us, 97 with the
// operands through LDS as in layer_split.hip); dense calls are faster there
// (16x8192x8192: 28 us here, 26 there).
//
// ANY: rows at any 2-byte alignment and any K. A piece is read as the dwords
// that cover it, from the one at or below its start, and shifted into place;
// elements past K are zeroed. Up to 64 rows here: one row of 4096x4096 weights
// of pitch 4097 took 70 us on the general kernel, which loads such rows element
// by element, and 18 us here.
#include "gemm_ring.h"
#include "layer_split.h"

namespace dgt {

namespace {

// Fragment pieces between their loads and their use.
template <bool ANY>
struct SkinnyPiece {
  u32x4 v;
};
template <>
struct SkinnyPiece<true> {
  u32x4 v;
  unsigned e;  // the dword after v
};

template <class Tag, int MODE, bool ANY, int MT, int NT, int D, int KW>
__global__ void __launch_bounds__(KW * 64) layer_skinny_kernel(const LayerArgs p) {
  using At = SplitAtom;
  using Sum = SplitSum<MT, NT, KW>;
  using Piece = SkinnyPiece<ANY>;
  __shared__ __attribute__((aligned(1024))) char smem[Sum::LDS_BYTES];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int total = layer_tiles<MODE, Sum::BM>(p, lane);
  if ((int)blockIdx.x >= total) return;  // by rows the grid is an upper bound
  const LayerTile q = layer_tile<MODE, Sum::BM, Sum::BN>(p, blockIdx.x, total, lane);

  // Resources start at the (ANY: dword of the) tile's first row and end at the
  // (ANY: dword of the) last byte of the operand's last row here, so no offset
  // below 2^31 reads past it.
  auto first = [](const char* x) { return ANY ? x - ((uintptr_t)x & 3) : x; };
  auto records = [](const char* x, int64_t rows, int64_t ld, int64_t cols) {
    const unsigned n = split_records(rows, ld, cols);
    return ANY ? (n + (unsigned)((uintptr_t)x & 3) + 3) & ~3u : n;
  };
  const char* const Ab = q.A + (int64_t)q.m0 * p.lda * 2;
  const char* const Bb = q.B + (int64_t)q.n0 * p.ldb * 2;
  const auto ra = make_rsrc_n(first(Ab), records(Ab, q.M - q.m0, p.lda, q.K));
  const auto rb = make_rsrc_n(first(Bb), records(Bb, q.N - q.n0, p.ldb, q.K));
  // This lane's piece of a slice: row l%16 of an atom, K values 8 (l/16) .. +7
  // of each half of 32. Row offsets from the resource's start; the last two
  // bits are the piece's place in its dword.
  const int r16 = lane & 15, kl = 8 * (lane >> 4);
  auto row_at = [&](const char* x, int r, int64_t ld, int rows) {
    return r < rows ? (int)(r * ld * 2) + (ANY ? (int)((uintptr_t)x & 3) : 0) : kOutOfRange;
  };
  int arow[MT], brow[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) arow[i] = row_at(Ab, 16 * i + r16, p.lda, q.M - q.m0);
#pragma unroll
  for (int n = 0; n < NT; ++n) brow[n] = row_at(Bb, 16 * n + r16, p.ldb, q.N - q.n0);
  auto along_k = [&](const __amdgpu_buffer_rsrc_t& rs, int row, int k) {
    Piece x;
    const int off = row != kOutOfRange && k < q.K ? (row & ~3) + k * 2 : kOutOfRange;
    x.v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
    if constexpr (ANY)
      x.e = __builtin_amdgcn_raw_buffer_load_b32(rs, off == kOutOfRange ? kOutOfRange : off + 16, 0, 0);
    return x;
  };
  // The piece's 8 values from K value k on.
  auto values = [&](const Piece& x, int row, int k, bool tail) {
    if constexpr (!ANY) {
      return x.v;
    } else {
      u32x4 r;
      const unsigned sh = (unsigned)row & 3;
      r[0] = __builtin_amdgcn_alignbyte(x.v[1], x.v[0], sh);
      r[1] = __builtin_amdgcn_alignbyte(x.v[2], x.v[1], sh);
      r[2] = __builtin_amdgcn_alignbyte(x.v[3], x.v[2], sh);
      r[3] = __builtin_amdgcn_alignbyte(x.e, x.v[3], sh);
      if (tail) r = keep_first(r, q.K - k < 8 ? (q.K - k > 0 ? q.K - k : 0) : 8);
      return r;
    }
  };

  At::acc_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][n][v] = 0.0f;

  const int KT = (q.K + 63) / 64;
  const int start = split_start(q.n0 / Sum::BN, KT);
  const int NJ = KT > w ? (KT - w + KW - 1) / KW : 0;  // this wave's slices
  auto first_k = [&](int j) {
    const int s = j * KW + w + start;
    return 64 * (s >= KT ? s - KT : s);
  };
  Piece fa[D][MT][2], fb[D][NT][2];
  // Slices beyond NJ are not asked for: even loads that fetch nothing take
  // their time in the address units.
  auto request = [&](int d, int j) {
    const int k0 = first_k(j);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) fb[d][n][h] = along_k(rb, brow[n], k0 + 32 * h + kl);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) fa[d][i][h] = along_k(ra, arow[i], k0 + 32 * h + kl);
  };
  auto multiply = [&](int d, int j) {
    const int k0 = first_k(j);
    const bool tail = ANY && k0 + 64 > q.K;  // uniform
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = k0 + 32 * h + kl;
      u32x4 b[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) b[n] = values(fb[d][n][h], brow[n], k, tail);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const u32x4 a = values(fa[d][i][h], arow[i], k, tail);
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[i][n] = At::mma(Tag{}, a, b[n], acc[i][n]);
      }
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (d < NJ) request(d, d);
  int j = 0;
  for (; j + 2 * D <= NJ; j += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      multiply(d, j + d);
      request(d, j + d + D);
    }
  }
  // At most 2 D - 1 slices are left, D of them in flight.
#pragma unroll
  for (int d = 0; d < D; ++d) {
    const int left = NJ - 1 - (j + d);  // slices after this one
    if (left >= 0) multiply(d, j + d);
    if (left >= D) request(d, j + d + D);
  }
  j += D;
#pragma unroll
  for (int d = 0; d < D - 1; ++d)
    if (j + d < NJ) multiply(d, j + d);

  Sum::template finish<Tag>(acc, p, q, smem, tid, w);
}

template <class Tag, int MODE>
hipError_t launch(bool any, int mt, const LayerArgs& a, int ntiles, hipStream_t s) {
  constexpr int KW = 8;
  const dim3 grid(ntiles), block(KW * 64);
  if (any) {
    if (mt == 1) return launch_kernel(layer_skinny_kernel<Tag, MODE, true, 1, 2, 3, KW>, grid, block, s, a);
    if (mt == 2) return launch_kernel(layer_skinny_kernel<Tag, MODE, true, 2, 2, 2, KW>, grid, block, s, a);
    return launch_kernel(layer_skinny_kernel<Tag, MODE, true, 4, 2, 2, KW>, grid, block, s, a);
  }
  // Aligned rows come here by rows alone: dense calls are faster through LDS.
  if constexpr (MODE == LAYER_ROWS)
    return launch_kernel(layer_skinny_kernel<Tag, MODE, false, 1, 2, 4, KW>, grid, block, s, a);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_layer_skinny(int dtype, bool any, int mt, const LayerArgs& a, int ntiles,
                               hipStream_t s) {
  if (dtype == 0)
    return a.mode == LAYER_ROWS ? launch<TagF16, LAYER_ROWS>(any, mt, a, ntiles, s)
                                : launch<TagF16, LAYER_DENSE>(any, mt, a, ntiles, s);
  return a.mode == LAYER_ROWS ? launch<TagBF16, LAYER_ROWS>(any, mt, a, ntiles, s)
                              : launch<TagBF16, LAYER_DENSE>(any, mt, a, ntiles, s);
}

}  // namespace dgt
