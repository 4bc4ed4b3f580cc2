// The layer operators' product on 256x256 tiles: the two-group loop of
// gemm_mfma_pingpong.h with the layer epilogue, for operands whose rows load in
// whole 16-byte pieces. Dense, by rows and by sum; pieces outside a group's
// rows, columns or sum read as zeros.
//
// By rows, and where pieces are masked one by one, a workgroup has one tile: by
// rows the grid is an upper bound (groups held on the GPU), and a workgroup past
// the last tile ends at once. Dense and by sum with the record count as the mask
// (PP_RECORDS), 256 workgroups walk the tiles of a larger call.
#include "gemm_mfma_pingpong.h"
#include "layer.h"

namespace dgt {

namespace {

template <int MODE, int MASK>
constexpr bool layer_pp256_walks() { return MASK == PP_RECORDS && MODE != LAYER_ROWS; }

template <class Tag, int MODE, bool AMN, bool BMN, int MASK>
__global__ void __launch_bounds__(PingPongCfg::THREADS) layer_pp256_kernel(const LayerArgs p) {
  using C = PingPongCfgT<AMN ? 32 : 16>;  // the atom: see gemm_mfma_pingpong.h
  using At = typename C::At;
  using acc_t = typename At::acc_t;
  constexpr bool WALK = layer_pp256_walks<MODE, MASK>();
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS_BYTES];
  static_assert(8 * layer_lds_bytes<C>() <= C::LDS_BYTES, "the epilogue's rows fit the operand LDS");

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave >> 2;
  const int wm = group, wn = wave & 3;
  const int total = layer_tiles<MODE, C::BM>(p, threadIdx.x & 63);
  for (int t = blockIdx.x; t < total; t += gridDim.x) {
    // The lane index, counted anew for every tile and opaque to loop-invariant
    // code motion: no register holds it, or what depends on it, across the loop
    // over K.
    int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    asm volatile("" : "+v"(lane));
    LayerTile q = layer_tile<MODE, C::BM, C::BN>(p, t, total, lane);
    GemmArgs ga{};  // what the loop reads of it
    ga.A = q.A;
    ga.B = q.B;
    ga.lda = p.lda;
    ga.ldb = p.ldb;
    ga.M = q.M;
    ga.N = q.N;
    ga.K = q.K;
    PingPongPipe<AMN, BMN, At::M, MASK> pipe;
    pipe.init(ga, smem, q.m0, q.n0, group, wave, lane, wm, wn);
    acc_t acc[C::TM][C::TN];
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int j = 0; j < C::TN; ++j)
#pragma unroll
        for (int v = 0; v < At::NACC; ++v) acc[i][j][v] = 0.0f;
    pp_mainloop<C, Tag, MODE, AMN, BMN, MASK>(acc, pipe, q.K, group);
    // The tile is found again rather than kept in scalar registers, which the
    // loop has none to spare of.
    int again = t;
    asm volatile("" : "+s"(again));
    lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    asm volatile("" : "+v"(lane));
    q = layer_tile<MODE, C::BM, C::BN>(p, again, total, lane);
    layer_store<C, Tag>(acc, p, q, q.m0 + wm * C::WTM, q.n0 + wn * C::WTN, lane,
                        reinterpret_cast<float*>(smem + wave * layer_lds_bytes<C>()));
    if constexpr (!WALK) break;
    // The next tile's loads overwrite the epilogue's rows, those of other waves
    // too, so every wave's own LDS operations end here. (A wave whose columns lie
    // past N writes rows that it never uses: nothing else waits for them.)
    pp_wait_lgkm0();
    pp_barrier();
  }
}

template <class Tag, int MASK>
hipError_t launch(bool ta, bool tb, const LayerArgs& a, int ntiles, hipStream_t s) {
  return layer_for_layout(a, ta, tb, [&](auto mode, auto la, auto lb) {
    return launch_kernel(layer_pp256_kernel<Tag, mode.value, la.value != 0, lb.value == 0, MASK>,
                         dim3(layer_pp256_walks<mode.value, MASK>() && ntiles > 256 ? 256 : ntiles), dim3(PingPongCfg::THREADS), s, a);
  });
}
template <class Tag>
hipError_t launch_mask(bool ta, bool tb, const LayerArgs& a, int ntiles, hipStream_t s) {
  // By sum, K is a group's rows: any number of them will do there, as for every
  // operand not stored along K.
  const bool records = (ta ? a.M % 256 == 0 : a.K % 64 == 0) && (tb ? a.K % 64 == 0 : a.N % 256 == 0);
  return records ? launch<Tag, PP_RECORDS>(ta, tb, a, ntiles, s)
                 : launch<Tag, PP_MASKED>(ta, tb, a, ntiles, s);
}

}  // namespace

hipError_t launch_layer_pp256(int dtype, bool ta, bool tb, const LayerArgs& a, int ntiles,
                              hipStream_t s) {
  if (dtype == 0) return launch_mask<TagF16>(ta, tb, a, ntiles, s);
  return launch_mask<TagBF16>(ta, tb, a, ntiles, s);
}

}  // namespace dgt
