// The layer operators' product on 128x128 tiles, two wave groups taking turns
// (the phase design of gemm_mfma_pingpong.h at the slot geometry of
// gemm_ring.h), for operands whose rows load in whole 16-byte pieces. For
// grids that 256x256 tiles would leave thin, and groups of fewer rows.
//
// Eight waves; group g owns rows [64g, 64g+64) of the tile, wave w of it the 32
// columns [32w, 32w+32). A of slice t lives in half-slot 2t % SLOTS, B in
// (2t+1) % SLOTS; in its memory phase for slice s group 1 loads A of slice
// s + AA and group 0 B of slice s + BA. With five half-slots two workgroups
// share a CU; DEEP has ten and asks further ahead, for grids of at most one
// tile per CU. Each refill goes into the slots of a slice whose last reader
// finished at least one phase earlier, and each group waits for its own loads
// of slice s+1 before the barrier after which that slice is read.
#include "gemm_ring.h"
#include "layer.h"

namespace dgt {

namespace {

struct Wave128 {  // the epilogue's view of a wave's 64x32 block
  using At = Atom<32>;
  static constexpr int TM = 2, TN = 1;
};

// s_waitcnt vmcnt(n * LOADS) and lgkmcnt(0) for a run-time n in 0..3.
template <int LOADS>
__device__ __forceinline__ void wait_slices(int n) {
  if (n >= 3) pp_wait_vm_lgkm0<3 * LOADS>();
  else if (n == 2) pp_wait_vm_lgkm0<2 * LOADS>();
  else if (n == 1) pp_wait_vm_lgkm0<LOADS>();
  else pp_wait_vm_lgkm0<0>();
}

template <class Tag, int MODE, bool AMN, bool BMN, bool DEEP>
__global__ void __launch_bounds__(2 * Ring128Cfg::THREADS, DEEP ? 1 : 2)
layer_pp128_kernel(const LayerArgs p) {
  using C = Ring128Cfg;
  using At = typename C::At;
  using acc_t = typename At::acc_t;
  constexpr int SLOTS = DEEP ? 10 : 5, AA = DEEP ? 4 : 2, BA = DEEP ? 3 : 1;
  static_assert(AA - 1 <= 3 && BA - 1 <= 3, "wait_slices counts up to three slices");
  __shared__ __attribute__((aligned(1024))) char smem[SLOTS * C::HALF_BYTES];
  static_assert(8 * layer_lds_bytes<Wave128>() <= SLOTS * C::HALF_BYTES, "the epilogue's rows fit");

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave >> 2, w = wave & 3;
  const int total = layer_tiles<MODE, C::BM>(p, lane);
  if ((int)blockIdx.x >= total) return;  // by rows the grid is an upper bound
  const LayerTile q = layer_tile<MODE, C::BM, C::BN>(p, blockIdx.x, total, lane);

  RingOperand<AMN, 128> a;
  RingOperand<BMN, 128> b;
  a.init(q.A, p.lda, q.m0, q.M, q.K, group, lane);   // atoms at rows 64 group + 32 t
  b.init(q.B, p.ldb, q.n0, q.N, q.K, w >> 1, lane);  // atoms at columns 64 (w/2) + 32 t
  const int boff = (w & 1) ? b.off[1] : b.off[0];    // this wave's columns 32 w .. +31

  acc_t acc[2][1];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int v = 0; v < At::NACC; ++v) acc[i][0][v] = 0.0f;

  const int KT = (q.K + C::BK - 1) / C::BK;
  auto slot = [&](int h) { return smem + (h % SLOTS) * C::HALF_BYTES; };
  // Slices of this group's loads that may stay in flight when slice t must
  // have landed and `last` was the last one requested.
  auto after = [](int t, int last) { return last - t < 0 ? 0 : last - t; };
  int alast = -1, blast = -1;
  if (group == 1) {
    for (int t = 0; t < AA && t < KT; ++t) a.issue_direct(slot(2 * t), t, w, lane);
    alast = (AA < KT ? AA : KT) - 1;
    wait_slices<C::LOADS>(after(0, alast));
  } else {
    for (int t = 0; t < BA && t < KT; ++t) b.issue_direct(slot(2 * t + 1), t, w, lane);
    blast = (BA < KT ? BA : KT) - 1;
    wait_slices<C::LOADS>(after(0, blast));
  }
  pp_barrier();
  if (group == 1) {
    wait_slices<C::LOADS>(after(1, alast));  // A of slice 1, read from phase 3 on
    pp_barrier();                            // and a phase behind group 0 from here
  }

  u32x4 fa[C::KSTEPS][2], fb[C::KSTEPS];
  for (int s = 0; s < KT; ++s) {
    const char* sa = slot(2 * s);
    const char* sb = slot(2 * s + 1);
    // Memory phase (issue priority over the other group's MFMA stream).
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int ks = 0; ks < C::KSTEPS; ++ks) {
      fa[ks][0] = a.read(sa, 0, ks);
      fa[ks][1] = a.read(sa, 1, ks);
      fb[ks] = RingOperand<BMN, 128>::read_at(sb, boff, ks);
    }
    if (group == 0) {
      if (s + BA < KT) {
        b.issue_direct(slot(2 * (s + BA) + 1), s + BA, w, lane);
        blast = s + BA;
      }
      pp_wait_lgkm0();
    } else {
      if (s + AA < KT) {
        a.issue_direct(slot(2 * (s + AA)), s + AA, w, lane);
        alast = s + AA;
      }
      wait_slices<C::LOADS>(after(s + 1, alast));
    }
    pp_barrier();
    __builtin_amdgcn_s_setprio(0);
    // Compute phase.
#pragma unroll
    for (int ks = 0; ks < C::KSTEPS; ++ks)
#pragma unroll
      for (int i = 0; i < 2; ++i) acc[i][0] = At::mma(Tag{}, fa[ks][i], fb[ks], acc[i][0]);
    if (group == 0) wait_slices<C::LOADS>(after(s + 1, blast));
    pp_barrier();
  }
  if (group == 0) pp_barrier();  // matches group 1's extra prologue barrier

  layer_store<Wave128, Tag>(acc, p, q, q.m0 + 64 * group, q.n0 + 32 * w, lane,
                            reinterpret_cast<float*>(smem + wave * layer_lds_bytes<Wave128>()));
}

template <class Tag, bool DEEP>
hipError_t launch(bool ta, bool tb, const LayerArgs& a, int ntiles, hipStream_t s) {
  return layer_for_layout(a, ta, tb, [&](auto mode, auto la, auto lb) {
    return launch_kernel(layer_pp128_kernel<Tag, mode.value, la.value != 0, lb.value == 0, DEEP>,
                         dim3(ntiles), dim3(2 * Ring128Cfg::THREADS), s, a);
  });
}

}  // namespace

hipError_t launch_layer_pp128(int dtype, bool ta, bool tb, bool deep, const LayerArgs& a,
                              int ntiles, hipStream_t s) {
  if (dtype == 0)
    return deep ? launch<TagF16, true>(ta, tb, a, ntiles, s) : launch<TagF16, false>(ta, tb, a, ntiles, s);
  return deep ? launch<TagBF16, true>(ta, tb, a, ntiles, s) : launch<TagBF16, false>(ta, tb, a, ntiles, s);
}

}  // namespace dgt
