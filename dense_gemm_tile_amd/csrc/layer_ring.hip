// The layer operators' product on 128x128 tiles where an operand that is not
// stored along K has rows that are not whole 16-byte pieces: the ring of
// gemm_ring.h, whose staged operands are read as the dwords that cover each
// piece, shifted into place in registers and written to LDS where a direct load
// would have put them (any 2-byte alignment; elements past an edge become zeros).
// The other operand, if its rows are 16-byte pieces, goes straight into LDS.
//
// Four waves of 64x64 outputs, two workgroups to a CU (five half-slots of LDS
// each); A of slice t lives in half-slot 2t % 5, B in (2t+1) % 5. Iteration t
// writes the staged pieces of slice t+1, asks for direct B of t+1 and direct A
// and staged pieces of t+2, and multiplies slice t. Against the general kernel,
// which transposes operands not stored along K in registers (4096^3 bf16, us):
// A stored [4096][4095] 246 instead of 357, B so 282 instead of 343; groups of
// about 2000 rows, weights' gradient of 1001 x 701, 89 instead of 137.
#include "gemm_ring.h"
#include "layer.h"

namespace dgt {

namespace {

template <class Tag, int MODE, bool AMN, bool BMN>
__global__ void __launch_bounds__(Ring128Cfg::THREADS, 2) layer_ring_kernel(const LayerArgs p) {
  using C = Ring128Cfg;
  using At = typename C::At;
  using acc_t = typename At::acc_t;
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS_BYTES];
  static_assert(4 * layer_lds_bytes<C>() <= C::LDS_BYTES, "the epilogue's rows fit the operand LDS");

  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w >> 1, wn = w & 1;
  const int total = layer_tiles<MODE, C::BM>(p, lane);
  if ((int)blockIdx.x >= total) return;  // by rows the grid is an upper bound
  const LayerTile q = layer_tile<MODE, C::BM, C::BN>(p, blockIdx.x, total, lane);

  RingOperand<AMN, 128> a;
  RingOperand<BMN, 128> b;
  a.init(q.A, p.lda, q.m0, q.M, q.K, wm, lane);
  b.init(q.B, p.ldb, q.n0, q.N, q.K, wn, lane);
  // Uniform over the launch (operands stored along K are direct); edges are those
  // that cut a piece of this tile.
  static_assert(AMN || BMN, "an operand to stage");
  const bool a_dir = !AMN || p.a_direct, b_dir = !BMN || p.b_direct, staged = !a_dir || !b_dir;
  const bool a_edge = q.m0 + C::BM > q.M && q.M % 8 != 0;
  const bool b_edge = q.n0 + C::BN > q.N && q.N % 8 != 0;

  acc_t acc[C::TM][C::TN];
#pragma unroll
  for (int i = 0; i < C::TM; ++i)
#pragma unroll
    for (int j = 0; j < C::TN; ++j)
#pragma unroll
      for (int v = 0; v < At::NACC; ++v) acc[i][j][v] = 0.0f;

  const int KT = (q.K + C::BK - 1) / C::BK;
  auto slot = [&](int h) { return smem + (h % C::SLOTS) * C::HALF_BYTES; };
  typename RingOperand<AMN, 128>::Staged ra;
  typename RingOperand<BMN, 128>::Staged rb;
  auto load = [&](int t) {
    if (!a_dir) a.load_staged(ra, t, w, lane);
    if (!b_dir) b.load_staged(rb, t, w, lane);
  };
  auto store = [&](int t) {
    if (!a_dir) a.store_staged(slot(2 * t), ra, t, w, lane, a_edge, 0);
    if (!b_dir) b.store_staged(slot(2 * t + 1), rb, t, w, lane, b_edge, 0);
  };

  if (KT > 0) {
    if (a_dir) a.issue_direct(slot(0), 0, w, lane);
    if (b_dir) b.issue_direct(slot(1), 0, w, lane);
    load(0);
    if (a_dir && KT > 1) a.issue_direct(slot(2), 1, w, lane);
    pp_wait_vm<0>();
    store(0);
    if (KT > 1) load(1);
    pp_wait_lgkm0();
  }
  pp_barrier();
  for (int t = 0; t < KT; ++t) {
    // Staged pieces of slice t+1 arrived during the last iteration (this waits
    // for every older load); their slots were left by slice t-1.
    if (staged && t + 1 < KT) {
      pp_wait_vm<0>();
      store(t + 1);
    }
    if (b_dir && t + 1 < KT) b.issue_direct(slot(2 * t + 3), t + 1, w, lane);
    if (a_dir && t + 2 < KT) a.issue_direct(slot(2 * t + 4), t + 2, w, lane);
    if (t + 2 < KT) load(t + 2);

    const char* sa = slot(2 * t);
    const char* sb = slot(2 * t + 1);
#pragma unroll
    for (int ks = 0; ks < C::KSTEPS; ++ks) {
      u32x4 fa[C::TM], fb[C::TN];
#pragma unroll
      for (int i = 0; i < C::TM; ++i) fa[i] = a.read(sa, i, ks);
#pragma unroll
      for (int j = 0; j < C::TN; ++j) fb[j] = b.read(sb, j, ks);
#pragma unroll
      for (int i = 0; i < C::TM; ++i)
#pragma unroll
        for (int j = 0; j < C::TN; ++j) acc[i][j] = At::mma(Tag{}, fa[i], fb[j], acc[i][j]);
    }
    // Direct loads of slice t+1 have to be in LDS at the barrier: B was asked for
    // first in this iteration, then one half slice of t+2 (4 direct loads of A,
    // or 8 staged ones), which may stay in flight.
    if (b_dir) {
      if (t + 2 < KT && a_dir) pp_wait_vm_lgkm0<C::LOADS>();
      else if (t + 2 < KT) pp_wait_vm_lgkm0<2 * C::LOADS>();
      else pp_wait_vm_lgkm0<0>();
    } else {
      pp_wait_lgkm0();
    }
    pp_barrier();
  }
  layer_store<C, Tag>(acc, p, q, q.m0 + wm * C::WTM, q.n0 + wn * C::WTN, lane,
                      reinterpret_cast<float*>(smem + w * layer_lds_bytes<C>()));
}

template <class Tag>
hipError_t launch(bool ta, bool tb, const LayerArgs& a, int ntiles, hipStream_t s) {
  return layer_for_layout(a, ta, tb, [&](auto mode, auto la, auto lb) {
    constexpr bool AMN = la.value != 0, BMN = lb.value == 0;
    if constexpr (AMN || BMN)
      return launch_kernel(layer_ring_kernel<Tag, mode.value, AMN, BMN>, dim3(ntiles),
                           dim3(Ring128Cfg::THREADS), s, a);
    else
      return hipErrorInvalidValue;  // never planned
  });
}

}  // namespace

hipError_t launch_layer_ring(int dtype, bool ta, bool tb, const LayerArgs& a, int ntiles,
                             hipStream_t s) {
  if (dtype == 0) return launch<TagF16>(ta, tb, a, ntiles, s);
  return launch<TagBF16>(ta, tb, a, ntiles, s);
}

}  // namespace dgt
