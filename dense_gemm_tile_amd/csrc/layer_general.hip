// The layer operators' product for any shape, layout, pitch and alignment:
// operands go through registers into two swizzled LDS stages (the stager and
// fragments of gemm_mfma_impl.h), every edge is masked. Calls whose operands
// can be loaded straight into LDS run on the other kernels; this one serves
// rows that are not 16-byte aligned, widths that cut a 16-byte piece, pitches
// past 32-bit offsets, and K == 0.
#include "layer.h"

namespace dgt {

namespace {

using GeneralBig = TileCfg<128, 128, 2, 2, 32>;   // 64 x 64 per wave
using GeneralSmall = TileCfg<64, 64, 2, 2, 16>;   // 32 x 32 per wave
// The same with the sum split over four groups of waves: group g takes K steps g,
// g + 4, ... through LDS of its own; their sums are added in group order.
using GeneralSplit = TileCfg<64, 64, 2, 2, 16, 4>;

template <class Cfg, class Tag, int MODE, bool TA, bool TB>
__global__ void __launch_bounds__(Cfg::THREADS) layer_general_kernel(const LayerArgs p) {
  using At = typename Cfg::At;
  using acc_t = typename At::acc_t;
  constexpr int EPI_BYTES = Cfg::WM * Cfg::WN * layer_lds_bytes<Cfg>();
  constexpr int LDS_BYTES = Cfg::LDS_BYTES > EPI_BYTES ? Cfg::LDS_BYTES : EPI_BYTES;
  __shared__ __attribute__((aligned(16))) char lds[LDS_BYTES];

  constexpr int GT = Cfg::GROUP_THREADS;
  const int lane = threadIdx.x & 63;
  const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / GT);  // K group
  const int tid = threadIdx.x % GT;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / Cfg::WN, wn = wave % Cfg::WN;
  char* const smem = lds + group * Cfg::GROUP_LDS_BYTES;
  const int total = layer_tiles<MODE, Cfg::BM>(p, lane);
  if ((int)blockIdx.x >= total) return;  // by rows the grid is an upper bound
  const LayerTile q = layer_tile<MODE, Cfg::BM, Cfg::BN>(p, blockIdx.x, total, lane);

  Stager<Cfg::BM, GT, !TA, true> sa;
  Stager<Cfg::BN, GT, TB, true> sb;
  acc_t acc[Cfg::TM][Cfg::TN];
#pragma unroll
  for (int i = 0; i < Cfg::TM; ++i)
#pragma unroll
    for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
      for (int v = 0; v < At::NACC; ++v) acc[i][j][v] = 0.0f;

  // This group's K steps: t counts group, group + KG, ...
  const int steps = (q.K + Cfg::BK - 1) / Cfg::BK;
  const int KT = steps > group ? (steps - group + Cfg::KG - 1) / Cfg::KG : 0;
  const int rounds = (steps + Cfg::KG - 1) / Cfg::KG;  // of every group
  // Boxes wholly inside an operand are loaded without bounds checks; with
  // 16-byte rows that takes 32-bit offsets over a box.
  auto fits = [](int64_t ld, int rows) { return ld * 2 * rows + 4096 < (int64_t{1} << 31); };
  const bool a_in = q.m0 + Cfg::BM <= q.M && (p.a_vw < 8 || fits(p.lda, Cfg::BM));
  const bool b_in = q.n0 + Cfg::BN <= q.N && (p.b_vw < 8 || fits(p.ldb, Cfg::BN));
  auto load = [&](int t) {
    const int k0 = (t * Cfg::KG + group) * Cfg::BK;
    const bool kin = k0 + Cfg::BK <= q.K;
    sa.load(q.A, p.lda, q.m0, q.M, k0, q.K, tid, p.a_vw, 0, a_in && kin);
    sb.load(q.B, p.ldb, q.n0, q.N, k0, q.K, tid, p.b_vw, 0, b_in && kin);
  };
  auto store = [&](int t) {
    char* s = smem + (t & 1) * Cfg::STAGE_BYTES;
    sa.store(s, tid);
    sb.store(s + Cfg::A_BYTES, tid);
  };
  if (KT > 0) {
    load(0);
    store(0);
  }
  __syncthreads();
  const int ar = wm * Cfg::WTM + At::frag_row(lane), br = wn * Cfg::WTN + At::frag_row(lane);
  for (int t = 0; t < rounds; ++t) {
    if (t + 1 < KT) load(t + 1);
    const char* As = smem + (t & 1) * Cfg::STAGE_BYTES;
    const char* Bs = As + Cfg::A_BYTES;
    if (Cfg::KG == 1 || t < KT)
#pragma unroll
    for (int ks = 0; ks < Cfg::KSTEPS; ++ks) {
      Frags<Cfg> f;
      read_frags<Cfg>(f, As, Bs, ar, br, ks * (At::K / 8) + At::frag_koct(lane));
      mma_step<Cfg, Tag>(acc, f);
    }
    // The other stage was last read one step ago, before the barrier that
    // ended it.
    if (t + 1 < KT) store(t + 1);
    __syncthreads();
  }
  if constexpr (Cfg::KG > 1) {
    // (Every group is past its last step's reads.)
    constexpr int NV = Cfg::TM * Cfg::TN * At::NACC;
    float* const x = reinterpret_cast<float*>(lds);
    auto sum_at = [&](int g) { return x + ((g - 1) * Cfg::WM * Cfg::WN + wave) * NV * 64 + lane; };
    if (group > 0) {
#pragma unroll
      for (int i = 0; i < Cfg::TM; ++i)
#pragma unroll
        for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
          for (int v = 0; v < At::NACC; ++v)
            sum_at(group)[((i * Cfg::TN + j) * At::NACC + v) * 64] = acc[i][j][v];
    }
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int g = 1; g < Cfg::KG; ++g)
#pragma unroll
      for (int i = 0; i < Cfg::TM; ++i)
#pragma unroll
        for (int j = 0; j < Cfg::TN; ++j)
#pragma unroll
          for (int v = 0; v < At::NACC; ++v)
            acc[i][j][v] += sum_at(g)[((i * Cfg::TN + j) * At::NACC + v) * 64];
    // The epilogue's rows lie past the sums, which other waves may still read.
    static_assert(Cfg::XFER_BYTES + EPI_BYTES <= LDS_BYTES, "sums and rows side by side");
  }
  constexpr int EPI_AT = Cfg::KG > 1 ? Cfg::XFER_BYTES : 0;
  layer_store<Cfg, Tag>(acc, p, q, q.m0 + wm * Cfg::WTM, q.n0 + wn * Cfg::WTN, lane,
                        reinterpret_cast<float*>(lds + EPI_AT + wave * layer_lds_bytes<Cfg>()));
}

template <class Cfg, class Tag>
hipError_t launch(bool ta, bool tb, const LayerArgs& a, int ntiles, hipStream_t s) {
  return layer_for_layout(a, ta, tb, [&](auto mode, auto la, auto lb) {
    return launch_kernel(layer_general_kernel<Cfg, Tag, mode.value, la.value, lb.value>,
                         dim3(ntiles), dim3(Cfg::THREADS), s, a);
  });
}

}  // namespace

hipError_t launch_layer_general(int dtype, bool ta, bool tb, int tile, const LayerArgs& a,
                                int ntiles, hipStream_t s) {
  if (tile == 2) {
    if (dtype == 0) return launch<GeneralSplit, TagF16>(ta, tb, a, ntiles, s);
    return launch<GeneralSplit, TagBF16>(ta, tb, a, ntiles, s);
  }
  if (tile == 1) {
    if (dtype == 0) return launch<GeneralSmall, TagF16>(ta, tb, a, ntiles, s);
    return launch<GeneralSmall, TagBF16>(ta, tb, a, ntiles, s);
  }
  if (dtype == 0) return launch<GeneralBig, TagF16>(ta, tb, a, ntiles, s);
  return launch<GeneralBig, TagBF16>(ta, tb, a, ntiles, s);
}

}  // namespace dgt
