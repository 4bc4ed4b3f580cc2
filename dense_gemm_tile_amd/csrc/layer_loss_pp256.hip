// The output layer's logits on 256x256 tiles, the two-group loop of gemm_mfma_pingpong.h,
// never written: the epilogue turns them into what the loss or its gradient needs.
//
// Rows are vocabulary entries and columns tokens, so that a token's logits lie in one lane's
// registers (32 of its column in each of four groups of lanes):
//   forward   largest logit and sum of exponentials of a tile's 256 entries for each token:
//             in the lane, over the lane groups, then over the two waves that share a
//             column; and the label's logit, where the tile has it
//   gradient  G = dloss / scale (exp(L - lse) - [v = label]), rounded to the operands' type,
//             which the matrix cores read next; rows through LDS so that stores are whole lines
//
// The exponentials take most of the epilogue: 128 a lane at 16 cycles a wave.
#include "gemm_mfma_pingpong.h"
#include "layer_loss.h"

namespace dgt {

namespace {

using C = PingPongCfgT<16>;
using At = C::At;

// Of the four lanes that hold a column: lanes l, l ^ 16, l ^ 32, l ^ 48.
template <class F>
__device__ __forceinline__ float loss_column(float v, F join) {
  v = join(v, __shfl_xor(v, 16, 64));
  return join(v, __shfl_xor(v, 32, 64));
}

__device__ __forceinline__ void loss_parts(At::acc_t (&acc)[C::TM][C::TN], const LossTileArgs& p, int tm, int tn, int wm,
                                           int wn, int lane, float2* lds) {
  const int m0 = tm * C::BM + wm * C::WTM, n0 = tn * C::BN + wn * C::WTN;
  const int left = p.n - m0;  // rows
  if (left < C::WTM) {
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (At::M * i + At::acc_row(lane, v) >= left)
#pragma unroll
          for (int j = 0; j < C::TN; ++j) acc[i][j][v] = -__builtin_inff();
  }
  int at[C::TN];  // the label's row of this wave's, for each column
  bool any = false;
#pragma unroll
  for (int j = 0; j < C::TN; ++j) {
    const int t = n0 + At::N * j + (lane & 15);
    const int label = t < p.T ? p.labels[t] : -1;
    at[j] = (unsigned)label < (unsigned)p.V ? label - p.v0 - m0 : -1;
    at[j] = at[j] >= 0 && at[j] < left && (at[j] >> 2 & 3) == lane >> 4 ? at[j] : -1;
    any |= at[j] >= 0 && at[j] < C::WTM;
  }
#pragma unroll
  for (int j = 0; j < C::TN; ++j) {
    float m = -__builtin_inff(), s = 0.0f;
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) m = __builtin_fmaxf(m, acc[i][j][v]);
    m = loss_column(m, [](float a, float b) { return __builtin_fmaxf(a, b); });
    const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) s += loss_exp(acc[i][j][v] - base);
    s = loss_column(s, [](float a, float b) { return a + b; });
    if (lane < 16) lds[wm * C::BN + wn * C::WTN + At::N * j + lane] = float2{m, s};
  }
  if (__ballot(any)) {
#pragma unroll
    for (int j = 0; j < C::TN; ++j) {
      float x = 0.0f;
#pragma unroll
      for (int i = 0; i < C::TM; ++i)
#pragma unroll
        for (int v = 0; v < 4; ++v) x = at[j] >= 0 && (at[j] >> 4) == i && (at[j] & 3) == v ? acc[i][j][v] : x;
      if (at[j] >= 0 && at[j] < C::WTM) p.target[n0 + At::N * j + (lane & 15)] = x;
    }
  }
}

template <class Tag>
__device__ __forceinline__ void loss_gradient(At::acc_t (&acc)[C::TM][C::TN], const LossTileArgs& p, int tm, int tn,
                                              int wm, int wn, int lane, float* lds) {
  using E = LayerEpi<C>;
  constexpr int AR = E::BATCH / At::M;
  const int cl = 8 * (lane % E::LPR), rl = lane / E::LPR;
  const int m0 = tm * C::BM + wm * C::WTM, c = tn * C::BN + wn * C::WTN + cl;
  float lse[8], d[8];
  int label[8];  // -1: no gradient
  const float scale = *p.scale;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int t = c + e;
    label[e] = t < p.T ? p.labels[t] : -1;
    if ((unsigned)label[e] >= (unsigned)p.V) label[e] = -1;
    lse[e] = label[e] >= 0 ? p.lse[t] : 0.0f;
    d[e] = label[e] >= 0 ? p.dloss[t] / scale : 0.0f;
  }
#pragma unroll
  for (int b = 0; b < C::TM / AR; ++b) {
    const int r = m0 + b * E::BATCH;
    if (r >= p.n) break;
#pragma unroll
    for (int i = 0; i < AR; ++i)
#pragma unroll
      for (int j = 0; j < C::TN; ++j)
#pragma unroll
        for (int v = 0; v < At::NACC; ++v)
          lds[(i * At::M + At::acc_row(lane, v)) * E::P + j * At::N + At::acc_col(lane)] = acc[b * AR + i][j][v];
    layer_wave_order();
#pragma unroll 1
    for (int s = 0; s < E::PASSES; ++s) {
      const int row = r + s * E::RPP + rl;
      const float* const from = lds + (s * E::RPP + rl) * E::P + cl;
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = loss_exp(from[e] - lse[e]) - (p.v0 + row == label[e] ? 1.0f : 0.0f);
        x[e] = label[e] >= 0 ? x[e] * d[e] : 0.0f;
      }
      if (row < p.n && c < p.T8)
        *reinterpret_cast<u32x4*>(static_cast<char*>(p.G) + ((int64_t)row * p.T8 + c) * 2) = layer_pack8<Tag>(x);
    }
    layer_wave_order();
  }
}

// Where the record count masks everything (PP_RECORDS), 256 workgroups walk the tiles.
template <class Tag, int MASK, bool GRAD>
__global__ void __launch_bounds__(C::THREADS) layer_loss_tile_kernel(const LossTileArgs p) {
  constexpr bool WALK = MASK == PP_RECORDS;
  __shared__ __attribute__((aligned(1024))) char smem[C::LDS_BYTES];
  static_assert(8 * layer_lds_bytes<C>() <= C::LDS_BYTES, "the epilogue's rows fit the operand LDS");
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int group = wave >> 2, wm = group, wn = wave & 3;
  const int total = p.tiles_m * p.tiles_n;
  for (int t = blockIdx.x; t < total; t += gridDim.x) {
    // The lane index, counted anew for every tile and opaque to loop-invariant code motion
    // (layer_pp256.hip).
    int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    asm volatile("" : "+v"(lane));
    int tm, tn;
    grouped_tile(xcd_remap(t, total), p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    GemmArgs ga{};  // what the loop reads of it
    ga.A = p.W;
    ga.B = p.X;
    ga.lda = p.ldw;
    ga.ldb = p.ldx;
    ga.M = p.n;
    ga.N = p.T;
    ga.K = p.H;
    PingPongPipe<false, false, At::M, MASK> pipe;
    pipe.init(ga, smem, tm * C::BM, tn * C::BN, group, wave, lane, wm, wn);
    At::acc_t acc[C::TM][C::TN];
#pragma unroll
    for (int i = 0; i < C::TM; ++i)
#pragma unroll
      for (int j = 0; j < C::TN; ++j)
#pragma unroll
        for (int v = 0; v < At::NACC; ++v) acc[i][j][v] = 0.0f;
    pp_mainloop<C, Tag, 16 + GRAD, false, false, MASK>(acc, pipe, p.H, group);
    int again = t;
    asm volatile("" : "+s"(again));
    lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0u));
    asm volatile("" : "+v"(lane));
    grouped_tile(xcd_remap(again, total), p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    if constexpr (GRAD) {
      loss_gradient<Tag>(acc, p, tm, tn, wm, wn, lane, reinterpret_cast<float*>(smem + wave * layer_lds_bytes<C>()));
    } else {
      float2* const lds = reinterpret_cast<float2*>(smem);
      loss_parts(acc, p, tm, tn, wm, wn, lane, lds);
      pp_wait_lgkm0();
      pp_barrier();
      const int col = threadIdx.x, at = tn * C::BN + col;
      if (col < C::BN && at < p.T) {
        const float2 a = lds[col], b = lds[C::BN + col];
        const float m = __builtin_fmaxf(a.x, b.x), base = m == -__builtin_inff() ? 0.0f : m;
        p.parts[(int64_t)tm * p.T + at] = float2{m, a.y * loss_exp(a.x - base) + b.y * loss_exp(b.x - base)};
      }
    }
    if constexpr (!WALK) break;
    // The next tile's loads overwrite the epilogue's LDS, other waves' too.
    pp_wait_lgkm0();
    pp_barrier();
  }
}

template <class Tag, bool GRAD>
hipError_t launch(const LossTileArgs& a, hipStream_t s) {
  const int tiles = a.tiles_m * a.tiles_n;
  if (a.H % 64 == 0)
    return launch_kernel(layer_loss_tile_kernel<Tag, PP_RECORDS, GRAD>, dim3(tiles < 256 ? tiles : 256), dim3(C::THREADS), s, a);
  return launch_kernel(layer_loss_tile_kernel<Tag, PP_MASKED, GRAD>, dim3(tiles), dim3(C::THREADS), s, a);
}

}  // namespace

hipError_t launch_loss_tiles(int dtype, bool grad, const LossTileArgs& args, hipStream_t s) {
  LossTileArgs a = args;
  a.tiles_m = (a.n + C::BM - 1) / C::BM;
  a.tiles_n = (a.T + C::BN - 1) / C::BN;
  a.group_m = 8;
  if (dtype == 0) return grad ? launch<TagF16, true>(a, s) : launch<TagF16, false>(a, s);
  return grad ? launch<TagBF16, true>(a, s) : launch<TagBF16, false>(a, s);
}

}  // namespace dgt
