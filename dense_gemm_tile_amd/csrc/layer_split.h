// Shared by the layer products that split the sum over a workgroup's waves
// (layer_skinny.hip, layer_split.hip): resources, waits, and the waves' sums
// joined and finished.
#pragma once

#include "gemm_mfma_pingpong.h"
#include "layer.h"

namespace dgt {

using SplitAtom = Atom<16>;

// No memory operation crosses, neither in the compiler's view nor in its
// schedule: loads that a wait counts have to be issued in the order written.
__device__ __forceinline__ void layer_fixed_order() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// A resource's record count: `rows` rows of a matrix of 16-bit elements, the
// last one cut after `cols`.
__device__ __forceinline__ unsigned split_records(int64_t rows, int64_t ld, int64_t cols) {
  const int64_t n = 2 * ((rows - 1) * ld + cols);
  return n > 0x7FFFFFFC ? 0x7FFFFFFCu : (rows <= 0 || n <= 0 ? 0u : (unsigned)n);
}

// Where a column tile's walk over the KT slices starts. Column tiles start at
// different slices and walk around: workgroups that all read the same part of
// rows a power of two apart would meet in few memory channels (16x8192x8192:
// 33 us from slice 0 everywhere, 28 so). Row tiles of one column tile walk
// alike and share B.
__device__ __forceinline__ int split_start(int column_tile, int KT) {
  return (int)(((uint64_t)((unsigned)column_tile * 0x9E3779B1u) * (unsigned)KT) >> 32);
}

// A workgroup of KW waves, each with sums of its own part of K for the same
// 16 MT x 16 NT outputs: they meet in LDS, are added in wave order, and go
// through the epilogue.
template <int MT, int NT, int KW>
struct SplitSum {
  static constexpr int BM = 16 * MT, BN = 16 * NT, THREADS = 64 * KW;
  static constexpr int PITCH = BN + 4;  // floats of an output row
  static constexpr int VALUES = MT * NT * 256;
  static constexpr int SUM_BYTES = KW * VALUES * 4;
  static constexpr int LDS_BYTES = SUM_BYTES + BM * PITCH * 4;

  // lds: LDS_BYTES, past its last use by any wave when this is called.
  template <class Tag>
  __device__ static __forceinline__ void finish(const SplitAtom::acc_t (&acc)[MT][NT],
                                                const LayerArgs& p, const LayerTile& q, char* lds,
                                                int tid, int w) {
    const int lane = tid & 63;
    float* sums = reinterpret_cast<float*>(lds);
    float* outs = reinterpret_cast<float*>(lds + SUM_BYTES);
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          sums[((w * MT + i) * NT + n) * 256 + v * 64 + lane] = acc[i][n][v];
    __syncthreads();
    for (int x = tid; x < VALUES; x += THREADS) {
      float s = sums[x];
#pragma unroll
      for (int u = 1; u < KW; ++u) s += sums[u * VALUES + x];
      const int ln = x & 63, v = (x >> 6) & 3, at = x >> 8;
      outs[(16 * (at / NT) + SplitAtom::acc_row(ln, v)) * PITCH + 16 * (at % NT) +
           SplitAtom::acc_col(ln)] = s;
    }
    __syncthreads();
    for (int x = tid; x < BM * (BN / 8); x += THREADS) {
      const int rr = x / (BN / 8), cl = 8 * (x % (BN / 8));
      const int r = q.m0 + rr, c = q.n0 + cl, nv = q.N - c >= 8 ? 8 : q.N - c;
      if (r < q.M && nv > 0) {
        float bias[8], v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          bias[e] = 0.0f;
          v[e] = outs[rr * PITCH + cl + e];
        }
        if (q.bias) layer_load8_16<Tag>(q.bias + (int64_t)c * 2, nv, bias);
        layer_finish8<Tag>(p, q, r, c, nv, bias, v);
      }
    }
  }
};

}  // namespace dgt
