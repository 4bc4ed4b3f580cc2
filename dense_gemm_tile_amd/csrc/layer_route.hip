// Tokens sorted by expert: a stable counting sort of the choices.
//
//   offsets[e] = choices of experts below e;  position of choice i of expert e
//   = offsets[e] + (choices of e before i)
//
// A choice is 4 bytes read and 8 written, so the sort is bound by latency:
// one launch of one workgroup for up to kOneBlock choices, two launches of up
// to kMaxBlocks workgroups past that. Each wave owns a run of consecutive
// choices and counts it in its own LDS row; the counts before it (earlier
// waves, earlier blocks, lower experts) give its starting positions, and it
// then walks its run again 64 choices at a time, placing equal ids by lane
// order. No atomics on positions, so the order never depends on the run.
#include "layer_rows.h"

namespace dgt {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kOneBlock = 16384, kMaxBlocks = 256;
constexpr int kRow = kRouteMaxExperts + 1;  // experts and the dropped ones

__device__ inline int route_key(int id, int E) { return (unsigned)id < (unsigned)E ? id : E; }

// The choices [lo, hi) of wave w of a block.
__device__ inline void route_run(const RouteArgs& p, int block, int w, int& lo, int& hi) {
  const int64_t b0 = (int64_t)block * p.chunk;
  const int64_t end = b0 + p.chunk < p.n ? b0 + p.chunk : p.n;
  const int64_t per = ((end > b0 ? end - b0 : 0) + kWaves - 1) / kWaves;
  const int64_t l = b0 + w * per < end ? b0 + w * per : end;
  const int64_t h = l + per < end ? l + per : end;
  lo = (int)l;
  hi = (int)h;
}

// Counts of each wave's run: hist[w][key].
__device__ inline void route_count(const RouteArgs& p, int (*hist)[kRow], int block) {
  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
  for (int e = lane; e <= p.E; e += 64) hist[w][e] = 0;
  __syncthreads();
  int lo, hi;
  route_run(p, block, w, lo, hi);
  for (int i = lo + lane; i < hi; i += 64) atomicAdd(&hist[w][route_key(p.ids[i], p.E)], 1);
  __syncthreads();
}

__global__ void __launch_bounds__(kThreads) layer_route_count_kernel(const RouteArgs p) {
  __shared__ int hist[kWaves][kRow];
  route_count(p, hist, blockIdx.x);
  for (int e = threadIdx.x; e <= p.E; e += kThreads) {
    int sum = 0;
    for (int w = 0; w < kWaves; ++w) sum += hist[w][e];
    p.counts[(int64_t)blockIdx.x * (p.E + 1) + e] = sum;
  }
}

__global__ void __launch_bounds__(kThreads) layer_route_place_kernel(const RouteArgs p) {
  __shared__ int hist[kWaves][kRow];
  __shared__ int wsum[kWaves];
  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
  const int E1 = p.E + 1;
  route_count(p, hist, blockIdx.x);

  // Of key e = tid (and the last one, which may lie past the threads): all
  // choices, and those in earlier blocks.
  int carry = 0;  // choices of the keys of earlier rounds
  for (int e0 = 0; e0 < E1; e0 += kThreads) {
    const int e = e0 + tid;
    int own = 0, all = 0, before = 0;
    if (e < E1) {
      for (int v = 0; v < kWaves; ++v) own += hist[v][e];
      all = own;
      if (p.blocks > 1) {
        all = 0;
        int b = 0;
        for (; b + 8 <= p.blocks; b += 8) {
          int c[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) c[u] = p.counts[(int64_t)(b + u) * E1 + e];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            before += b + u < (int)blockIdx.x ? c[u] : 0;
            all += c[u];
          }
        }
        for (; b < p.blocks; ++b) {
          const int c = p.counts[(int64_t)b * E1 + e];
          before += b < (int)blockIdx.x ? c : 0;
          all += c;
        }
      }
    }
    // Exclusive scan of `all` over the keys.
    int incl = all;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(incl, d, 64);
      if (lane >= d) incl += o;
    }
    if (lane == 63) wsum[w] = incl;
    __syncthreads();
    int base = carry;
    for (int v = 0; v < w; ++v) base += wsum[v];
    const int start = base + incl - all;
    for (int v = 0; v < kWaves; ++v) carry += wsum[v];
    __syncthreads();
    if (e < E1) {
      if (blockIdx.x == 0) p.offsets[e] = start;  // offsets[E]: the first dropped one
      int at = start + before;
      for (int v = 0; v < kWaves; ++v) {
        const int c = hist[v][e];
        hist[v][e] = at;
        at += c;
      }
    }
  }
  __syncthreads();

  int lo, hi;
  route_run(p, blockIdx.x, w, lo, hi);
  for (int i0 = lo; i0 < hi; i0 += 64) {
    const int i = i0 + lane;
    const bool in = i < hi;
    const int key = in ? route_key(p.ids[i], p.E) : -1;
    // Lanes with the same key, found bit by bit.
    uint64_t same = __ballot(in);
    for (int b = 0; (1 << b) <= p.E; ++b) {
      const uint64_t set = __ballot((key >> b) & 1);
      same &= (key >> b) & 1 ? set : ~set;
    }
    const uint64_t below = same & ((uint64_t{1} << lane) - 1);
    if (in) {
      const int pos = hist[w][key] + __popcll(below);
      p.order[pos] = i;
      p.slot[i] = key < p.E ? pos : -1;
    }
    __builtin_amdgcn_wave_barrier();
    if (in && below == 0) hist[w][key] += __popcll(same);
    __builtin_amdgcn_wave_barrier();
  }
}

}  // namespace

void route_blocks(int64_t n, int& blocks, int& chunk) {
  if (n <= kOneBlock) {
    blocks = 1;
    chunk = kOneBlock;
    return;
  }
  int64_t c = 4096;
  if ((n + c - 1) / c > kMaxBlocks) c = (n + kMaxBlocks - 1) / kMaxBlocks;
  chunk = (int)c;
  blocks = (int)((n + c - 1) / c);
}

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  if (a.blocks > 1) {
    const hipError_t e = launch_kernel(layer_route_count_kernel, dim3(a.blocks), dim3(kThreads), s, a);
    if (e != hipSuccess) return e;
  }
  return launch_kernel(layer_route_place_kernel, dim3(a.blocks), dim3(kThreads), s, a);
}

}  // namespace dgt
