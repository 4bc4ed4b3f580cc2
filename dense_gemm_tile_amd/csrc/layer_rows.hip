// The layer operators that move rows: activation gradients with bias sums,
// rows sent to their experts, rows joined again with weights, and the
// gradients of that. All are bound by memory: each input is read once, each
// output written once, 16 bytes a lane where alignment allows.
#include "layer.h"
#include "layer_rows.h"

namespace dgt {

namespace {

// This workgroup's index in a layer_grid().
template <class Args>
__device__ __forceinline__ unsigned layer_block(const Args& p) { return blockIdx.z * p.grid_x + blockIdx.x; }

// ------------------------------------------------- activation and bias grads --
// dZ = dY * act'(Z), and sums of dZ over rows before it is rounded. dZ itself is
// rounded to the layer's type, since the matrix cores take 16-bit operands: dX and
// dW, which are rounded once more, come out 1.4 times as far from 64 bits as from a
// float32 dZ (bf16 2.35e-3 against 1.66e-3 in norm, f16 2.9e-4 against 2.1e-4; a
// second product with what the rounding left of dZ would take their time again).
// A wave
// takes p.rows rows of 512 columns (8 a lane) and keeps 8 float32 sums;
// where its rows cross from one group to the next it starts new ones. Neighbouring
// waves take neighbouring columns of the same rows (16384 x 2048 with SiLU 59 us
// where they took other rows, 64 KiB apart, 48 so). Rows
// block b and group g meet in at most one run of rows, and b + g is another
// number for each run (each next run has the next b or the next g), so the
// sums go to row b + g of the workspace. A second kernel adds each group's
// runs in order.
template <class Tag, int ACT>
__global__ void __launch_bounds__(256) layer_act_grad_kernel(const ActGradArgs p) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int blocks = (p.N + 511) / 512;  // of columns
  const unsigned id = layer_block(p) * 4 + w;
  const int b = id / blocks;
  const int c = (id - (unsigned)b * blocks) * 512 + lane * 8;
  const int nv = p.N - c >= 8 ? 8 : p.N - c;
  if ((int64_t)b * p.rows >= p.M || nv <= 0) return;
  const int r0 = b * p.rows, r1 = r0 + p.rows < p.M ? r0 + p.rows : p.M;
  // The group of the first row: the last one that starts at or before it.
  int g = 0, lo = 0, end = p.M;
  if (p.offsets) {
    int hi = p.G - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.offsets[mid] <= r0) lo = mid;
      else hi = mid - 1;
    }
    g = lo;
    end = p.offsets[g + 1];
  }
  const char* dY = static_cast<const char*>(p.dY);
  const char* Z = static_cast<const char*>(p.Z);
  char* dZ = static_cast<char*>(p.dZ);
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.0f;
  int r = r0;
  while (r < r1) {
    while (g < p.G && r >= end) {  // the next group with rows
      ++g;
      if (g < p.G) end = p.offsets[g + 1];
    }
    if (g >= p.G) break;  // rows of no group
    const int stop = end < r1 ? end : r1;
    // Rows in batches whose loads are all requested before the first store
    // (dZ may be dY or Z, so the compiler would not move them across).
    auto batch = [&](auto count) {
      constexpr int R = count.value;
      float d[R][8], z[R][8];
#pragma unroll
      for (int u = 0; u < R; ++u) {
        layer_load8_16<Tag>(dY + ((int64_t)(r + u) * p.lddy + c) * 2, nv, d[u]);
        if constexpr (ACT != ACT_NONE)
          layer_load8_16<Tag>(Z + ((int64_t)(r + u) * p.ldz + c) * 2, nv, z[u]);
      }
#pragma unroll
      for (int u = 0; u < R; ++u) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if constexpr (ACT != ACT_NONE) d[u][e] *= layer_slope<ACT>(z[u][e]);
          sum[e] += d[u][e];
        }
        if (dZ) layer_store8_16<Tag>(dZ + ((int64_t)(r + u) * p.lddz + c) * 2, nv, d[u]);
      }
      r += R;
    };
    while (r + 4 <= stop) batch(LayerConst<4>{});
    while (r < stop) batch(LayerConst<1>{});
    if (p.db) {
      float* out = p.part + (int64_t)(b + g) * p.N + c;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e < nv) out[e] = sum[e];
        sum[e] = 0.0f;
      }
    }
  }
}

// db[g][n]: the group's partial sums, every kSumWaves-th of them for each wave,
// joined in wave order.
constexpr int kSumWaves = 16;
__global__ void __launch_bounds__(64 * kSumWaves) layer_bias_sum_kernel(const ActGradArgs p) {
  __shared__ float x[kSumWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int g = blockIdx.y, n = layer_block(p) * 64 + lane;
  int first = 0, count = p.M;
  if (p.offsets) layer_group(p.offsets, g, p.M, first, count);
  float s = 0.0f;
  if (count > 0 && n < p.N) {
    const int b0 = first / p.rows, b1 = (first + count - 1) / p.rows;
    const float* part = p.part + (int64_t)g * p.N + n;
    int b = b0 + w;
    for (; b + 7 * kSumWaves <= b1; b += 8 * kSumWaves) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = part[(int64_t)(b + u * kSumWaves) * p.N];
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
    for (; b <= b1; b += kSumWaves) s += part[(int64_t)b * p.N];
  }
  x[w][lane] = s;
  __syncthreads();
  if (w == 0 && n < p.N) {
    s = x[0][lane];
#pragma unroll
    for (int u = 1; u < kSumWaves; ++u) s += x[u][lane];
    p.db[(int64_t)g * p.N + n] = s;
  }
}

template <class Tag>
hipError_t launch_act(const ActGradArgs& a, dim3 grid, hipStream_t s) {
  const dim3 block(256);
  switch (a.act) {
    case ACT_RELU:
      return launch_kernel(layer_act_grad_kernel<Tag, ACT_RELU>, grid, block, s, a);
    case ACT_GELU:
      return launch_kernel(layer_act_grad_kernel<Tag, ACT_GELU>, grid, block, s, a);
    case ACT_GELU_ERF:
      return launch_kernel(layer_act_grad_kernel<Tag, ACT_GELU_ERF>, grid, block, s, a);
    case ACT_SILU:
      return launch_kernel(layer_act_grad_kernel<Tag, ACT_SILU>, grid, block, s, a);
    default:
      return launch_kernel(layer_act_grad_kernel<Tag, ACT_NONE>, grid, block, s, a);
  }
}

// ----------------------------------------------------------------- dispatch --
template <int PIECE>
struct RowPiece;
template <>
struct RowPiece<16> { using type = u32x4; };
template <>
struct RowPiece<8> { using type = u32x2; };
template <>
struct RowPiece<4> { using type = unsigned; };
template <>
struct RowPiece<2> { using type = unsigned short; };

// A wave takes one token and kDispatchSpan pieces a lane: the row is read
// once, whatever the number of experts it goes to.
template <int PIECE>
__global__ void __launch_bounds__(256) layer_dispatch_kernel(const DispatchArgs p) {
  using V = typename RowPiece<PIECE>::type;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const unsigned t = layer_block(p) * 4 + w;
  if (t >= (unsigned)p.T) return;
  const int64_t at = ((int64_t)blockIdx.y * kDispatchSpan * 64 + lane) * PIECE;
  const char* src = p.X + (int64_t)t * p.ldx + at;
  V v[kDispatchSpan];
#pragma unroll
  for (int u = 0; u < kDispatchSpan; ++u)
    if (at + u * 64 * PIECE < p.bytes) v[u] = *reinterpret_cast<const V*>(src + u * 64 * PIECE);
  const int rows = p.T * p.top;
  for (int j = 0; j < p.top; ++j) {
    const int to = p.slot[(int64_t)t * p.top + j];
    if ((unsigned)to >= (unsigned)rows) continue;
    char* dst = p.Xs + (int64_t)to * p.ldxs + at;
#pragma unroll
    for (int u = 0; u < kDispatchSpan; ++u)
      if (at + u * 64 * PIECE < p.bytes) *reinterpret_cast<V*>(dst + u * 64 * PIECE) = v[u];
  }
}

// ------------------------------------------------------------------ combine --
// Elements of rows: loads and stores of E consecutive ones, as float32.
struct RowF32 {};
// ONCE: with the hint not to keep the bytes in the caches.
template <class Row, int E>
struct RowIo {  // 16-bit types
  using V = typename RowPiece<2 * E>::type;
  template <bool ONCE = false>
  __device__ static __forceinline__ void load(const void* base, int64_t at, float (&f)[E]) {
    const V* p = reinterpret_cast<const V*>(static_cast<const unsigned short*>(base) + at);
    const V v = ONCE ? __builtin_nontemporal_load(p) : *p;
    const unsigned short* s = reinterpret_cast<const unsigned short*>(&v);
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = layer_f32(Row{}, s[e]);
  }
  template <bool ONCE = false>
  __device__ static __forceinline__ void store(void* base, int64_t at, const float (&f)[E]) {
    V v;
    unsigned short* s = reinterpret_cast<unsigned short*>(&v);
#pragma unroll
    for (int e = 0; e < E; ++e) s[e] = layer_16(Row{}, f[e]);
    V* p = reinterpret_cast<V*>(static_cast<unsigned short*>(base) + at);
    if constexpr (ONCE) __builtin_nontemporal_store(v, p);
    else *p = v;
  }
};
template <int E>
struct RowIo<RowF32, E> {
  using V = typename RowPiece<4 * E>::type;
  template <bool ONCE = false>
  __device__ static __forceinline__ void load(const void* base, int64_t at, float (&f)[E]) {
    const V* p = reinterpret_cast<const V*>(static_cast<const float*>(base) + at);
    const V v = ONCE ? __builtin_nontemporal_load(p) : *p;
    __builtin_memcpy(f, &v, 4 * E);
  }
  template <bool ONCE = false>
  __device__ static __forceinline__ void store(void* base, int64_t at, const float (&f)[E]) {
    V v;
    __builtin_memcpy(&v, f, 4 * E);
    V* p = reinterpret_cast<V*>(static_cast<float*>(base) + at);
    if constexpr (ONCE) __builtin_nontemporal_store(v, p);
    else *p = v;
  }
};

// A wave takes SPAN pieces of E columns a lane of one token, and neighbouring
// waves the token's other columns, so that whole rows are read at about the same
// time. Four of the token's rows are in flight at a time, added in the order of
// its choices. ONCE: calls that move more than the caches hold ask them not to
// keep anything (16384 tokens of 4 rows of 4096: 158 us without, 127 for the
// rows that are read alone, 111 for all).
template <class Row, int E, int SPAN, bool ONCE>
__global__ void __launch_bounds__(256) layer_combine_kernel(const CombineArgs p) {
  using Io = RowIo<Row, E>;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const unsigned wid = layer_block(p) * 4 + w;
  const unsigned across = (p.H + SPAN * 64 * E - 1) / (SPAN * 64 * E);
  const unsigned t = __builtin_amdgcn_readfirstlane(wid / across);
  if (t >= (unsigned)p.T) return;
  const int c0 = ((wid - t * across) * SPAN * 64 + lane) * E;  // piece s: c0 + s * 64 * E
  const int rows = p.T * p.top;
  const int64_t t0 = (int64_t)t * p.top;
  float sum[SPAN][E];
#pragma unroll
  for (int s = 0; s < SPAN; ++s)
#pragma unroll
    for (int e = 0; e < E; ++e) sum[s][e] = 0.0f;
  for (int j0 = 0; j0 < p.top; j0 += 4) {
    float f[4][SPAN][E], wt[4];
    bool in[4];  // uniform
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + u;
      const int at = j < p.top ? p.slot[t0 + j] : -1;
      in[u] = (unsigned)at < (unsigned)rows;
      if (in[u]) {
#pragma unroll
        for (int s = 0; s < SPAN; ++s)
          if (c0 + s * 64 * E < p.H)
            Io::template load<ONCE>(p.Ys, (int64_t)at * p.ldys + c0 + s * 64 * E, f[u][s]);
        wt[u] = p.weights ? p.weights[t0 + j] : 1.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (in[u]) {
#pragma unroll
        for (int s = 0; s < SPAN; ++s)
#pragma unroll
          for (int e = 0; e < E; ++e) sum[s][e] = __builtin_fmaf(wt[u], f[u][s][e], sum[s][e]);
      }
  }
#pragma unroll
  for (int s = 0; s < SPAN; ++s) {
    const int64_t c = c0 + s * 64 * E;
    if (c >= p.H) continue;
    if (p.R) {
      float r[E];
      Io::template load<ONCE>(p.R, (int64_t)t * p.ldr + c, r);
#pragma unroll
      for (int e = 0; e < E; ++e) sum[s][e] += r[e];
    }
    Io::template store<ONCE>(p.Y, (int64_t)t * p.ldy + c, sum[s]);
  }
}

// W waves take one token; their lanes share the columns, and their parts of each
// choice's product are joined in lane and wave order. One wave where a row is
// short (10012 tokens of 2 rows of 144, with the forward pass: 30 us
// with four waves a token, 15 with one).
template <class Row, int E, int W>
__global__ void __launch_bounds__(256) layer_combine_grad_kernel(const CombineGradArgs p) {
  using Io = RowIo<Row, E>;
  __shared__ float part[4][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, w = wave % W;
  const int tid = w * 64 + lane;
  const unsigned t = W == 4 ? layer_block(p) : layer_block(p) * (4 / W) + wave / W;
  if (t >= (unsigned)p.T) return;  // (W == 4: the whole workgroup)
  const int rows = p.T * p.top;
  const int64_t t0 = (int64_t)t * p.top;
  for (int j0 = 0; j0 < p.top; j0 += 4) {
    int at[4];
    float wt[4], dot[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = j0 + u;
      at[u] = j < p.top ? p.slot[t0 + j] : -1;
      if ((unsigned)at[u] >= (unsigned)rows) at[u] = -1;
      wt[u] = at[u] >= 0 && p.weights ? p.weights[t0 + j] : 1.0f;
      dot[u] = 0.0f;
    }
    // S pieces of every row at once, 16 bytes or so a lane and row.
    constexpr int S = E >= 4 ? 1 : 4 / E;
    for (int64_t c0 = (int64_t)tid * E; c0 < p.H; c0 += 64 * W * E * S) {
      float d[S][E], y[4][S][E];
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int64_t c = c0 + s * 64 * W * E;
        if (c >= p.H) continue;
        Io::template load<true>(p.dY, (int64_t)t * p.lddy + c, d[s]);
        if (p.dw) {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (at[u] >= 0) Io::template load<true>(p.Ys, (int64_t)at[u] * p.ldys + c, y[u][s]);
        }
      }
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int64_t c = c0 + s * 64 * W * E;
        if (c >= p.H) continue;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (at[u] < 0) continue;
          if (p.dw) {
#pragma unroll
            for (int e = 0; e < E; ++e) dot[u] = __builtin_fmaf(d[s][e], y[u][s][e], dot[u]);
          }
          if (p.dYs) {
            float o[E];
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = wt[u] * d[s][e];
            Io::store(p.dYs, (int64_t)at[u] * p.lddys + c, o);
          }
        }
      }
    }
    if (p.dw) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
#pragma unroll
        for (int x = 1; x < 64; x <<= 1) dot[u] += __shfl_xor(dot[u], x, 64);
        if (W > 1 && lane == 0) part[w][u] = dot[u];
      }
      if constexpr (W == 1) {
        if (lane < 4 && j0 + lane < p.top)
          p.dw[t0 + j0 + lane] = lane == 0 ? dot[0] : lane == 1 ? dot[1] : lane == 2 ? dot[2] : dot[3];
      } else {
        __syncthreads();
        if (tid < 4 && j0 + tid < p.top)
          p.dw[t0 + j0 + tid] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
        __syncthreads();
      }
    }
  }
}

template <class Row, int E>
hipError_t combine(CombineArgs a, hipStream_t s) {
  const dim3 grid = layer_grid((combine_waves(a) + 3) / 4, 256, a.grid_x), block(256);
  if (a.once) return launch_kernel(layer_combine_kernel<Row, E, 2, true>, grid, block, s, a);
  if (combine_span(a) == 2) return launch_kernel(layer_combine_kernel<Row, E, 2, false>, grid, block, s, a);
  return launch_kernel(layer_combine_kernel<Row, E, 1, false>, grid, block, s, a);
}
template <class Row, int E>
hipError_t combine_grad(CombineGradArgs a, hipStream_t s) {
  const dim3 block(256);
  if (a.H <= 2 * 64 * E) {
    const dim3 grid = layer_grid(((int64_t)a.T + 3) / 4, 256, a.grid_x);
    return launch_kernel(layer_combine_grad_kernel<Row, E, 1>, grid, block, s, a);
  }
  const dim3 grid = layer_grid(a.T, 256, a.grid_x);
  return launch_kernel(layer_combine_grad_kernel<Row, E, 4>, grid, block, s, a);
}

}  // namespace

hipError_t launch_act_grad(int dtype, ActGradArgs a, hipStream_t s) {
  if (a.M > 0) {
    const dim3 grid = layer_grid((act_grad_waves(a.M, a.N) + 3) / 4, 256, a.grid_x);
    const hipError_t e = dtype == 0 ? launch_act<TagF16>(a, grid, s) : launch_act<TagBF16>(a, grid, s);
    if (e != hipSuccess) return e;
  }
  if (!a.db) return hipSuccess;
  const dim3 grid = layer_grid(((int64_t)a.N + 63) / 64, 64 * kSumWaves, a.grid_x, a.G);
  return launch_kernel(layer_bias_sum_kernel, grid, dim3(64 * kSumWaves), s, a);
}

hipError_t launch_dispatch(DispatchArgs a, hipStream_t s) {
  const dim3 grid = layer_grid(((int64_t)a.T + 3) / 4, 256, a.grid_x, (unsigned)dispatch_column_blocks(a));
  const dim3 block(256);
  if (a.piece == 16) return launch_kernel(layer_dispatch_kernel<16>, grid, block, s, a);
  if (a.piece == 8) return launch_kernel(layer_dispatch_kernel<8>, grid, block, s, a);
  if (a.piece == 4) return launch_kernel(layer_dispatch_kernel<4>, grid, block, s, a);
  return launch_kernel(layer_dispatch_kernel<2>, grid, block, s, a);
}

hipError_t launch_combine(int rowtype, const CombineArgs& a, hipStream_t s) {
  if (rowtype == ROW_F32) {
    if (a.piece == 4) return combine<RowF32, 4>(a, s);
    if (a.piece == 2) return combine<RowF32, 2>(a, s);
    return combine<RowF32, 1>(a, s);
  }
  if (rowtype == ROW_F16) {
    if (a.piece == 8) return combine<TagF16, 8>(a, s);
    if (a.piece == 4) return combine<TagF16, 4>(a, s);
    if (a.piece == 2) return combine<TagF16, 2>(a, s);
    return combine<TagF16, 1>(a, s);
  }
  if (a.piece == 8) return combine<TagBF16, 8>(a, s);
  if (a.piece == 4) return combine<TagBF16, 4>(a, s);
  if (a.piece == 2) return combine<TagBF16, 2>(a, s);
  return combine<TagBF16, 1>(a, s);
}

hipError_t launch_combine_grad(int rowtype, const CombineGradArgs& a, hipStream_t s) {
  if (rowtype == ROW_F32) {
    if (a.piece == 4) return combine_grad<RowF32, 4>(a, s);
    if (a.piece == 2) return combine_grad<RowF32, 2>(a, s);
    return combine_grad<RowF32, 1>(a, s);
  }
  if (rowtype == ROW_F16) {
    if (a.piece == 8) return combine_grad<TagF16, 8>(a, s);
    if (a.piece == 4) return combine_grad<TagF16, 4>(a, s);
    if (a.piece == 2) return combine_grad<TagF16, 2>(a, s);
    return combine_grad<TagF16, 1>(a, s);
  }
  if (a.piece == 8) return combine_grad<TagBF16, 8>(a, s);
  if (a.piece == 4) return combine_grad<TagBF16, 4>(a, s);
  if (a.piece == 2) return combine_grad<TagBF16, 2>(a, s);
  return combine_grad<TagBF16, 1>(a, s);
}

}  // namespace dgt
