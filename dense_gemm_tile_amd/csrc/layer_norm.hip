// Layer norm and its gradients.
//
//   mean, rstd of a row;  U = (X - mean) rstd;  Y = U gamma + beta
//   H = dY gamma:  dX = rstd (H - mean(H) - U mean(H U)) + R
//   dgamma = sum over rows of dY U,  dbeta = sum over rows of dY
//
// All sums are float32. The variance is summed from differences to the mean, never
// as a difference of two sums.
#include "layer.h"
#include "layer_checks.h"
#include "layer_norm.h"

namespace dgt {

namespace {

// Eight elements of a row of any type. ONCE: with the hint not to keep the bytes in the
// caches, for calls whose rows fill half of the last one (256 MiB) or more (gradients of
// 16384 x 4096 bf16: 113 us without, 93 so).
struct NormF32 {};
template <bool ONCE, class V>
__device__ __forceinline__ V norm_load(const V* p) {
  if constexpr (ONCE) return __builtin_nontemporal_load(p);
  else return *p;
}
template <bool ONCE, class V>
__device__ __forceinline__ void norm_store(V* p, V v) {
  if constexpr (ONCE) __builtin_nontemporal_store(v, p);
  else *p = v;
}
template <class Row>
struct NormIo {
  static constexpr int SIZE = 2;
  template <bool ONCE = false>
  __device__ static __forceinline__ void load(const char* p, int nv, float (&f)[8]) {
    if (ONCE && nv == 8) layer_unpack8<Row>(norm_load<ONCE>(reinterpret_cast<const u32x4_at2*>(p)), f);
    else layer_load8_16<Row>(p, nv, f);
  }
  template <bool ONCE = false>
  __device__ static __forceinline__ void store(char* p, int nv, const float (&f)[8]) {
    if (ONCE && nv == 8) norm_store<ONCE>(reinterpret_cast<u32x4_at2*>(p), u32x4_at2(layer_pack8<Row>(f)));
    else layer_store8_16<Row>(p, nv, f);
  }
};
template <>
struct NormIo<NormF32> {
  static constexpr int SIZE = 4;
  template <bool ONCE = false>
  __device__ static __forceinline__ void load(const char* p, int nv, float (&f)[8]) {
    if (ONCE && nv == 8) {
      const u32x4_at4* v = reinterpret_cast<const u32x4_at4*>(p);
      const f32x4 lo = __builtin_bit_cast(f32x4, u32x4(norm_load<ONCE>(v))), hi = __builtin_bit_cast(f32x4, u32x4(norm_load<ONCE>(v + 1)));
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] = lo[e], f[e + 4] = hi[e];
    } else {
      layer_load8_32(p, nv, f);
    }
  }
  template <bool ONCE = false>
  __device__ static __forceinline__ void store(char* p, int nv, const float (&f)[8]) {
    if (ONCE && nv == 8) {
      u32x4_at4* v = reinterpret_cast<u32x4_at4*>(p);
      norm_store<ONCE>(v, u32x4_at4(__builtin_bit_cast(u32x4, f32x4{f[0], f[1], f[2], f[3]})));
      norm_store<ONCE>(v + 1, u32x4_at4(__builtin_bit_cast(u32x4, f32x4{f[4], f[5], f[6], f[7]})));
    } else {
      layer_store8_32(p, nv, f);
    }
  }
};

// Gamma and beta: eight elements, or a constant where there are none.
template <class Row>
__device__ __forceinline__ void norm_param(const char* p, int c, int nv, float none, float (&f)[8]) {
  if (p) {
    NormIo<Row>::load(p + (int64_t)c * NormIo<Row>::SIZE, nv, f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = none;
  }
}

__device__ __forceinline__ int norm_left(int N, int c) { return N - c >= 8 ? 8 : N - c; }

// A sum over the wave, the same in every lane.
__device__ __forceinline__ float norm_wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}
// Two sums over a workgroup of `waves` waves, the same in every thread. part: 2 * waves floats.
__device__ __forceinline__ void norm_block_sum(float& a, float& b, float* part, int waves) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  a = norm_wave_sum(a);
  b = norm_wave_sum(b);
  __syncthreads();  // the last use of part is over
  if (lane == 0) {
    part[2 * w] = a;
    part[2 * w + 1] = b;
  }
  __syncthreads();
  a = b = 0.0f;
  for (int u = 0; u < waves; ++u) {
    a += part[2 * u];
    b += part[2 * u + 1];
  }
}

// A piece as it is stored, between its load and its use.
template <class Row>
struct NormRaw {
  u32x4 v;
  template <bool ONCE>
  __device__ __forceinline__ void load(const char* p, int nv) {
    if (nv == 8) {
      v = norm_load<ONCE>(reinterpret_cast<const u32x4_at2*>(p));
    } else {
      v = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int e = 0; e < 7; ++e)
        if (e < nv) v[e / 2] |= (unsigned)reinterpret_cast<const unsigned short*>(p)[e] << (16 * (e % 2));
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const { layer_unpack8<Row>(v, f); }
};
template <>
struct NormRaw<NormF32> {
  float v[8];
  template <bool ONCE>
  __device__ __forceinline__ void load(const char* p, int nv) { NormIo<NormF32>::load<ONCE>(p, nv, v); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = v[e];
  }
};

// -------------------------------------------------- rows held in registers --
// W waves take a row, V pieces of 8 columns a lane (piece v at column 8 (lane of the row + 64 W
// v)), and hold it from its one reading to its writing. Four waves a workgroup, or one row
// of more.

// A sum over each group of W waves that share a row. part: two places per wave, used in turn.
template <int W>
__device__ __forceinline__ void norm_join(float& a, float& b, float (*part)[2]) {
  a = norm_wave_sum(a);
  b = norm_wave_sum(b);
  if constexpr (W > 1) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      part[wave][0] = a;
      part[wave][1] = b;
    }
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int u = 0; u < W; ++u) {
      a += part[wave / W * W + u][0];
      b += part[wave / W * W + u][1];
    }
  }
}

template <class Row, int W, int V, bool ONCE>
__global__ void __launch_bounds__(W > 4 ? 64 * W : 256) layer_norm_kernel(const NormArgs p) {
  using Io = NormIo<Row>;
  constexpr int ROWS = W > 4 ? 1 : 4 / W, SPAN = 64 * W * 8;
  __shared__ float part[2][W * ROWS][2];
  const int lane = threadIdx.x % (64 * W);
  const int64_t at = (int64_t)layer_block(p) * ROWS + threadIdx.x / (64 * W);
  const int64_t row = at < p.M ? at : p.M - 1;  // (waves past the last row meet its barriers)
  const char* x = static_cast<const char*>(p.X) + row * p.ldx * Io::SIZE;
  const float inv = 1.0f / (float)p.N;
  float f[V][8], sum = 0.0f, sq = 0.0f, none = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * lane + v * SPAN, nv = norm_left(p.N, c);
    if (nv > 0) Io::template load<ONCE>(x + (int64_t)c * Io::SIZE, nv, f[v]);
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (8 * lane + v * SPAN + e >= p.N) f[v][e] = 0.0f;
      sum += f[v][e];
    }
  norm_join<W>(sum, none, part[0]);
  const float mean = sum * inv;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float d = f[v][e] - mean;
      sq = 8 * lane + v * SPAN + e < p.N ? __builtin_fmaf(d, d, sq) : sq;
    }
  none = 0.0f;
  norm_join<W>(sq, none, part[1]);
  const float rstd = 1.0f / __builtin_sqrtf(sq * inv + p.eps);
  if (at >= p.M) return;
  char* y = static_cast<char*>(p.Y) + row * p.ldy * Io::SIZE;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * lane + v * SPAN, nv = norm_left(p.N, c);
    if (nv <= 0) continue;
    float g[8], b[8];
    norm_param<Row>(static_cast<const char*>(p.gamma), c, nv, 1.0f, g);
    norm_param<Row>(static_cast<const char*>(p.beta), c, nv, 0.0f, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[v][e] = __builtin_fmaf((f[v][e] - mean) * rstd, g[e], b[e]);
    Io::template store<ONCE>(y + (int64_t)c * Io::SIZE, nv, f[v]);
  }
  if (lane == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
}

// Each workgroup takes rows a grid apart, with the next row's pieces asked for before the row
// at hand is finished; dY U and dY are summed over them in registers, then over the rows
// that the workgroup has at hand, and written as one part.
template <class Row, int W, int V, bool ONCE>
__global__ void __launch_bounds__(W > 4 ? 64 * W : 256) layer_norm_grad_kernel(const NormGradArgs p) {
  using Io = NormIo<Row>;
  constexpr int ROWS = W > 4 ? 1 : 4 / W, SPAN = 64 * W * 8;
  __shared__ float part[2][W * ROWS][2];
  __shared__ float joined[ROWS > 1 ? 2 * SPAN * V : 1];
  const int lane = threadIdx.x % (64 * W), sub = threadIdx.x / (64 * W);
  const int64_t block = layer_block(p), first = block * ROWS + sub;
  if (block >= p.parts) return;
  const float inv = 1.0f / (float)p.N;
  float g[V][8], sg[V][8], sb[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = 8 * lane + v * SPAN, nv = norm_left(p.N, c);
    if (nv > 0) norm_param<Row>(static_cast<const char*>(p.gamma), c, nv, 1.0f, g[v]);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (c + e >= p.N) g[v][e] = 0.0f;
      sg[v][e] = sb[v][e] = 0.0f;
    }
  }
  NormRaw<Row> x[V], d[V], r[V];
  float mean = 0.0f, rstd = 0.0f;
  auto request = [&](int64_t row) {
    mean = p.mean[row];
    rstd = p.rstd[row];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int64_t c = 8 * lane + v * SPAN;
      const int nv = norm_left(p.N, (int)c);
      if (nv <= 0) continue;
      x[v].template load<ONCE>(static_cast<const char*>(p.X) + (row * p.ldx + c) * Io::SIZE, nv);
      d[v].template load<ONCE>(static_cast<const char*>(p.dY) + (row * p.lddy + c) * Io::SIZE, nv);
      if (p.R) r[v].template load<ONCE>(static_cast<const char*>(p.R) + (row * p.ldr + c) * Io::SIZE, nv);
    }
  };
  // Every wave of a workgroup takes as many turns, so that all meet the barriers.
  const int64_t step = (int64_t)p.parts * ROWS, turns = (p.M - block * ROWS + step - 1) / step;
  auto clamp = [&](int64_t row) { return row < p.M ? row : p.M - 1; };
  request(clamp(first));
  for (int64_t turn = 0; turn < turns; ++turn) {
    const int64_t row = first + turn * step;
    const bool in = row < p.M;
    float u[V][8], h[V][8], rr[V][8], s1 = 0.0f, s2 = 0.0f;
    const float m = mean, rs = rstd;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      x[v].get(u[v]);
      d[v].get(h[v]);
      if (p.R) r[v].get(rr[v]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // (A row that is not there reads the last one, where dX may stand by now: no element of it counts.)
        const bool has = in && 8 * lane + v * SPAN + e < p.N;
        u[v][e] = has ? (u[v][e] - m) * rs : 0.0f;
        h[v][e] = has ? h[v][e] : 0.0f;
        sg[v][e] = __builtin_fmaf(h[v][e], u[v][e], sg[v][e]);
        sb[v][e] += h[v][e];
        h[v][e] *= g[v][e];
        s1 += h[v][e];
        s2 = __builtin_fmaf(h[v][e], u[v][e], s2);
      }
    }
    if (turn + 1 < turns) request(clamp(row + step));
    norm_join<W>(s1, s2, part[turn & 1]);
    s1 *= inv;
    s2 *= inv;
    if (p.dX && in) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int64_t c = 8 * lane + v * SPAN;
        const int nv = norm_left(p.N, (int)c);
        if (nv <= 0) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          h[v][e] = rs * (h[v][e] - s1 - u[v][e] * s2);
          if (p.R) h[v][e] += rr[v][e];
        }
        Io::template store<ONCE>(static_cast<char*>(p.dX) + (row * p.lddx + c) * Io::SIZE, nv, h[v]);
      }
    }
  }
  if (!p.part) return;
  if constexpr (ROWS > 1) {
#pragma unroll
    for (int turn = 0; turn < ROWS; ++turn) {
      if (sub == turn) {
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float* const at = joined + (v * 8 + e) * 64 * W + lane;
            sg[v][e] = turn ? at[0] + sg[v][e] : sg[v][e];
            sb[v][e] = turn ? at[SPAN * V] + sb[v][e] : sb[v][e];
            at[0] = sg[v][e];
            at[SPAN * V] = sb[v][e];
          }
      }
      __syncthreads();
    }
    if (sub != ROWS - 1) return;
  }
  float* out = p.part + 2 * block * p.N;
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = 8 * lane + v * SPAN + e;
      if (c < p.N) {
        out[c] = sg[v][e];
        out[p.N + c] = sb[v][e];
      }
    }
}

// ------------------------------------------------------------------ any row --
// A workgroup a row, which it reads once for every sum.
constexpr int kLongThreads = 512, kLongWaves = kLongThreads / 64;

template <class Row>
__global__ void __launch_bounds__(kLongThreads) layer_norm_long_kernel(const NormArgs p) {
  using Io = NormIo<Row>;
  __shared__ float part[2 * kLongWaves];
  const int64_t row = layer_block(p);
  if (row >= p.M) return;
  const char* x = static_cast<const char*>(p.X) + row * p.ldx * Io::SIZE;
  char* y = static_cast<char*>(p.Y) + row * p.ldy * Io::SIZE;
  const float inv = 1.0f / (float)p.N;
  float sum = 0.0f, none = 0.0f;
  for (int64_t c = 8 * threadIdx.x; c < p.N; c += 8 * kLongThreads) {
    float f[8];
    const int nv = norm_left(p.N, (int)c);
    Io::load(x + c * Io::SIZE, nv, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum += e < nv ? f[e] : 0.0f;
  }
  norm_block_sum(sum, none, part, kLongWaves);
  const float mean = sum * inv;
  float sq = 0.0f;
  for (int64_t c = 8 * threadIdx.x; c < p.N; c += 8 * kLongThreads) {
    float f[8];
    const int nv = norm_left(p.N, (int)c);
    Io::load(x + c * Io::SIZE, nv, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) sq += e < nv ? (f[e] - mean) * (f[e] - mean) : 0.0f;
  }
  none = 0.0f;
  norm_block_sum(sq, none, part, kLongWaves);
  const float rstd = 1.0f / __builtin_sqrtf(sq * inv + p.eps);
  for (int64_t c = 8 * threadIdx.x; c < p.N; c += 8 * kLongThreads) {
    float f[8], g[8], b[8];
    const int nv = norm_left(p.N, (int)c);
    Io::load(x + c * Io::SIZE, nv, f);
    norm_param<Row>(static_cast<const char*>(p.gamma), (int)c, nv, 1.0f, g);
    norm_param<Row>(static_cast<const char*>(p.beta), (int)c, nv, 0.0f, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = __builtin_fmaf((f[e] - mean) * rstd, g[e], b[e]);
    Io::store(y + c * Io::SIZE, nv, f);
  }
  if (threadIdx.x == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
}

// dX of one row.
template <class Row>
__global__ void __launch_bounds__(kLongThreads) layer_norm_grad_long_kernel(const NormGradArgs p) {
  using Io = NormIo<Row>;
  __shared__ float part[2 * kLongWaves];
  const int64_t row = layer_block(p);
  if (row >= p.M) return;
  const char* x = static_cast<const char*>(p.X) + row * p.ldx * Io::SIZE;
  const char* dy = static_cast<const char*>(p.dY) + row * p.lddy * Io::SIZE;
  const char* r = static_cast<const char*>(p.R) + row * p.ldr * Io::SIZE;
  char* dx = static_cast<char*>(p.dX) + row * p.lddx * Io::SIZE;
  const float mean = p.mean[row], rstd = p.rstd[row], inv = 1.0f / (float)p.N;
  auto piece = [&](int64_t c, int nv, float (&h)[8], float (&u)[8]) {
    float g[8];
    Io::load(x + c * Io::SIZE, nv, u);
    Io::load(dy + c * Io::SIZE, nv, h);
    norm_param<Row>(static_cast<const char*>(p.gamma), (int)c, nv, 1.0f, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      u[e] = (u[e] - mean) * rstd;
      h[e] *= g[e];
    }
  };
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t c = 8 * threadIdx.x; c < p.N; c += 8 * kLongThreads) {
    float h[8], u[8];
    const int nv = norm_left(p.N, (int)c);
    piece(c, nv, h, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s1 += e < nv ? h[e] : 0.0f;
      s2 += e < nv ? h[e] * u[e] : 0.0f;
    }
  }
  norm_block_sum(s1, s2, part, kLongWaves);
  s1 *= inv;
  s2 *= inv;
  for (int64_t c = 8 * threadIdx.x; c < p.N; c += 8 * kLongThreads) {
    float h[8], u[8];
    const int nv = norm_left(p.N, (int)c);
    piece(c, nv, h, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) h[e] = rstd * (h[e] - s1 - u[e] * s2);
    if (p.R) {
      Io::load(r + c * Io::SIZE, nv, u);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] += u[e];
    }
    Io::store(dx + c * Io::SIZE, nv, h);
  }
}

// Partial sums of dgamma and dbeta: a wave takes 512 columns (8 a lane) of p.rows rows.
template <class Row>
__global__ void __launch_bounds__(256) layer_norm_grad_columns_kernel(const NormGradArgs p) {
  using Io = NormIo<Row>;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t across = ((int64_t)p.N + 511) / 512, id = (int64_t)layer_block(p) * 4 + w;
  const int64_t b = id / across, c = (id - b * across) * 512 + 8 * lane;
  if (b >= p.parts || c >= p.N) return;
  const int nv = norm_left(p.N, (int)c);
  const int64_t r0 = b * p.rows, r1 = r0 + p.rows < p.M ? r0 + p.rows : p.M;
  float sg[8], sb[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sg[e] = sb[e] = 0.0f;
  for (int64_t r = r0; r < r1; ++r) {
    float x[8], d[8];
    const float mean = p.mean[r], rstd = p.rstd[r];
    Io::load(static_cast<const char*>(p.X) + (r * p.ldx + c) * Io::SIZE, nv, x);
    Io::load(static_cast<const char*>(p.dY) + (r * p.lddy + c) * Io::SIZE, nv, d);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sg[e] = __builtin_fmaf(d[e], (x[e] - mean) * rstd, sg[e]);
      sb[e] += d[e];
    }
  }
  float* out = p.part + 2 * b * p.N + c;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < nv) {
      out[e] = sg[e];
      out[p.N + e] = sb[e];
    }
}

// dgamma and dbeta: the parts, every kSumWaves-th of them for each wave, joined in wave order.
constexpr int kSumWaves = 16;
__global__ void __launch_bounds__(64 * kSumWaves) layer_norm_sum_kernel(const NormGradArgs p) {
  __shared__ float x[kSumWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  float* const to = blockIdx.y ? p.dbeta : p.dgamma;
  if (!to) return;
  const int64_t n = (int64_t)layer_block(p) * 64 + lane;
  float s = 0.0f;
  if (n < p.N) {
    const float* part = p.part + (blockIdx.y ? p.N : 0) + n;
    int b = w;
    for (; b + 7 * kSumWaves < p.parts; b += 8 * kSumWaves) {
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = part[2 * (int64_t)(b + u * kSumWaves) * p.N];
#pragma unroll
      for (int u = 0; u < 8; ++u) s += v[u];
    }
    for (; b < p.parts; b += kSumWaves) s += part[2 * (int64_t)b * p.N];
  }
  x[w][lane] = s;
  __syncthreads();
  if (w == 0 && n < p.N) {
    s = x[0][lane];
#pragma unroll
    for (int u = 1; u < kSumWaves; ++u) s += x[u][lane];
    to[n] = s;
  }
}

// Waves a row and pieces a lane that hold N columns, by rising width.
constexpr int kNormForms = 7;
constexpr int kNormWaves[kNormForms] = {1, 1, 2, 4, 4, 16, 16}, kNormPieces[kNormForms] = {1, 2, 2, 2, 4, 2, 4};
int norm_form(int64_t N) {
  int f = 0;
  while (f < kNormForms && (int64_t)kNormWaves[f] * kNormPieces[f] * 512 < N) ++f;
  return f;
}
int norm_form_rows(int form) { return kNormWaves[form] > 4 ? 1 : 4 / kNormWaves[form]; }
template <class F>
hipError_t norm_for(int form, F f) {
  switch (form) {
    case 0: return f(LayerConst<1>{}, LayerConst<1>{});
    case 1: return f(LayerConst<1>{}, LayerConst<2>{});
    case 2: return f(LayerConst<2>{}, LayerConst<2>{});
    case 3: return f(LayerConst<4>{}, LayerConst<2>{});
    case 4: return f(LayerConst<4>{}, LayerConst<4>{});
    case 5: return f(LayerConst<16>{}, LayerConst<2>{});
    default: return f(LayerConst<16>{}, LayerConst<4>{});
  }
}

template <class Row, class Args>
bool norm_once(const Args& a) { return (int64_t)a.M * a.N * NormIo<Row>::SIZE >= (int64_t{128} << 20); }

template <class Row>
hipError_t norm(NormArgs a, hipStream_t s) {
  const int form = norm_form(a.N);
  if (form < kNormForms) {
    const int rows = norm_form_rows(form), threads = kNormWaves[form] > 4 ? 64 * kNormWaves[form] : 256;
    const dim3 grid = layer_grid(((int64_t)a.M + rows - 1) / rows, threads, a.grid_x);
    return norm_for(form, [&](auto w, auto v) {
      constexpr int W = decltype(w)::value, V = decltype(v)::value;
      if (norm_once<Row>(a)) return launch_kernel(layer_norm_kernel<Row, W, V, true>, grid, dim3(threads), s, a);
      return launch_kernel(layer_norm_kernel<Row, W, V, false>, grid, dim3(threads), s, a);
    });
  }
  const dim3 grid = layer_grid(a.M, kLongThreads, a.grid_x);
  return launch_kernel(layer_norm_long_kernel<Row>, grid, dim3(kLongThreads), s, a);
}

// The same for the gradients, which hold more for each column: wider rows are read again.
constexpr int kNormGradForms = 5;
constexpr int kNormGradWaves[kNormGradForms] = {1, 1, 2, 4, 8}, kNormGradPieces[kNormGradForms] = {1, 2, 2, 2, 2};
int norm_grad_form(int64_t N) {
  int f = 0;
  while (f < kNormGradForms && (int64_t)kNormGradWaves[f] * kNormGradPieces[f] * 512 < N) ++f;
  return f;
}
int norm_grad_rows(int form) { return form == kNormGradForms || kNormGradWaves[form] > 4 ? 1 : 4 / kNormGradWaves[form]; }
template <class F>
hipError_t norm_grad_for(int form, F f) {
  switch (form) {
    case 0: return f(LayerConst<1>{}, LayerConst<1>{});
    case 1: return f(LayerConst<1>{}, LayerConst<2>{});
    case 2: return f(LayerConst<2>{}, LayerConst<2>{});
    case 3: return f(LayerConst<4>{}, LayerConst<2>{});
    default: return f(LayerConst<8>{}, LayerConst<2>{});
  }
}

template <class Row>
hipError_t norm_grad(NormGradArgs a, hipStream_t s) {
  const int form = norm_grad_form(a.N);
  const bool sums = a.dgamma || a.dbeta;
  if (!sums) a.part = nullptr;
  if (form < kNormGradForms) {
    if (a.M > 0) {
      const int threads = kNormGradWaves[form] > 4 ? 64 * kNormGradWaves[form] : 256;
      const dim3 grid = layer_grid(a.parts, threads, a.grid_x);
      const hipError_t e = norm_grad_for(form, [&](auto w, auto v) {
        constexpr int W = decltype(w)::value, V = decltype(v)::value;
        if (norm_once<Row>(a)) return launch_kernel(layer_norm_grad_kernel<Row, W, V, true>, grid, dim3(threads), s, a);
        return launch_kernel(layer_norm_grad_kernel<Row, W, V, false>, grid, dim3(threads), s, a);
      });
      if (e != hipSuccess) return e;
    }
  } else if (sums && a.M > 0) {
    const dim3 grid = layer_grid((a.parts * (((int64_t)a.N + 511) / 512) + 3) / 4, 256, a.grid_x);
    const hipError_t e = launch_kernel(layer_norm_grad_columns_kernel<Row>, grid, dim3(256), s, a);
    if (e != hipSuccess) return e;
  }
  if (sums) {
    const dim3 grid = layer_grid(((int64_t)a.N + 63) / 64, 64 * kSumWaves, a.grid_x, 2);
    const hipError_t e = launch_kernel(layer_norm_sum_kernel, grid, dim3(64 * kSumWaves), s, a);
    if (e != hipSuccess) return e;
  }
  if (form < kNormGradForms || !a.dX || a.M == 0) return hipSuccess;
  const dim3 grid = layer_grid(a.M, kLongThreads, a.grid_x);
  return launch_kernel(layer_norm_grad_long_kernel<Row>, grid, dim3(kLongThreads), s, a);
}

// Workgroups, and so partial sums of dgamma and dbeta: two a CU (16384 x 4096 bf16, us: 256
// workgroups 128, 512 117, 1024 128 with the partial sums joined).
int64_t norm_parts(int64_t m, int64_t n) {
  const int64_t rows = norm_grad_rows(norm_grad_form(n)), most = 512;
  const int64_t all = (m + rows - 1) / rows;
  return all < most ? all : most;
}

int64_t norm_grad_bytes(int64_t M, int64_t N) {
  if (M < 0 || N < 0 || M > kMaxDim || N > kMaxDim) return 0;
  return norm_parts(M, N) * N * 8;
}

int check_norm(int64_t M, int64_t N, int dtype, int& rowtype, int& elem) {
  CHECK(check_dim("M", M));
  CHECK(check_dim("N", N));
  if (N < 1) return bad("%s=%lld: a row needs an element", "N", N);
  return check_rowtype(dtype, rowtype, elem);
}

}  // namespace
}  // namespace dgt

using namespace dgt;

extern "C" {

int gemm_norm(int64_t M, int64_t N, int dtype, const void* X, int64_t ldx, const void* gamma,
              const void* beta, float eps, void* Y, int64_t ldy, float* mean, float* rstd,
              void* stream) {
  return entry("norm", M, N, 0, [&]() -> int {
    int rowtype, elem;
    CHECK(check_norm(M, N, dtype, rowtype, elem));
    const Mat mx{"X", X, M, N, ldx, elem}, my{"Y", Y, M, N, ldy, elem};
    const Mat mg{"gamma", gamma, 1, N, N, elem}, mb{"beta", beta, 1, N, N, elem};
    const Mat mm{"mean", mean, 1, M, M, 4}, mr{"rstd", rstd, 1, M, M, 4};
    CHECK(check_ld(mx));
    CHECK(check_ld(my));
    if (!(eps >= 0.0f) || eps > 3.4028234e38f)
      return fail(GEMM_ERR_INVALID_ARG, "eps is negative or not finite");
    if (M == 0) {
      set_path("noop: empty output");
      return GEMM_OK;
    }
    CHECK(check_ptr(mx));
    CHECK(check_ptr(my));
    for (const Mat* m : {&mg, &mb, &mm, &mr})
      if (m->ptr) CHECK(check_ptr(*m));
    CHECK(check_apart_or_same(my, mx));
    for (const Mat* w : {&my, &mm, &mr})
      for (const Mat* r : {&mg, &mb}) CHECK(check_apart(*w, *r));
    for (const Mat* w : {&mm, &mr})
      for (const Mat* r : {&mx, &my}) CHECK(check_apart(*w, *r));
    CHECK(check_apart(mr, mm));
    NormArgs a{};
    a.X = X;
    a.gamma = gamma;
    a.beta = beta;
    a.Y = Y;
    a.mean = mean;
    a.rstd = rstd;
    a.ldx = ldx;
    a.ldy = ldy;
    a.eps = eps;
    a.M = (int)M;
    a.N = (int)N;
    hipStream_t s = static_cast<hipStream_t>(stream);
    set_path("norm row by row");
    return launched(rowtype == ROW_F32   ? norm<NormF32>(a, s)
                    : rowtype == ROW_F16 ? norm<TagF16>(a, s)
                                         : norm<TagBF16>(a, s));
  });
}

int64_t gemm_norm_grad_workspace(int64_t M, int64_t N) { return norm_grad_bytes(M, N); }

int gemm_norm_grad(int64_t M, int64_t N, int dtype, const void* dY, int64_t lddy, const void* X,
                   int64_t ldx, const void* gamma, const float* mean, const float* rstd,
                   const void* R, int64_t ldr, void* dX, int64_t lddx, float* dgamma, float* dbeta,
                   void* workspace, int64_t workspace_bytes, void* stream) {
  return entry("norm_grad", M, N, 0, [&]() -> int {
    int rowtype, elem;
    CHECK(check_norm(M, N, dtype, rowtype, elem));
    const bool sums = dgamma || dbeta;
    const int64_t need = sums ? norm_grad_bytes(M, N) : 0;
    const Mat my{"dY", dY, M, N, lddy, elem}, mx{"X", X, M, N, ldx, elem};
    const Mat mr{"R", dX ? R : nullptr, M, N, ldr, elem}, md{"dX", dX, M, N, lddx, elem};
    const Mat mg{"gamma", gamma, 1, N, N, elem};
    const Mat mm{"mean", mean, 1, M, M, 4}, ms{"rstd", rstd, 1, M, M, 4};
    const Mat mdg{"dgamma", dgamma, 1, N, N, 4}, mdb{"dbeta", dbeta, 1, N, N, 4};
    const Mat mw{"workspace", need ? workspace : nullptr, 1, need, need, 1};
    CHECK(check_ld(my));
    CHECK(check_ld(mx));
    if (R && dX) CHECK(check_ld(mr));
    if (dX) CHECK(check_ld(md));
    if ((M == 0 && !sums) || (!dX && !sums)) {
      set_path("noop: empty output");
      return GEMM_OK;
    }
    if (M > 0) {
      for (const Mat* m : {&my, &mx, &mm, &ms}) CHECK(check_ptr(*m));
      for (const Mat* m : {&mr, &md, &mg})
        if (m->ptr) CHECK(check_ptr(*m));
    }
    for (const Mat* m : {&mdg, &mdb})
      if (m->ptr) CHECK(check_ptr(*m));
    CHECK(check_workspace(workspace, workspace_bytes, need));
    for (const Mat* r : {&my, &mx, &mr}) CHECK(check_apart_or_same(md, *r));
    for (const Mat* r : {&mg, &mm, &ms}) CHECK(check_apart(md, *r));
    const Mat* writes[] = {&md, &mdg, &mdb, &mw};
    for (const Mat* w : {&mdg, &mdb, &mw})
      for (const Mat* r : {&my, &mx, &mr, &mg, &mm, &ms}) CHECK(check_apart(*w, *r));
    for (int i = 0; i < 4; ++i)
      for (int j = i + 1; j < 4; ++j) CHECK(check_apart(*writes[j], *writes[i]));
    NormGradArgs a{};
    a.dY = dY;
    a.X = X;
    a.gamma = gamma;
    a.mean = mean;
    a.rstd = rstd;
    a.R = dX ? R : nullptr;
    a.dX = dX;
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.part = static_cast<float*>(workspace);
    a.lddy = lddy;
    a.ldx = ldx;
    a.ldr = ldr;
    a.lddx = lddx;
    a.M = (int)M;
    a.N = (int)N;
    a.parts = (int)norm_parts(M, N);
    a.rows = M ? (int)((M + a.parts - 1) / a.parts) : 1;
    hipStream_t s = static_cast<hipStream_t>(stream);
    set_path("norm_grad row by row");
    return launched(rowtype == ROW_F32   ? norm_grad<NormF32>(a, s)
                    : rowtype == ROW_F16 ? norm_grad<TagF16>(a, s)
                                         : norm_grad<TagBF16>(a, s));
  });
}

}  // extern "C"
