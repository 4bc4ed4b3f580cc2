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

// Eight elements of a row of any type.
struct NormF32 {};
template <class Row>
struct NormIo {
  static constexpr int SIZE = 2;
  __device__ static __forceinline__ void load(const char* p, int nv, float (&f)[8]) { layer_load8_16<Row>(p, nv, f); }
  __device__ static __forceinline__ void store(char* p, int nv, const float (&f)[8]) { layer_store8_16<Row>(p, nv, f); }
};
template <>
struct NormIo<NormF32> {
  static constexpr int SIZE = 4;
  __device__ static __forceinline__ void load(const char* p, int nv, float (&f)[8]) { layer_load8_32(p, nv, f); }
  __device__ static __forceinline__ void store(char* p, int nv, const float (&f)[8]) { layer_store8_32(p, nv, f); }
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

template <class Row>
hipError_t norm(NormArgs a, hipStream_t s) {
  const dim3 grid = layer_grid(a.M, kLongThreads, a.grid_x);
  return launch_kernel(layer_norm_long_kernel<Row>, grid, dim3(kLongThreads), s, a);
}

template <class Row>
hipError_t norm_grad(NormGradArgs a, hipStream_t s) {
  if (a.dgamma || a.dbeta) {
    if (a.M > 0) {
      const dim3 grid = layer_grid((a.parts * (((int64_t)a.N + 511) / 512) + 3) / 4, 256, a.grid_x);
      const hipError_t e = launch_kernel(layer_norm_grad_columns_kernel<Row>, grid, dim3(256), s, a);
      if (e != hipSuccess) return e;
    }
    const dim3 grid = layer_grid(((int64_t)a.N + 63) / 64, 64 * kSumWaves, a.grid_x, 2);
    const hipError_t e = launch_kernel(layer_norm_sum_kernel, grid, dim3(64 * kSumWaves), s, a);
    if (e != hipSuccess) return e;
  }
  if (!a.dX || a.M == 0) return hipSuccess;
  const dim3 grid = layer_grid(a.M, kLongThreads, a.grid_x);
  return launch_kernel(layer_norm_grad_long_kernel<Row>, grid, dim3(kLongThreads), s, a);
}

// Rows of one partial sum: at most 1024 parts.
int64_t norm_rows(int64_t m) { return (m + 1023) / 1024 > 0 ? (m + 1023) / 1024 : 1; }
int64_t norm_parts(int64_t m) { return (m + norm_rows(m) - 1) / norm_rows(m); }

int64_t norm_grad_bytes(int64_t M, int64_t N) {
  if (M < 0 || N < 0 || M > kMaxDim || N > kMaxDim) return 0;
  return norm_parts(M) * N * 8;
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
    a.rows = (int)norm_rows(M);
    a.parts = (int)norm_parts(M);
    hipStream_t s = static_cast<hipStream_t>(stream);
    set_path("norm_grad row by row");
    return launched(rowtype == ROW_F32   ? norm_grad<NormF32>(a, s)
                    : rowtype == ROW_F16 ? norm_grad<TagF16>(a, s)
                                         : norm_grad<TagBF16>(a, s));
  });
}

}  // extern "C"
