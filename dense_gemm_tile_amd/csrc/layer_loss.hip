// Cross entropy of an output layer: logits L = X W^T made in pieces of the
// vocabulary, and never all of them held.
//
//   lse = log sum exp L,  loss = lse - L[label]
//   G = dloss (exp(L - lse) - [v = label]),  dX = G W,  dW = G^T X
//
// A piece's logits are a product of gemm_linear in float32. Each row keeps the largest
// logit so far and the sum of exponentials relative to it; the gradient makes the
// logits again, turns a piece of them into G, and multiplies it from both sides.
#include "layer.h"
#include "layer_checks.h"

namespace dgt {

namespace {

// One piece of the vocabulary, columns [v0, v0 + n).
struct LossArgs {
  const float* L;       // logits of the piece, T x n, pitch ldl
  const int* labels;
  float* state;         // [3][T]: largest logit, sum, the label's logit
  float* loss;
  float* lse;           // null: not wanted
  int64_t ldl;
  int T, V, v0, n;
  int first, last;      // whether this is the first, the last piece
  unsigned grid_x;
};
struct LossGradArgs {
  const float* L;
  const int* labels;
  const float* lse;
  const float* dloss;
  void* G;              // T x n, pitch ldg
  int64_t ldl, ldg;
  int T, V, v0, n;
  unsigned grid_x;
};

// Two partial (largest, sum) as one. A side without logits has (-inf, 0).
__device__ __forceinline__ void loss_join(float& m, float& s, float om, float os) {
  const float top = om > m ? om : m;
  const float base = top == -__builtin_inff() ? 0.0f : top;
  s = s * __expf(m - base) + os * __expf(om - base);
  m = top;
}

// A workgroup a row of the piece.
__global__ void __launch_bounds__(256) layer_loss_rows_kernel(const LossArgs p) {
  __shared__ float part[8];
  const int64_t t = layer_block(p);
  if (t >= p.T) return;
  const float* l = p.L + t * p.ldl;
  float m = -__builtin_inff(), s = 0.0f;
  for (int c = threadIdx.x; c < p.n; c += 256) loss_join(m, s, l[c], 1.0f);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) loss_join(m, s, __shfl_xor(m, d, 64), __shfl_xor(s, d, 64));
  if ((threadIdx.x & 63) == 0) {
    part[threadIdx.x >> 6] = m;
    part[4 + (threadIdx.x >> 6)] = s;
  }
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < 4; ++w) loss_join(m, s, part[w], part[4 + w]);
  float at = 0.0f;
  const int label = p.labels[t];
  const bool has = (unsigned)label < (unsigned)p.V;
  if (!p.first) {
    loss_join(m, s, p.state[t], p.state[p.T + t]);
    at = p.state[2 * (int64_t)p.T + t];
  }
  if (has && label >= p.v0 && label - p.v0 < p.n) at = l[label - p.v0];
  if (p.last) {
    const float lse = m + logf(s);
    p.loss[t] = has ? lse - at : 0.0f;
    if (p.lse) p.lse[t] = lse;
  } else {
    p.state[t] = m;
    p.state[p.T + t] = s;
    p.state[2 * (int64_t)p.T + t] = at;
  }
}

// G of a piece.
template <class Tag>
__global__ void __launch_bounds__(256) layer_loss_grad_kernel(const LossGradArgs p) {
  const int64_t t = layer_block(p);
  if (t >= p.T) return;
  const int label = p.labels[t];
  const bool has = (unsigned)label < (unsigned)p.V;
  const float lse = has ? p.lse[t] : 0.0f, d = has ? p.dloss[t] : 0.0f;
  const float* l = p.L + t * p.ldl;
  char* g = static_cast<char*>(p.G) + t * p.ldg * 2;
  for (int64_t c = 8 * threadIdx.x; c < p.n; c += 8 * 256) {
    const int nv = p.n - c >= 8 ? 8 : (int)(p.n - c);
    float f[8];
    layer_load8_32(reinterpret_cast<const char*>(l + c), nv, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[e] = __expf(f[e] - lse) - (p.v0 + (int)c + e == label ? 1.0f : 0.0f);
      f[e] = has ? f[e] * d : 0.0f;
    }
    layer_store8_16<Tag>(g + c * 2, nv, f);
  }
}

// dX from its float32 sums.
template <class Tag>
__global__ void __launch_bounds__(256) layer_loss_round_kernel(const float* from, char* to, int64_t ld, int64_t n, int H) {
  for (int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x; at < n; at += (int64_t)gridDim.x * 256) {
    const int64_t t = at / H;
    reinterpret_cast<unsigned short*>(to)[t * ld + (at - t * H)] = layer_16(Tag{}, from[at]);
  }
}

// Columns of a piece: as many as 256 MiB of logits hold, whole tiles.
int64_t loss_piece(int64_t T, int64_t V) {
  int64_t n = ((int64_t{1} << 26) / (T > 0 ? T : 1)) / 256 * 256;
  if (n < 1024) n = 1024;
  return n < V ? n : (V + 7) / 8 * 8;
}
int64_t round16(int64_t b) { return (b + 15) / 16 * 16; }
int64_t loss_bytes(int64_t T, int64_t V, int64_t H) {
  if (T < 1 || V < 1 || H < 0 || T > kMaxDim || V > kMaxDim || H > kMaxDim) return 0;
  const int64_t p = loss_piece(T, V);
  return round16(T * 12) + T * p * 4;
}
int64_t loss_grad_bytes(int64_t T, int64_t V, int64_t H) {
  if (T < 1 || V < 1 || H < 0 || T > kMaxDim || V > kMaxDim || H > kMaxDim) return 0;
  const int64_t p = loss_piece(T, V);
  const unsigned __int128 b = (unsigned __int128)T * p * 6 + (unsigned __int128)T * H * 4 + 48;
  return b > (unsigned __int128)INT64_MAX ? 0 : (int64_t)b;
}

int check_loss(int64_t T, int64_t V, int64_t H, int dtype, const Mat& mx, const Mat& mw) {
  CHECK(check_dim("T", T));
  CHECK(check_dim("V", V));
  CHECK(check_dim("H", H));
  CHECK(check_dtype16(dtype));
  if (V < 1) return bad("%s=%lld: a vocabulary needs an entry", "V", V);
  CHECK(check_ld(mx));
  return check_ld(mw);
}

template <class Tag>
int run_grad(const LossGradArgs& g0, const DenseCall& logits, float* acc, int64_t piece, const Mat& mx, const Mat& mw,
             const Mat& mdx, const Mat& mdw, bool accumulate, int dtype, int dw_dtype, hipStream_t s) {
  const int64_t T = g0.T, V = g0.V, H = mx.cols;
  const bool single = piece >= V;
  // The plan of every piece before any of them runs, so that a call is refused as a whole.
  for (int launch = 0; launch < 2; ++launch)
    for (int64_t v0 = 0; v0 < V; v0 += piece) {
      const int64_t n = V - v0 < piece ? V - v0 : piece;
      const char* const w = static_cast<const char*>(mw.ptr) + v0 * mw.ld * 2;
      DenseCall c = logits;
      c.N = n;
      c.B = w;
      CHECK(run_dense(c, launch, s));
      if (launch) {
        LossGradArgs g = g0;
        g.v0 = (int)v0;
        g.n = (int)n;
        const dim3 grid = layer_grid(T, 256, g.grid_x);
        CHECK(launched(launch_kernel(layer_loss_grad_kernel<Tag>, grid, dim3(256), s, g)));
      }
      if (mdx.ptr && H > 0) {
        void* const to = single ? const_cast<void*>(mdx.ptr) : acc;
        const int64_t ld = single ? mdx.ld : H;
        const DenseCall dx{T, H, n, dtype, false, false, g0.G, g0.ldg, w, mw.ld, v0 ? acc : nullptr, H, to, ld,
                           single ? dtype : GEMM_DTYPE_F32};
        CHECK(run_dense(dx, launch, s));
      }
      if (mdw.ptr && H > 0) {
        char* const to = static_cast<char*>(const_cast<void*>(mdw.ptr)) + v0 * mdw.ld * mdw.elem;
        const DenseCall dw{n, H, T, dtype, true, false, g0.G, g0.ldg, mx.ptr, mx.ld, accumulate ? to : nullptr, mdw.ld, to,
                           mdw.ld, dw_dtype};
        CHECK(run_dense(dw, launch, s));
      }
    }
  if (!mdx.ptr || H == 0 || single) return GEMM_OK;
  const int64_t n = T * H, blocks = (n + 255) / 256;
  return launched(launch_kernel(layer_loss_round_kernel<Tag>, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), s,
                                (const float*)acc, static_cast<char*>(const_cast<void*>(mdx.ptr)), mdx.ld, n, (int)H));
}

}  // namespace
}  // namespace dgt

using namespace dgt;

extern "C" {

int64_t gemm_loss_workspace(int64_t T, int64_t V, int64_t H) { return loss_bytes(T, V, H); }

int gemm_loss(int64_t T, int64_t V, int64_t H, int dtype, const void* X, int64_t ldx, const void* W, int64_t ldw,
              const int32_t* labels, float* loss, float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
  return entry("loss", T, V, H, [&]() -> int {
    const Mat mx{"X", X, T, H, ldx, 2}, mw{"W", W, V, H, ldw, 2};
    CHECK(check_loss(T, V, H, dtype, mx, mw));
    if (T == 0) {
      set_path("noop: empty output");
      return GEMM_OK;
    }
    const int64_t need = loss_bytes(T, V, H);
    const Mat ml{"labels", labels, 1, T, T, 4}, mo{"loss", loss, 1, T, T, 4}, me{"lse", lse, 1, T, T, 4};
    const Mat ms{"workspace", workspace, 1, need, need, 1};
    if (H > 0) {
      CHECK(check_ptr(mx));
      CHECK(check_ptr(mw));
    }
    CHECK(check_ptr(ml));
    CHECK(check_ptr(mo));
    if (lse) CHECK(check_ptr(me));
    CHECK(check_workspace(workspace, workspace_bytes, need));
    for (const Mat* w : {&mo, &me, &ms})
      for (const Mat* r : {&mx, &mw, &ml}) CHECK(check_apart(*w, *r));
    CHECK(check_apart(me, mo));
    CHECK(check_apart(ms, mo));
    CHECK(check_apart(ms, me));
    hipStream_t s = static_cast<hipStream_t>(stream);
    const int64_t piece = loss_piece(T, V);
    LossArgs a{};
    a.state = static_cast<float*>(workspace);
    float* const l = reinterpret_cast<float*>(static_cast<char*>(workspace) + round16(T * 12));
    a.L = l;
    a.labels = labels;
    a.loss = loss;
    a.lse = lse;
    a.ldl = piece;
    a.T = (int)T;
    a.V = (int)V;
    for (int launch = 0; launch < 2; ++launch)
      for (int64_t v0 = 0; v0 < V; v0 += piece) {
        const int64_t n = V - v0 < piece ? V - v0 : piece;
        const DenseCall c{T, n, H, dtype, false, true, X, ldx, static_cast<const char*>(W) + v0 * ldw * 2, ldw,
                          nullptr, 0, l, piece, GEMM_DTYPE_F32};
        CHECK(run_dense(c, launch, s));
        if (!launch) continue;
        a.v0 = (int)v0;
        a.n = (int)n;
        a.first = v0 == 0;
        a.last = v0 + piece >= V;
        const dim3 grid = layer_grid(T, 256, a.grid_x);
        CHECK(launched(launch_kernel(layer_loss_rows_kernel, grid, dim3(256), s, a)));
      }
    set_path("loss in pieces of " + std::to_string(piece));
    return GEMM_OK;
  });
}

int64_t gemm_loss_grad_workspace(int64_t T, int64_t V, int64_t H) { return loss_grad_bytes(T, V, H); }

int gemm_loss_grad(int64_t T, int64_t V, int64_t H, int dtype, const void* X, int64_t ldx, const void* W, int64_t ldw,
                   const int32_t* labels, const float* lse, const float* dloss, void* dX, int64_t lddx, void* dW,
                   int64_t lddw, int dw_dtype, int accumulate, void* workspace, int64_t workspace_bytes, void* stream) {
  return entry("loss_grad", T, V, H, [&]() -> int {
    const Mat mx{"X", X, T, H, ldx, 2}, mw{"W", W, V, H, ldw, 2};
    CHECK(check_loss(T, V, H, dtype, mx, mw));
    CHECK(check_out_dtype(dtype, dw_dtype));
    const Mat mdx{"dX", dX, T, H, lddx, 2}, mdw{"dW", dW, V, H, lddw, dw_dtype == GEMM_DTYPE_F32 ? 4 : 2};
    if (dX) CHECK(check_ld(mdx));
    if (dW) CHECK(check_ld(mdw));
    if (H == 0 || (!dX && !dW) || (T == 0 && (!dW || accumulate))) {
      set_path("noop: empty output");
      return GEMM_OK;
    }
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (dX && T > 0) CHECK(check_ptr(mdx));
    if (dW) CHECK(check_ptr(mdw));
    if (T == 0) {  // no rows: zeros
      const DenseCall c{V, H, 0, dtype, true, false, nullptr, V, nullptr, H, nullptr, 0, dW, lddw, dw_dtype};
      return run_dense(c, true, s);
    }
    const int64_t need = loss_grad_bytes(T, V, H);
    if (!need) return fail(GEMM_ERR_UNSUPPORTED, "the workspace would be too large");
    const Mat ml{"labels", labels, 1, T, T, 4}, me{"lse", lse, 1, T, T, 4}, md{"dloss", dloss, 1, T, T, 4};
    const Mat ms{"workspace", workspace, 1, need, need, 1};
    for (const Mat* m : {&mx, &mw, &ml, &me, &md}) CHECK(check_ptr(*m));
    CHECK(check_workspace(workspace, workspace_bytes, need));
    for (const Mat* w : {&mdx, &mdw, &ms})
      for (const Mat* r : {&mx, &mw, &ml, &me, &md}) CHECK(check_apart(*w, *r));
    CHECK(check_apart(mdw, mdx));
    CHECK(check_apart(ms, mdx));
    CHECK(check_apart(ms, mdw));
    const int64_t piece = loss_piece(T, V);
    char* const ws = static_cast<char*>(workspace);
    float* const l = reinterpret_cast<float*>(ws);
    void* const g = ws + round16(T * piece * 4);
    float* const acc = reinterpret_cast<float*>(static_cast<char*>(g) + round16(T * piece * 2));
    LossGradArgs a{};
    a.L = l;
    a.labels = labels;
    a.lse = lse;
    a.dloss = dloss;
    a.G = g;
    a.ldl = a.ldg = piece;
    a.T = (int)T;
    a.V = (int)V;
    const DenseCall c{T, 0, H, dtype, false, true, X, ldx, nullptr, ldw, nullptr, 0, l, piece, GEMM_DTYPE_F32};
    CHECK(dtype == GEMM_DTYPE_F16
              ? run_grad<TagF16>(a, c, acc, piece, mx, mw, mdx, mdw, accumulate != 0, dtype, dw_dtype, s)
              : run_grad<TagBF16>(a, c, acc, piece, mx, mw, mdx, mdw, accumulate != 0, dtype, dw_dtype, s));
    set_path("loss_grad in pieces of " + std::to_string(piece));
    return GEMM_OK;
  });
}

}  // extern "C"
