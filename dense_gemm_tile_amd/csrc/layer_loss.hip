// Cross entropy of an output layer: logits L = X W^T, of which pieces of the vocabulary are held
// at a time.
//
//   lse = log sum exp L,  loss = lse - L[label]
//   G = dloss (exp(L - lse) - [v = label]),  dX = G W,  dW = G^T X
//
// Forward: parts of the vocabulary leave their largest logit and their sum of
// exponentials for each token, which a second kernel joins. Gradient: a piece's logits
// are made again and turned into G, stored as G^T (n x T8: a vocabulary entry's row,
// tokens in whole pieces of 8, zeros past T), whose two products follow:
//   dW   G^T X, each piece its own rows
//   dX   G W, a sum over the vocabulary: both operands lie along it, so it can be cut into S
//        parts that fill the CUs where T x H has few tiles; parts and pieces are added
//        in float32
// X is copied to T8 rows where T is not a multiple of 8.
//
// The matrix cores take G in 16 bits. It is held relative to the largest |dloss| (scale:
// 2^-15 of it), which its products multiply back in float32: f16 has room for probabilities
// down to 2^-39 beside 1 whatever dloss is, and where all tokens weigh the same, as in a mean,
// dloss is not rounded at all, nor, nearly, is the label's element of a token far from its
// label, the row's largest.
//
// The logits come from layer_loss_pp256.hip, which turns them into parts or G in
// registers. Fewer tokens, and operands not in whole 16-byte pieces, take a product of
// gemm_linear in float32 and a kernel over its rows instead. The workspace has room for those
// float32 logits whatever a call takes, since its size is asked for before pitches and
// addresses are known.
#include "layer_loss.h"

#include "layer_checks.h"

namespace dgt {

namespace {

constexpr int kLossStep = 4096;  // logits of a row that a workgroup holds at a time

// Sub-piece of float32 logits, T x n: columns [v0, v0 + n) of the vocabulary.
struct LossRowsArgs {
  const float* L;
  const int* labels;
  float2* parts;        // of this sub-piece: [T]; null: it is the only one
  float* target;
  float* loss;          // (the only one)
  float* lse;           // null: not wanted
  int64_t ldl;
  int T, V, v0, n;
  unsigned grid_x;
};
struct LossJoinArgs {
  const float2* parts;  // [Q][T]
  const float* target;
  const int* labels;
  float* loss;
  float* lse;           // null: not wanted
  int T, V, Q;
  unsigned grid_x;
};
struct LossGradArgs {
  const float* L;
  const int* labels;
  const float* lse;
  const float* dloss;
  const float* scale;
  void* G;              // n x T8
  int64_t ldl;
  int T, T8, V, v0, n;
  unsigned grid_x;
};

// Two partial (largest, sum) as one. A side without logits has (-inf, 0).
__device__ __forceinline__ float2 loss_join(float2 a, float2 b) {
  const float m = __builtin_fmaxf(a.x, b.x), base = m == -__builtin_inff() ? 0.0f : m;
  return float2{m, a.y * loss_exp(a.x - base) + b.y * loss_exp(b.x - base)};
}

// A workgroup takes a row. (Rows cut over workgroups and joined by a second kernel: 61 rows of
// 32001 9 us for both, 6 so.)
constexpr int kRowThreads = 1024;
__global__ void __launch_bounds__(kRowThreads) layer_loss_rows_kernel(const LossRowsArgs p) {
  __shared__ float2 part[kRowThreads / 64];
  const int64_t t = layer_block(p);
  if (t >= p.T) return;
  const float* l = p.L + t * p.ldl;
  constexpr int PER = 8 * kLossStep / (4 * kRowThreads);  // fours of eight steps, in flight together
  float2 a{-__builtin_inff(), 0.0f};
  for (int64_t c0 = 0; c0 < p.n; c0 += 8 * kLossStep) {
    f32x4 f[PER];
    float m = a.x;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int64_t c = c0 + kLossStep * i + 4 * threadIdx.x;
      if (c + 4 <= p.n) {
        f[i] = *reinterpret_cast<const f32x4*>(l + c);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) f[i][e] = c + e < p.n ? l[c + e] : -__builtin_inff();
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) m = __builtin_fmaxf(m, f[i][e]);
    const float base = m == -__builtin_inff() ? 0.0f : m;
    a.y *= loss_exp(a.x - base);
    a.x = m;
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) a.y += loss_exp(f[i][e] - base);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) a = loss_join(a, float2{__shfl_xor(a.x, d, 64), __shfl_xor(a.y, d, 64)});
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = a;
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < kRowThreads / 64; ++w) a = loss_join(a, part[w]);
  const int label = p.labels[t];
  const bool has = (unsigned)label < (unsigned)p.V, here = has && label >= p.v0 && label - p.v0 < p.n;
  if (p.parts) {
    p.parts[t] = a;
    if (here) p.target[t] = l[label - p.v0];
  } else {
    const float lse = a.x + logf(a.y);
    p.loss[t] = has ? lse - l[label] : 0.0f;
    if (p.lse) p.lse[t] = lse;
  }
}

// The parts of 64 tokens: every kJoinWaves-th for each wave, joined in wave order.
constexpr int kJoinWaves = 16;
__global__ void __launch_bounds__(64 * kJoinWaves) layer_loss_join_kernel(const LossJoinArgs p) {
  __shared__ float2 part[kJoinWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t t = (int64_t)layer_block(p) * 64 + lane;
  float2 a{-__builtin_inff(), 0.0f};
  if (t < p.T) {
    constexpr int AHEAD = 8;  // parts in flight together
    for (int64_t q = w; q < p.Q; q += AHEAD * kJoinWaves) {
      float2 v[AHEAD];
#pragma unroll
      for (int u = 0; u < AHEAD; ++u)
        v[u] = q + u * kJoinWaves < p.Q ? p.parts[(q + u * kJoinWaves) * p.T + t] : float2{-__builtin_inff(), 0.0f};
#pragma unroll
      for (int u = 0; u < AHEAD; ++u) a = loss_join(a, v[u]);
    }
  }
  part[w][lane] = a;
  __syncthreads();
  if (w || t >= p.T) return;
  for (int u = 1; u < kJoinWaves; ++u) a = loss_join(a, part[u][lane]);
  const float lse = a.x + logf(a.y);
  const bool has = (unsigned)p.labels[t] < (unsigned)p.V;
  p.loss[t] = has ? lse - p.target[t] : 0.0f;
  if (p.lse) p.lse[t] = lse;
}

// G^T of 64 tokens and 64 entries, through LDS.
template <class Tag>
__global__ void __launch_bounds__(256) layer_loss_grad_kernel(const LossGradArgs p) {
  __shared__ unsigned short x[64][72];  // [entry][token]; rows 16-byte aligned, banks apart
  const unsigned across = (unsigned)(p.T8 + 63) / 64, id = layer_block(p);
  const int64_t r = id / across;
  const int t0 = (int)(id - (unsigned)r * across) * 64, e0 = (int)(r * 64);
  if (r * 64 >= p.n) return;
  const int lane = threadIdx.x & 63;
  for (int i = threadIdx.x >> 6; i < 64; i += 4) {  // a wave a token
    const int t = t0 + i, c = e0 + lane, label = t < p.T ? p.labels[t] : -1;
    float g = 0.0f;
    if ((unsigned)label < (unsigned)p.V && c < p.n)
      g = p.dloss[t] / *p.scale * (loss_exp(p.L[t * p.ldl + c] - p.lse[t]) - (p.v0 + c == label ? 1.0f : 0.0f));
    x[lane][i] = layer_16(Tag{}, g);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * 8; i += 256) {
    const int e = i >> 3, t = 8 * (i & 7);
    if (e0 + e < p.n && t0 + t < p.T8)
      *reinterpret_cast<u32x4*>(static_cast<unsigned short*>(p.G) + (int64_t)(e0 + e) * p.T8 + t0 + t) =
          *reinterpret_cast<const u32x4*>(&x[e][t]);
  }
}

// X with T8 rows, zeros from row T on.
struct LossPadArgs {
  const unsigned short* X;
  unsigned short* to;
  int64_t ldx, n, live;  // elements: all of them, and those of X
  int H;
};
__global__ void __launch_bounds__(256) layer_loss_pad_kernel(const LossPadArgs p) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < p.n; i += (int64_t)gridDim.x * 256) {
    const int64_t t = i / p.H;
    p.to[i] = i < p.live ? p.X[t * p.ldx + (i - t * p.H)] : (unsigned short)0;
  }
}
// What a gradient's other kernels read: the scale of G, 2^-15 of the largest finite |dloss| of a
// token that has a label, and offsets that cut n rows into S parts, for the pieces of n and for
// the last one.
struct LossStartArgs {
  const int* labels;
  const float* dloss;
  float* scale;
  int* offsets;
  int T, V, S, n, last;
};
__global__ void __launch_bounds__(1024) layer_loss_start_kernel(const LossStartArgs p) {
  __shared__ float part[16];
  for (int i = threadIdx.x; i <= p.S; i += 1024) {
    p.offsets[i] = (int)((int64_t)p.n * i / p.S);
    p.offsets[p.S + 1 + i] = (int)((int64_t)p.last * i / p.S);
  }
  float m = 0.0f;
#pragma unroll 8
  for (int64_t t = threadIdx.x; t < p.T; t += 1024) {
    const float d = __builtin_fabsf(p.dloss[t]);
    if ((unsigned)p.labels[t] < (unsigned)p.V && d < __builtin_inff()) m = __builtin_fmaxf(m, d);
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) m = __builtin_fmaxf(m, __shfl_xor(m, d, 64));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < 16; ++w) m = __builtin_fmaxf(m, part[w]);
  m *= 0x1p-15f;
  *p.scale = m > 0.0f ? m : 1.0f;
}
// dX from S float32 parts of T8 x H.
struct LossRoundArgs {
  const float* from;
  const float* scale;
  unsigned short* to;
  int64_t ld, n, stride;
  int H, S;
};
template <class Tag>
__global__ void __launch_bounds__(256) layer_loss_round_kernel(const LossRoundArgs p) {
  const float scale = *p.scale;
  for (int64_t i = 4 * ((int64_t)blockIdx.x * 256 + threadIdx.x); i < p.n; i += 4 * (int64_t)gridDim.x * 256) {
    f32x4 s = *reinterpret_cast<const f32x4*>(p.from + i);  // (parts are whole fours: T8 is a multiple of 8)
    for (int u = 1; u < p.S; ++u) {
      const f32x4 o = *reinterpret_cast<const f32x4*>(p.from + u * p.stride + i);
      for (int e = 0; e < 4; ++e) s[e] += o[e];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t t = (i + e) / p.H;
      if (i + e < p.n) p.to[t * p.ld + (i + e - t * p.H)] = layer_16(Tag{}, s[e] * scale);
    }
  }
}

// ------------------------------------------------------------------ the plan --
int64_t round16(int64_t b) { return (b + 15) / 16 * 16; }

// Sizes of a call, and where its buffers lie in the workspace (bytes).
struct LossPlan {
  int64_t T8, piece, sub;  // G's rows at a time, float32 logits' columns at a time
  int64_t Q;               // parts, at most
  int S;                   // parts of dX's sum
  bool direct;             // dX needs no float32 sums
  int64_t parts, target, logits, forward;      // forward: all bytes of gemm_loss
  int64_t glogits, g, xpad, sums, offsets, scale, grad;  // grad: all bytes of gemm_loss_grad
};
// False where the bytes pass 63 bits.
bool loss_plan(int64_t T, int64_t V, int64_t H, LossPlan& q) {
  if (T < 1 || V < 1 || H < 0 || T > kMaxDim || V > kMaxDim || H > kMaxDim) return false;
  auto columns = [&](int64_t elements) {  // of T tokens each, whole steps, at least one
    int64_t n = elements / T / kLossStep * kLossStep;
    if (n < kLossStep) n = kLossStep;
    return n < V ? n : (V + 7) / 8 * 8;
  };
  q.T8 = (T + 7) / 8 * 8;
  q.piece = columns(int64_t{1} << 28);  // 512 MiB of G
  q.sub = columns(int64_t{1} << 25);    // 128 MiB of logits
  q.Q = (V + 255) / 256;
  const int64_t tiles = ((q.T8 + 255) / 256) * ((H + 255) / 256);
  const int64_t rows = q.piece < V ? q.piece : V;
  q.S = 1;
  if (tiles > 0 && tiles <= 128) {
    int64_t s = 256 / tiles;
    if (s > rows / 1024) s = rows / 1024;
    q.S = s > 1 ? (int)s : 1;
  }
  q.direct = q.S == 1 && q.piece >= V && q.T8 == T;
  unsigned __int128 at = 0;
  auto place = [&](int64_t& where, unsigned __int128 bytes) {
    where = (int64_t)at;
    at += (bytes + 15) / 16 * 16;
  };
  const unsigned __int128 max = INT64_MAX;
  place(q.parts, (unsigned __int128)q.Q * T * 8);
  place(q.target, (unsigned __int128)T * 4);
  place(q.logits, (unsigned __int128)T * q.sub * 4);
  if (at > max) return false;
  q.forward = (int64_t)at;
  at = 0;
  place(q.glogits, (unsigned __int128)T * q.sub * 4);
  place(q.g, (unsigned __int128)q.piece * q.T8 * 2);
  place(q.xpad, q.T8 == T ? 0 : (unsigned __int128)q.T8 * H * 2);
  place(q.sums, q.direct ? 0 : (unsigned __int128)q.S * q.T8 * H * 4);
  place(q.offsets, (unsigned __int128)2 * (q.S + 1) * 4);
  place(q.scale, 4);
  if (at > max) return false;
  q.grad = (int64_t)at;
  return true;
}

// Whether the logits are made on 256x256 tiles: operands in whole 16-byte pieces, and enough
// tokens for half of a tile's columns or more than one tile.
bool loss_tiles(const Mat& x, const Mat& w, int64_t n) {
  auto whole = [](const Mat& m) {
    return (uintptr_t)m.ptr % 16 == 0 && m.ld % 8 == 0 && m.ld < (int64_t{1} << 31) / (2 * 257) - 4096;
  };
  const int64_t tiles = ((x.rows + 255) / 256) * ((n + 255) / 256);
  return x.cols > 0 && x.cols % 8 == 0 && whole(x) && whole(w) && x.rows > 64 && tiles < (1 << 22);
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

// f(v0, n) for pieces of V columns; the first status that is not GEMM_OK.
template <class F>
int loss_pieces(int64_t V, int64_t piece, F f) {
  for (int64_t v0 = 0; v0 < V; v0 += piece) CHECK(f(v0, V - v0 < piece ? V - v0 : piece));
  return GEMM_OK;
}
const char* loss_row(const Mat& m, int64_t row) { return static_cast<const char*>(m.ptr) + row * m.ld * m.elem; }

// The float32 logits of columns [v0, v0 + n).
DenseCall loss_logits(const Mat& mx, const Mat& mw, int dtype, int64_t v0, int64_t n, void* to, int64_t ld) {
  return {mx.rows, n, mx.cols, dtype, false, true, mx.ptr, mx.ld, loss_row(mw, v0), mw.ld, nullptr, 0, to, ld, GEMM_DTYPE_F32,
          nullptr};
}

// Both run through a call twice: without launches, so that a refusal comes before any work, and with.
int run_loss(const LossPlan& q, const Mat& mx, const Mat& mw, int dtype, const int32_t* labels, float* loss, float* lse,
             char* ws, bool launch, hipStream_t s) {
  const int64_t T = mx.rows, V = mw.rows;
  float2* const parts = reinterpret_cast<float2*>(ws + q.parts);
  float* const target = reinterpret_cast<float*>(ws + q.target);
  const bool tiles = loss_tiles(mx, mw, V);
  int64_t Q = q.Q;
  if (tiles) {
    LossTileArgs a{};
    a.W = mw.ptr;
    a.X = mx.ptr;
    a.ldw = mw.ld;
    a.ldx = mx.ld;
    a.n = (int)V;
    a.T = (int)T;
    a.H = (int)mx.cols;
    a.labels = labels;
    a.V = (int)V;
    a.parts = parts;
    a.target = target;
    if (launch) CHECK(launched(launch_loss_tiles(dtype, false, a, s)));
  } else {
    Q = 0;
    CHECK(loss_pieces(V, q.sub, [&](int64_t v0, int64_t n) -> int {
      float* const l = reinterpret_cast<float*>(ws + q.logits);
      CHECK(run_dense(loss_logits(mx, mw, dtype, v0, n, l, q.sub), launch, s));
      LossRowsArgs a{};
      a.L = l;
      a.labels = labels;
      a.parts = n < V ? parts + Q * T : nullptr;
      a.target = target;
      a.loss = loss;
      a.lse = lse;
      a.ldl = q.sub;
      a.T = (int)T;
      a.V = (int)V;
      a.v0 = (int)v0;
      a.n = (int)n;
      ++Q;
      if (!launch) return GEMM_OK;
      const dim3 grid = layer_grid(T, kRowThreads, a.grid_x);
      return launched(launch_kernel(layer_loss_rows_kernel, grid, dim3(kRowThreads), s, a));
    }));
  }
  if (!launch) return GEMM_OK;
  set_path(tiles ? "loss on 256x256 tiles" : "loss in pieces of " + std::to_string(q.sub));
  if (!tiles && Q == 1) return GEMM_OK;
  LossJoinArgs j{};
  j.parts = parts;
  j.target = target;
  j.labels = labels;
  j.loss = loss;
  j.lse = lse;
  j.T = (int)T;
  j.V = (int)V;
  j.Q = (int)Q;
  const dim3 grid = layer_grid((T + 63) / 64, 64 * kJoinWaves, j.grid_x);
  return launched(launch_kernel(layer_loss_join_kernel, grid, dim3(64 * kJoinWaves), s, j));
}

template <class Tag>
int run_grad(const LossPlan& q, const Mat& mx, const Mat& mw, const Mat& mdx, const Mat& mdw, int dtype, int dw_dtype,
             bool accumulate, const int32_t* labels, const float* lse, const float* dloss, char* ws, bool launch, hipStream_t s) {
  const int64_t T = mx.rows, V = mw.rows, H = mx.cols;
  const unsigned most = 4096;  // workgroups of the kernels that walk
  auto blocks = [&](int64_t n) { return dim3((unsigned)(n < most ? (n ? n : 1) : most)); };
  const void* x = mx.ptr;
  int64_t ldx = mx.ld;
  if (q.T8 != T && mdw.ptr) {
    const LossPadArgs a{static_cast<const unsigned short*>(mx.ptr), reinterpret_cast<unsigned short*>(ws + q.xpad), mx.ld,
                        q.T8 * H, T * H, (int)H};
    x = a.to;
    ldx = H;
    if (launch) CHECK(launched(launch_kernel(layer_loss_pad_kernel, blocks((a.n + 255) / 256), dim3(256), s, a)));
  }
  int* const offsets = reinterpret_cast<int*>(ws + q.offsets);
  float* const scale = reinterpret_cast<float*>(ws + q.scale);
  if (launch) {
    const int64_t last = V - (V - 1) / q.piece * q.piece;
    const LossStartArgs a{labels, dloss, scale, offsets, (int)T, (int)V, q.S, (int)(q.piece < V ? q.piece : V), (int)last};
    CHECK(launched(launch_kernel(layer_loss_start_kernel, dim3(1), dim3(1024), s, a)));
  }
  void* const G = ws + q.g;
  const bool tiles = loss_tiles(mx, mw, q.piece);
  CHECK(loss_pieces(V, q.piece, [&](int64_t v0, int64_t n) -> int {
    if (tiles) {
      LossTileArgs a{};
      a.W = loss_row(mw, v0);
      a.X = mx.ptr;
      a.ldw = mw.ld;
      a.ldx = mx.ld;
      a.n = (int)n;
      a.T = (int)T;
      a.H = (int)H;
      a.v0 = (int)v0;
      a.labels = labels;
      a.V = (int)V;
      a.lse = lse;
      a.dloss = dloss;
      a.scale = scale;
      a.G = G;
      a.T8 = (int)q.T8;
      if (launch) CHECK(launched(launch_loss_tiles(dtype, true, a, s)));
    } else {
      CHECK(loss_pieces(n, q.sub, [&](int64_t c0, int64_t m) -> int {
        float* const l = reinterpret_cast<float*>(ws + q.glogits);
        CHECK(run_dense(loss_logits(mx, mw, dtype, v0 + c0, m, l, q.sub), launch, s));
        LossGradArgs a{};
        a.L = l;
        a.labels = labels;
        a.lse = lse;
        a.dloss = dloss;
        a.scale = scale;
        a.G = static_cast<unsigned short*>(G) + c0 * q.T8;
        a.ldl = q.sub;
        a.T = (int)T;
        a.T8 = (int)q.T8;
        a.V = (int)V;
        a.v0 = (int)(v0 + c0);
        a.n = (int)m;
        const int64_t squares = ((m + 63) / 64) * ((q.T8 + 63) / 64);
        if (squares > 0x7ffffff0) return fail(GEMM_ERR_UNSUPPORTED, "too many pieces of rows for one launch");
        if (!launch) return GEMM_OK;
        const dim3 grid = layer_grid(squares, 256, a.grid_x);
        return launched(launch_kernel(layer_loss_grad_kernel<Tag>, grid, dim3(256), s, a));
      }));
    }
    if (mdx.ptr) {
      const SumsCall c{q.S, n, q.T8, H, dtype, offsets + (v0 + q.piece >= V ? q.S + 1 : 0), G, q.T8, loss_row(mw, v0), mw.ld,
                       q.direct ? const_cast<void*>(mdx.ptr) : ws + q.sums, q.direct ? mdx.ld : H, q.T8 * H,
                       q.direct ? dtype : GEMM_DTYPE_F32, v0 > 0,
                       q.direct ? scale : nullptr};
      CHECK(run_sums(c, launch, s));
    }
    if (mdw.ptr) {
      void* const to = const_cast<char*>(loss_row(mdw, v0));
      const DenseCall c{n, H, q.T8, dtype, false, false, G, q.T8, x, ldx, accumulate ? to : nullptr, mdw.ld, to, mdw.ld, dw_dtype,
                        scale};
      CHECK(run_dense(c, launch, s));
    }
    return GEMM_OK;
  }));
  if (!launch) return GEMM_OK;
  if (mdx.ptr && !q.direct) {
    const LossRoundArgs a{reinterpret_cast<const float*>(ws + q.sums), scale, static_cast<unsigned short*>(const_cast<void*>(mdx.ptr)),
                          mdx.ld, T * H, q.T8 * H, (int)H, q.S};
    CHECK(launched(launch_kernel(layer_loss_round_kernel<Tag>, blocks((a.n + 1023) / 1024), dim3(256), s, a)));
  }
  set_path(std::string(tiles ? "loss_grad on 256x256 tiles" : "loss_grad from float32 logits") + " in pieces of " +
           std::to_string(q.piece));
  return GEMM_OK;
}

}  // namespace
}  // namespace dgt

using namespace dgt;

extern "C" {

int64_t gemm_loss_workspace(int64_t T, int64_t V, int64_t H) {
  LossPlan q{};
  return loss_plan(T, V, H, q) ? q.forward : 0;
}

int gemm_loss(int64_t T, int64_t V, int64_t H, int dtype, const void* X, int64_t ldx, const void* W, int64_t ldw,
              const int32_t* labels, float* loss, float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
  return entry("loss", T, V, H, [&]() -> int {
    const Mat mx{"X", X, T, H, ldx, 2}, mw{"W", W, V, H, ldw, 2};
    CHECK(check_loss(T, V, H, dtype, mx, mw));
    if (T == 0) {
      set_path("noop: empty output");
      return GEMM_OK;
    }
    LossPlan q{};
    if (!loss_plan(T, V, H, q)) return fail(GEMM_ERR_UNSUPPORTED, "the workspace would be too large");
    const Mat ml{"labels", labels, 1, T, T, 4}, mo{"loss", loss, 1, T, T, 4}, me{"lse", lse, 1, T, T, 4};
    const Mat ms{"workspace", workspace, 1, q.forward, q.forward, 1};
    if (H > 0) {
      CHECK(check_ptr(mx));
      CHECK(check_ptr(mw));
    }
    CHECK(check_ptr(ml));
    CHECK(check_ptr(mo));
    if (lse) CHECK(check_ptr(me));
    CHECK(check_workspace(workspace, workspace_bytes, q.forward));
    for (const Mat* w : {&mo, &me, &ms})
      for (const Mat* r : {&mx, &mw, &ml}) CHECK(check_apart(*w, *r));
    CHECK(check_apart(me, mo));
    CHECK(check_apart(ms, mo));
    CHECK(check_apart(ms, me));
    for (int launch = 0; launch < 2; ++launch)
      CHECK(run_loss(q, mx, mw, dtype, labels, loss, lse, static_cast<char*>(workspace), launch, static_cast<hipStream_t>(stream)));
    return GEMM_OK;
  });
}

int64_t gemm_loss_grad_workspace(int64_t T, int64_t V, int64_t H) {
  LossPlan q{};
  return loss_plan(T, V, H, q) ? q.grad : 0;
}

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
      const DenseCall c{V, H, 0, dtype, true, false, nullptr, V, nullptr, H, nullptr, 0, dW, lddw, dw_dtype,
                        nullptr};
      return run_dense(c, true, s);
    }
    LossPlan q{};
    if (!loss_plan(T, V, H, q)) return fail(GEMM_ERR_UNSUPPORTED, "the workspace would be too large");
    const Mat ml{"labels", labels, 1, T, T, 4}, me{"lse", lse, 1, T, T, 4}, md{"dloss", dloss, 1, T, T, 4};
    const Mat ms{"workspace", workspace, 1, q.grad, q.grad, 1};
    for (const Mat* m : {&mx, &mw, &ml, &me, &md}) CHECK(check_ptr(*m));
    CHECK(check_workspace(workspace, workspace_bytes, q.grad));
    for (const Mat* w : {&mdx, &mdw, &ms})
      for (const Mat* r : {&mx, &mw, &ml, &me, &md}) CHECK(check_apart(*w, *r));
    CHECK(check_apart(mdw, mdx));
    CHECK(check_apart(ms, mdx));
    CHECK(check_apart(ms, mdw));
    for (int launch = 0; launch < 2; ++launch) {
      char* const ws = static_cast<char*>(workspace);
      CHECK(dtype == GEMM_DTYPE_F16 ? run_grad<TagF16>(q, mx, mw, mdx, mdw, dtype, dw_dtype, accumulate != 0, labels, lse, dloss,
                                                       ws, launch, s)
                                    : run_grad<TagBF16>(q, mx, mw, mdx, mdw, dtype, dw_dtype, accumulate != 0, labels, lse, dloss,
                                                        ws, launch, s));
    }
    return GEMM_OK;
  });
}

}  // extern "C"
