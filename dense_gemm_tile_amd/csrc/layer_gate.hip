// The gate: which experts a token goes to, with what weights, and the gradient of
// the logits from the weights'.
//
//   s = softmax(L) or 1 / (1 + exp(-L)),  key = s + bias
//   groups by the sum of their group_top largest keys, experts of the best groups by
//   key;  w = scale s[id]  (renorm: / sum of the chosen s)
//
// A wave takes a token; lane l holds experts l, l + 64, ... Keys are compared as
// integers that order as the numbers do, with a place for NaN (1) and for masked
// experts (0) below them.
#include "layer.h"
#include "layer_checks.h"

namespace dgt {

namespace {

constexpr int kGateTop = 64;  // a choice a lane

struct GateArgs {
  const void* L;
  const float* bias;    // null: none
  int* ids;
  float* weights;
  int64_t ldl;
  int T, E, top, score;
  int groups, top_groups, group_top, renorm;
  float scale;
  unsigned grid_x;
};
struct GateGradArgs {
  const void* L;
  const int* ids;
  const float* dweights;
  void* dL;
  int64_t ldl, lddl;
  int T, E, top, score, renorm;
  float scale;
  unsigned grid_x;
};

struct GateF32 {};
__device__ __forceinline__ float gate_load(GateF32, const void* p, int64_t at) { return static_cast<const float*>(p)[at]; }
template <class Tag>
__device__ __forceinline__ float gate_load(Tag t, const void* p, int64_t at) {
  return layer_f32(t, static_cast<const unsigned short*>(p)[at]);
}
__device__ __forceinline__ void gate_store(GateF32, void* p, int64_t at, float v) { static_cast<float*>(p)[at] = v; }
template <class Tag>
__device__ __forceinline__ void gate_store(Tag t, void* p, int64_t at, float v) {
  static_cast<unsigned short*>(p)[at] = layer_16(t, v);
}

template <class T>
__device__ __forceinline__ T gate_wave_sum(T v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}
template <class T>
__device__ __forceinline__ T gate_wave_max(T v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const T o = __shfl_xor(v, d, 64);
    v = o > v ? o : v;
  }
  return v;
}

constexpr uint64_t kGateMasked = 0, kGateNan = 1;
__device__ __forceinline__ uint64_t gate_order(double v) {
  if (v != v) return kGateNan;
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return u >> 63 ? ~u : u | ((uint64_t)1 << 63);
}

// The largest of the wave's keys, and of equal ones the first; every lane gets both.
struct GateBest {
  uint64_t key;
  int at;
};
__device__ __forceinline__ GateBest gate_best(GateBest b) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t k = __shfl_xor((unsigned long long)b.key, d, 64);
    const int at = __shfl_xor(b.at, d, 64);
    if (k > b.key || (k == b.key && at < b.at)) b = {k, at};
  }
  return b;
}

template <class Row, int PER, bool GROUPS>
__global__ void __launch_bounds__(256) layer_gate_kernel(const GateArgs p) {
  __shared__ uint64_t lds[GROUPS ? 4 * 2 * 64 * PER : 1];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t t = (int64_t)layer_block(p) * 4 + w;
  if (t >= p.T) return;
  double s[PER];
  uint64_t key[PER];
  // Scores.
  double top = -__builtin_inf();
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 64 + lane;
    s[i] = e < p.E ? (double)gate_load(Row{}, p.L, t * p.ldl + e) : -__builtin_inf();
    key[i] = s[i] == -__builtin_inf() ? kGateMasked : kGateNan;  // (any other for now)
    top = s[i] > top ? s[i] : top;
  }
  if (p.score == GEMM_SCORE_SOFTMAX) {
    top = gate_wave_max(top);
    double sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      s[i] = key[i] == kGateMasked ? 0.0 : exp(s[i] - top);
      sum += s[i];
    }
    sum = gate_wave_sum(sum);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] != kGateMasked) s[i] /= sum;
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = key[i] == kGateMasked ? 0.0 : 1.0 / (1.0 + exp(-s[i]));
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 64 + lane;
    const double bias = p.bias && e < p.E ? (double)p.bias[e] : 0.0;
    if (key[i] != kGateMasked) key[i] = bias == -__builtin_inf() ? kGateMasked : gate_order(s[i] + bias);
  }
  if constexpr (GROUPS) {
    // Each lane ranks groups lane, lane + 64, ... from the keys in LDS.
    uint64_t* const all = lds + w * 2 * 64 * PER;
    uint64_t* const rank = all + 64 * PER;
    const int size = p.E / p.groups;
#pragma unroll
    for (int i = 0; i < PER; ++i) all[i * 64 + lane] = key[i];
    layer_wave_order();
    for (int g = lane; g < p.groups; g += 64) {
      uint64_t a = 0, b = 0;
      for (int e = g * size; e < (g + 1) * size; ++e) {
        const uint64_t k = all[e];
        if (k > a) {
          b = a;
          a = k;
        } else if (k > b) {
          b = k;
        }
      }
      if (p.group_top > 1 && b != kGateMasked) {
        auto value = [](uint64_t k) {
          return k == kGateNan ? __builtin_nan("") : __builtin_bit_cast(double, k >> 63 ? k & ~((uint64_t)1 << 63) : ~k);
        };
        a = gate_order(value(a) + value(b));
      }
      rank[g] = a;
    }
    layer_wave_order();
    // The best groups are marked with the largest number, which no rank has.
    for (int j = 0; j < p.top_groups; ++j) {
      GateBest b = {0, 0x7fffffff};
      for (int g = lane; g < p.groups; g += 64)
        if (rank[g] != ~(uint64_t)0 && (b.at == 0x7fffffff || rank[g] > b.key)) b = {rank[g], g};
      b = gate_best(b);
      layer_wave_order();
      if (lane == 0) rank[b.at] = ~(uint64_t)0;
      layer_wave_order();
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = i * 64 + lane;
      if (e < p.E && rank[e / size] != ~(uint64_t)0) key[i] = kGateMasked;
    }
  }
  // Choices in falling order: lane j keeps choice j.
  int id = -1;
  double weight = 0;
  for (int j = 0; j < p.top; ++j) {
    GateBest b = {kGateMasked, 0x7fffffff};
    double v = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] > b.key) {
        b = {key[i], i * 64 + lane};
        v = s[i];
      }
    b = gate_best(b);
    if (b.key == kGateMasked) break;
    v = __shfl(v, b.at & 63, 64);
    if (lane == j) {
      id = b.at;
      weight = v;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (b.at == i * 64 + lane) key[i] = kGateMasked;
  }
  if (p.renorm) {
    const double sum = gate_wave_sum(weight);
    weight = sum == 0 ? 0 : weight / sum;
  }
  if (lane < p.top) {
    p.ids[t * p.top + lane] = id;
    p.weights[t * p.top + lane] = (float)(weight * (double)p.scale);
  }
}

// With the chosen s_j, their sum S and g_j = scale dw_j:
//   ds_j = g_j, or renormalised (g_j - sum_k g_k s_k / S) / S
//   softmax: dl_e = s_e (ds_e - sum_j ds_j s_j), the sum 0 where renormalised
//   sigmoid: dl_j = s_j (1 - s_j) ds_j
// Renormalised softmax weights need the chosen logits alone: s_j / S is their own
// softmax.
template <class Row, int PER>
__global__ void __launch_bounds__(256) layer_gate_grad_kernel(const GateGradArgs p) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t t = (int64_t)layer_block(p) * 4 + w;
  if (t >= p.T) return;
  const int id = lane < p.top ? p.ids[t * p.top + lane] : -1;
  float l = -__builtin_inff();
  if ((unsigned)id < (unsigned)p.E) l = gate_load(Row{}, p.L, t * p.ldl + id);
  const bool chosen = l != -__builtin_inff();  // (a masked one has the score 0, and no gradient)
  const float g = chosen ? p.scale * p.dweights[t * p.top + lane] : 0.0f;
  float s = 0.0f, ds = g, d[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) d[i] = 0.0f;
  if (p.score == GEMM_SCORE_SIGMOID) {
    const float z = expf(-l), r = 1.0f / (1.0f + z);
    s = chosen ? r : 0.0f;
    if (p.renorm) {
      const float sum = gate_wave_sum(s), mean = gate_wave_sum(g * s) / sum;
      ds = sum == 0.0f ? 0.0f : (g - mean) / sum;
    }
    ds = chosen ? s * (l > 0.0f ? z * r : 1.0f - s) * ds : 0.0f;  // (1 - s = z / (1 + z))
  } else if (p.renorm) {
    const float top = gate_wave_max(l);
    s = chosen ? expf(l - top) : 0.0f;
    const float sum = gate_wave_sum(s);
    s = chosen ? s / sum : 0.0f;
    const float mean = gate_wave_sum(g * s);  // (every lane takes part)
    ds = s * (g - mean);
  } else {
    float top = -__builtin_inff(), sum = 0.0f, e[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      e[i] = i * 64 + lane < p.E ? gate_load(Row{}, p.L, t * p.ldl + i * 64 + lane) : -__builtin_inff();
      top = e[i] > top ? e[i] : top;
    }
    top = gate_wave_max(top);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      e[i] = e[i] == -__builtin_inff() ? 0.0f : expf(e[i] - top);
      sum += e[i];
    }
    sum = gate_wave_sum(sum);
    s = chosen ? expf(l - top) / sum : 0.0f;
    const float mean = gate_wave_sum(g * s);
    ds = g * s;
#pragma unroll
    for (int i = 0; i < PER; ++i) d[i] = sum == 0.0f ? 0.0f : -(e[i] / sum) * mean;
  }
  for (int j = 0; j < p.top; ++j) {
    const int at = __shfl(id, j, 64);
    const float v = __shfl(ds, j, 64);
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (at == i * 64 + lane && at < p.E) d[i] += v;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if (i * 64 + lane < p.E) gate_store(Row{}, p.dL, t * p.lddl + i * 64 + lane, d[i]);
}

template <class F>
hipError_t gate_for(int rowtype, int E, F f) {
  auto per = [&](auto row) {
    if (E <= 64) return f(row, LayerConst<1>{});
    if (E <= 128) return f(row, LayerConst<2>{});
    if (E <= 256) return f(row, LayerConst<4>{});
    if (E <= 512) return f(row, LayerConst<8>{});
    return f(row, LayerConst<16>{});
  };
  return rowtype == ROW_F32 ? per(GateF32{}) : rowtype == ROW_F16 ? per(TagF16{}) : per(TagBF16{});
}

int check_gate(int64_t T, int64_t E, int64_t top, int dtype, int score, float scale, int& rowtype, int& elem) {
  CHECK(check_choices(T, top));
  CHECK(check_dim("E", E));
  CHECK(check_rowtype(dtype, rowtype, elem));
  if (E > kRouteMaxExperts) return fail(GEMM_ERR_UNSUPPORTED, "more than 1024 experts");
  if (top > kGateTop) return fail(GEMM_ERR_UNSUPPORTED, "more than 64 experts a token");
  if (score != GEMM_SCORE_SOFTMAX && score != GEMM_SCORE_SIGMOID)
    return bad("%s code %lld is not one of GEMM_SCORE_* (0 or 1)", "score", score);
  if (!(scale - scale == 0.0f)) return fail(GEMM_ERR_INVALID_ARG, "scale is not finite");
  return GEMM_OK;
}

}  // namespace
}  // namespace dgt

using namespace dgt;

extern "C" {

int gemm_gate(int64_t T, int64_t E, int64_t top, int dtype, const void* L, int64_t ldl, int score,
              const float* bias, int64_t groups, int64_t top_groups, int64_t group_top, int renorm,
              float scale, int32_t* ids, float* weights, void* stream) {
  return entry("gate", T, top, E, [&]() -> int {
    int rowtype, elem;
    CHECK(check_gate(T, E, top, dtype, score, scale, rowtype, elem));
    if (groups < 1 || E % groups) return bad("%s=%lld does not divide %lld experts", "groups", groups, E);
    if (top_groups < 1 || top_groups > groups)
      return bad("%s=%lld is not between 1 and %lld groups", "top_groups", top_groups, groups);
    const int64_t size = E / groups;
    if (group_top < 1 || group_top > 2 || (group_top > 1 && (groups == 1 || group_top > size)))
      return bad("%s=%lld is neither 1 nor 2, or more than a group's %lld experts", "group_top", group_top, size);
    if (top > top_groups * size) return bad("%s=%lld is more than the %lld experts to choose from", "top", top, top_groups * size);
    const int64_t n = T * top;
    const Mat ml{"L", L, T, E, ldl, elem}, mb{"bias", bias, 1, E, E, 4};
    const Mat mi{"ids", ids, 1, n, n, 4}, mw{"weights", weights, 1, n, n, 4};
    CHECK(check_ld(ml));
    if (n == 0) {
      set_path("noop: empty output");
      return GEMM_OK;
    }
    CHECK(check_ptr(ml));
    if (bias) CHECK(check_ptr(mb));
    CHECK(check_ptr(mi));
    CHECK(check_ptr(mw));
    for (const Mat* w : {&mi, &mw})
      for (const Mat* r : {&ml, &mb}) CHECK(check_apart(*w, *r));
    CHECK(check_apart(mw, mi));
    GateArgs a{};
    a.L = L;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.ldl = ldl;
    a.T = (int)T;
    a.E = (int)E;
    a.top = (int)top;
    a.score = score;
    a.groups = (int)groups;
    a.top_groups = (int)top_groups;
    a.group_top = (int)group_top;
    a.renorm = renorm != 0;
    a.scale = scale;
    set_path("gate, a wave a token");
    const dim3 grid = layer_grid((T + 3) / 4, 256, a.grid_x);
    return launched(gate_for(rowtype, a.E, [&](auto row, auto per) {
      hipStream_t s = static_cast<hipStream_t>(stream);
      if (a.groups > 1)
        return launch_kernel(layer_gate_kernel<decltype(row), decltype(per)::value, true>, grid, dim3(256), s, a);
      return launch_kernel(layer_gate_kernel<decltype(row), decltype(per)::value, false>, grid, dim3(256), s, a);
    }));
  });
}

int gemm_gate_grad(int64_t T, int64_t E, int64_t top, int dtype, const void* L, int64_t ldl, int score,
                   int renorm, float scale, const int32_t* ids, const float* dweights, void* dL,
                   int64_t lddl, void* stream) {
  return entry("gate_grad", T, top, E, [&]() -> int {
    int rowtype, elem;
    CHECK(check_gate(T, E, top, dtype, score, scale, rowtype, elem));
    const int64_t n = T * top;
    const Mat ml{"L", L, T, E, ldl, elem}, md{"dL", dL, T, E, lddl, elem};
    const Mat mi{"ids", ids, 1, n, n, 4}, mw{"dweights", dweights, 1, n, n, 4};
    CHECK(check_ld(ml));
    CHECK(check_ld(md));
    if (T == 0 || E == 0) {
      set_path("noop: empty output");
      return GEMM_OK;
    }
    CHECK(check_ptr(ml));
    CHECK(check_ptr(md));
    if (n > 0) {
      CHECK(check_ptr(mi));
      CHECK(check_ptr(mw));
    }
    CHECK(check_apart_or_same(md, ml));
    CHECK(check_apart(md, mi));
    CHECK(check_apart(md, mw));
    GateGradArgs a{};
    a.L = L;
    a.ids = ids;
    a.dweights = dweights;
    a.dL = dL;
    a.ldl = ldl;
    a.lddl = lddl;
    a.T = (int)T;
    a.E = (int)E;
    a.top = (int)top;
    a.score = score;
    a.renorm = renorm != 0;
    a.scale = scale;
    set_path("gate_grad, a wave a token");
    const dim3 grid = layer_grid((T + 3) / 4, 256, a.grid_x);
    return launched(gate_for(rowtype, a.E, [&](auto row, auto per) {
      return launch_kernel(layer_gate_grad_kernel<decltype(row), decltype(per)::value>, grid, dim3(256),
                           static_cast<hipStream_t>(stream), a);
    }));
  });
}

}  // extern "C"
