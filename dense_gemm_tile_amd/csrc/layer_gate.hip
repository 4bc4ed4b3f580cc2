// The gate: which experts a token goes to, with what weights, and the gradient of
// the logits from the weights'.
//
//   s = softmax(L) or 1 / (1 + exp(-L)),  key = s + bias
//   groups by the sum of their group_top largest keys, experts of the best groups by
//   key;  w = scale s[id]  (renorm: / sum of the chosen s)
//
// A wave takes a token. Choices are whole numbers and must not hang on a rounding, so
// keys count as they are in 64 bits; in 64 bits throughout, the exponentials and the
// search take most of the time (16384 tokens, 8 of 256 experts in groups, with the
// gradient: 68 us, 24 so). So keys are made and searched in float32, with a bound
// of their error, and what comes too close for it is decided in 64 bits.
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
  int lanes;            // 1 << lanes lanes hold a group
  int bits;             // that number an expert
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
template <class Row>
struct GateElemOf { using type = unsigned short; };
template <>
struct GateElemOf<GateF32> { using type = float; };
template <class Row>
using GateElem = typename GateElemOf<Row>::type;
__device__ __forceinline__ float gate_float(GateF32, float v) { return v; }
template <class Tag>
__device__ __forceinline__ float gate_float(Tag t, unsigned short v) { return layer_f32(t, v); }
__device__ __forceinline__ float gate_load(GateF32, const void* p, int64_t at) { return static_cast<const float*>(p)[at]; }
template <class Tag>
__device__ __forceinline__ float gate_load(Tag t, const void* p, int64_t at) {
  return layer_f32(t, static_cast<const unsigned short*>(p)[at]);
}
__device__ __forceinline__ float gate_elem(GateF32, float v) { return v; }
template <class Tag>
__device__ __forceinline__ unsigned short gate_elem(Tag t, float v) { return layer_16(t, v); }

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

__device__ __forceinline__ double gate_value(uint64_t k) {
  return k == kGateNan ? __builtin_nan("") : __builtin_bit_cast(double, k >> 63 ? k & ~((uint64_t)1 << 63) : ~k);
}

// Reductions over groups of 16 or of all 64 lanes, by lane swaps; every lane gets the result.
template <int CTRL>
__device__ __forceinline__ unsigned gate_swap(unsigned v) {
  return (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
template <int LANES, class F>
__device__ __forceinline__ unsigned gate_reduce(unsigned v, F join) {
  static_assert(LANES == 16 || LANES == 64, "");
  v = join(v, gate_swap<0xB1>(v));   // lanes 1 0 3 2 of each 4
  v = join(v, gate_swap<0x4E>(v));   // 2 3 0 1
  v = join(v, gate_swap<0x141>(v));  // 8 lanes mirrored
  v = join(v, gate_swap<0x140>(v));  // 16 lanes mirrored
  if constexpr (LANES == 64) {
    const auto h = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = join(h[0], h[1]);
    const auto w = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = join(w[0], w[1]);
  }
  return v;
}
template <int LANES>
__device__ __forceinline__ unsigned gate_max32(unsigned v) {
  return gate_reduce<LANES>(v, [](unsigned a, unsigned b) { return a > b ? a : b; });
}
template <int LANES>
__device__ __forceinline__ float gate_sum32(float v) {
  return __builtin_bit_cast(float, gate_reduce<LANES>(__builtin_bit_cast(unsigned, v), [](unsigned a, unsigned b) {
    return __builtin_bit_cast(unsigned, __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b));
  }));
}
// The largest of the wave's keys, and of equal ones the first; every lane gets both.
struct GateBest {
  uint64_t key;
  int at;
};
__device__ __forceinline__ GateBest gate_best(GateBest b) {
  const unsigned high = gate_max32<64>((unsigned)(b.key >> 32));
  const unsigned low = gate_max32<64>((unsigned)(b.key >> 32) == high ? (unsigned)b.key : 0u);
  const uint64_t key = (uint64_t)high << 32 | low;
  const unsigned at = ~gate_max32<64>(b.key == key ? ~(unsigned)b.at : 0u);
  return {key, (int)at};
}

// The choices of token t in 64 bits: lane j gets the id and the score of choice j (-1 and 0
// past the last), renormalised softmax scores over the largest of them. Lane l holds experts
// l, l + 64, ... all: 2 * 64 * PER numbers of LDS, this wave's own (GROUPS).
template <class Row, int PER, bool GROUPS>
__device__ __forceinline__ void gate_in_64_bits(const GateArgs& p, int64_t t, uint64_t* all, int& id, double& weight) {
  const int lane = threadIdx.x & 63;
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
  // Without a bias the order is the logits', also where scores are equal; groups that two scores
  // rank have their sum.
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 64 + lane;
    const double bias = p.bias && e < p.E ? (double)p.bias[e] : 0.0;
    if (key[i] != kGateMasked) key[i] = bias == -__builtin_inf() ? kGateMasked : gate_order(s[i] + bias);
  }
  auto by_logits = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < PER; ++i)  // (+ 0: -0 is no other number)
      if (key[i] != kGateMasked && key[i] != kGateNan)
        key[i] = gate_order((double)gate_load(Row{}, p.L, t * p.ldl + i * 64 + lane) + 0.0);
  };
  if (!p.bias && !(GROUPS && p.group_top > 1)) by_logits();
  if constexpr (GROUPS) {
    // Each lane ranks groups lane, lane + 64, ... from the keys in LDS.
    uint64_t* const rank = all + 64 * PER;
    const int size = p.E / p.groups;
#pragma unroll
    for (int i = 0; i < PER; ++i) all[i * 64 + lane] = key[i];
    layer_wave_order();
    for (int g = lane; g < p.groups; g += 64) {
      uint64_t a = 0, b = 0;
#pragma unroll 4
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
        a = gate_order(gate_value(a) + gate_value(b));
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
    if (!p.bias && p.group_top > 1) by_logits();
  }
  // Choices in falling order.
  id = -1;
  weight = 0;
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
  // Renormalised softmax scores are the softmax of the chosen logits, which has a sum also where
  // all chosen scores are 0 in 64 bits, as far below the largest logit as a bias can reach.
  if (p.score == GEMM_SCORE_SOFTMAX && p.renorm) {
    const double l = id >= 0 ? (double)gate_load(Row{}, p.L, t * p.ldl + id) : -__builtin_inf();
    const double best = gate_wave_max(l);
    if (id >= 0 && weight == weight) weight = exp(l - best);
  }
}

// The weight of a choice of score s among scores that sum to `total`: 0 without a choice, also
// beside a NaN.
__device__ __forceinline__ float gate_weight(const GateArgs& p, int id, double s, double total) {
  return id < 0 || total == 0 ? 0.0f : (float)(s / total * (double)p.scale);
}

// A sigmoid score and one less it, each to a few half steps of itself, also among float32's
// subnormal numbers.
struct GateScore {
  float s, rest, t;  // t: exp(-|l|)
};
__device__ __forceinline__ GateScore gate_scores(float l) {
  const float t = expf(-__builtin_fabsf(l)), one = 1.0f / (1.0f + t), small = t / (1.0f + t);
  return l < 0.0f ? GateScore{small, one, t} : GateScore{one, small, t};
}

// For keys: exp(x) within 2^-22 of itself, and 1 / (1 + exp(-x)) within 2^-21, where |x| is below
// 87; below 2^-125 both may be 0, which the 1e-30 of unsure() covers. The exponent of 2 in
// two floats, so that its rounding does not grow with it. (The library's exponential
// and division: 16384 tokens, 8 of 256 experts with a bias 18 us, 16 so.)
__device__ __forceinline__ float gate_exp(float x) {
  const float c = __builtin_amdgcn_fmed3f(x, -200.0f, 200.0f);
  const float hi = c * kLog2e, lo = __builtin_fmaf(c, 1.92596298e-8f, __builtin_fmaf(c, kLog2e, -hi));
  const float e = __builtin_amdgcn_exp2f(hi);
  return e < __builtin_inff() ? __builtin_fmaf(e, 0.6931471805599453f * lo, e) : e;
}
__device__ __forceinline__ float gate_sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + gate_exp(-x)); }
// Numbers as integers of the same order (NaN has no place).
__device__ __forceinline__ unsigned gate_order32(float v) {
  const unsigned u = __builtin_bit_cast(unsigned, v);
  return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float gate_value32(unsigned k) {
  return __builtin_bit_cast(float, k >> 31 ? k & 0x7fffffffu : ~k);
}
// PER elements of `size` neighbouring ones, shared by LANES lanes four at a time: item i of
// lane `in` is element 4 (i / 4 LANES + in) + i % 4.
__device__ __forceinline__ int gate_item(int i, int lanes, int in) { return 4 * ((i >> 2) * lanes + in) + (i & 3); }
template <class Row>
struct __attribute__((packed, aligned(sizeof(GateElem<Row>)))) GateFour {
  GateElem<Row> e[4];
};
template <class Row, int PER>
__device__ __forceinline__ void gate_load_row(const void* p, int64_t at, int lanes, int in, int size, float none,
                                              float (&f)[PER]) {
  static_assert(PER % 4 == 0, "whole fours");
#pragma unroll
  for (int i = 0; i < PER; i += 4) {
    const int first = gate_item(i, lanes, in);
    if (first + 4 <= size) {
      const auto v = *reinterpret_cast<const GateFour<Row>*>(static_cast<const GateElem<Row>*>(p) + at + first);
#pragma unroll
      for (int e = 0; e < 4; ++e) f[i + e] = gate_float(Row{}, v.e[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) f[i + e] = first + e < size ? gate_load(Row{}, p, at + first + e) : none;
    }
  }
}
template <class Row, int PER>
__device__ __forceinline__ void gate_store_row(void* p, int64_t at, int lanes, int in, int size, const float (&f)[PER]) {
#pragma unroll
  for (int i = 0; i < PER; i += 4) {
    const int first = gate_item(i, lanes, in);
    if (first + 4 <= size) {
      GateFour<Row> v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v.e[e] = gate_elem(Row{}, f[i + e]);
      *reinterpret_cast<GateFour<Row>*>(static_cast<GateElem<Row>*>(p) + at + first) = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (first + e < size) static_cast<GateElem<Row>*>(p)[at + first + e] = gate_elem(Row{}, f[i + e]);
    }
  }
}

// A group's place among its token's by their ranks in 64 bits, for sigmoid scores: the group is
// shared by `lanes` lanes, of which this is the in-th; items: bits of this lane's experts that
// count; base: the token's first lane.
template <class Row>
__device__ __forceinline__ int gate_group_place(const GateArgs& p, int64_t t, unsigned items, int group, int in, int lanes, int base) {
  const int first = group * (p.E / p.groups);
  uint64_t a = kGateMasked, b = kGateMasked;  // the two largest keys
  auto enter = [&](uint64_t k) __attribute__((always_inline)) {
    const uint64_t least = k < a ? k : a;
    a = k > a ? k : a;
    b = least > b ? least : b;
  };
  for (; items; items &= items - 1) {
    const int e = first + gate_item(__builtin_ctz(items), lanes, in);
    enter(gate_order(1.0 / (1.0 + exp(-(double)gate_load(Row{}, p.L, t * p.ldl + e))) + (p.bias ? (double)p.bias[e] : 0.0)));
  }
  for (int d = 1; d < lanes; d <<= 1) {
    const uint64_t oa = __shfl_xor(a, d, 64), ob = __shfl_xor(b, d, 64);
    enter(oa);
    enter(ob);
  }
  if (p.group_top > 1 && b != kGateMasked) a = gate_order(gate_value(a) + gate_value(b));
  int at = 0;
  for (int g = 0; g < p.groups; ++g) {
    const uint64_t k = __shfl(a, base + g * lanes, 64);
    at += k > a || (k == a && g < group);
  }
  return at;
}

// The float32 search. LANES lanes take a token (four tokens a wave, or one). A key is an
// integer of the float32 key's order; the largest one below the last choice is the largest of
// (key - last) as unsigned numbers, so nothing is removed. Its lowest bits say whose it
// is, in place of a search:
//   experts ranked by logits (without a bias their order is the scores'): the expert's
//     number from behind, so that keys of a token differ and of equal logits the first
//     expert's is larger. Exact for 16-bit logits, which have zeros there, and for
//     float32 ones that differ above these bits.
//   experts ranked by scores and a bias: the lane's item from behind; the lane is the one
//     that has the key, the first of several. Two keys next to each other in the order have
//     to be further apart than their errors: relative to the score 1.25 2^-21 (sigmoid: 2^-21,
//     and half a step for the bias) or 2^-17 (softmax: the largest logit taken off first,
//     half a step of a number below 128 where the score is not 0 to float32, 2^-18; the
//     sum, whose additions one after the other are PER + 6 at most), and relative to the
//     key 2^-19 for the lowest bits.
//   groups: ranks without such bits, apart by their keys' errors and half a step of the sum.
// (Experts' numbers in the lowest bits of biased keys too: one token in ten of the case above
// was too close, 54 us for the choices alone.)
//
// Neighbours that are too close are one token in 300 there, and one token done again in 64 bits
// takes about 10 us more than the others (22 us in all; 16.5 so). So with sigmoid scores, whose keys do not
// hang on each other, what is close is put right alone: groups are ranked by their keys in 64
// bits before the search, and behind it, which then goes on to the first key that is clear of
// the last choice, the choices and those beyond them, a lane each, are sorted.
template <class Row, int LANES, int PER, bool GROUPS>
__global__ void __launch_bounds__(256) layer_gate_kernel(const GateArgs p) {
  constexpr int WIDE = 64 / LANES;                     // tokens a wave
  constexpr int PER64 = PER / WIDE > 0 ? PER / WIDE : 1;
  __shared__ uint64_t lds[GROUPS ? 4 * 2 * 64 * PER64 : 1];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, li = lane & (LANES - 1);
  const int64_t t0 = ((int64_t)layer_block(p) * 4 + w) * WIDE;
  if (t0 >= p.T) return;
  const int64_t mine = t0 + lane / LANES, t = mine < p.T ? mine : p.T - 1;  // (the last token again past it)
  const bool soft = p.score == GEMM_SCORE_SOFTMAX;
  const bool scored = p.bias != nullptr, ranked = GROUPS && (scored || p.group_top > 1);  // by scores: experts, groups
  // The group that this lane holds a part of.
  const int lanes = GROUPS ? 1 << p.lanes : LANES, group = GROUPS ? li >> p.lanes : 0;
  const int in = GROUPS ? li & (lanes - 1) : li;
  const int size = GROUPS ? (group < p.groups ? p.E / p.groups : 0) : p.E, first = GROUPS ? group * (p.E / p.groups) : 0;
  const unsigned low = scored ? PER - 1 : (1u << p.bits) - 1;
  const float inf = __builtin_inff();

  float l[PER];
  gate_load_row<Row, PER>(p.L, t * p.ldl + first, lanes, in, size, -inf, l);
  unsigned key[PER];
  bool close = false, odd = false;
  float top = -inf, sum = 0.0f, bmax = 0.0f;
#pragma unroll
  for (int i = 0; i < PER; ++i) odd |= soft ? !(l[i] < inf) : l[i] != l[i];
  float s[PER];  // scores, where they rank
  if (soft && (scored || ranked || !p.renorm)) {
#pragma unroll
    for (int i = 0; i < PER; ++i) top = l[i] > top ? l[i] : top;
    top = gate_value32(gate_max32<LANES>(gate_order32(top)));
    const float base = top == -inf ? 0.0f : top;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      s[i] = l[i] == -inf ? 0.0f : gate_exp(l[i] - base);
      sum += s[i];
    }
    sum = gate_sum32<LANES>(sum);
    if (scored || ranked) {
      const float inv = 1.0f / sum;
#pragma unroll
      for (int i = 0; i < PER; ++i) s[i] = s[i] * inv;
    }
  } else if (scored || ranked) {
#pragma unroll
    for (int i = 0; i < PER; ++i) s[i] = gate_sigmoid(l[i]);
  }
  if (p.bias) {
    float b[PER];
    gate_load_row<GateF32, PER>(p.bias, first, lanes, in, size, -inf, b);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool masked = l[i] == -inf || b[i] == -inf;
      odd |= !masked && !(__builtin_fabsf(b[i]) < inf);
      l[i] = masked ? -inf : s[i] + b[i];
      bmax = !masked && __builtin_fabsf(b[i]) > bmax ? __builtin_fabsf(b[i]) : bmax;
    }
    bmax = gate_value32(gate_max32<LANES>(gate_order32(bmax)));
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)  // (+ 0: -0 is no other number)
    key[i] = l[i] == -inf ? 0u : (gate_order32(l[i] + 0.0f) & ~low) | (low - (scored ? i : first + gate_item(i, lanes, in)));
  // Whether two keys, or two ranks, a above b, are too close for their errors.
  const float err = soft ? 0x1p-17f : 0x1.4p-21f;
  auto unsure = [&](unsigned a, unsigned b, unsigned rest, float cut, float bias) {
    const float u = gate_value32(a & ~rest), v = gate_value32(b & ~rest), size = __builtin_fabsf(u) + __builtin_fabsf(v);
    return u - v <= cut * size + err * (size + 2.0f * bias) + 1e-30f;
  };
  auto same = [&](unsigned a, unsigned b) { return sizeof(GateElem<Row>) == 4 && ((a ^ b) & ~low) == 0; };
  constexpr uint64_t all = LANES == 64 ? ~(uint64_t)0 : ((uint64_t)1 << (LANES & 63)) - 1;
  if constexpr (GROUPS) {
    // The two largest keys (where scores rank groups: without their lowest bits' numbers) of the
    // group, in each of its lanes.
    unsigned a = 0, b = 0;
    auto enter = [&](unsigned k) {
      const unsigned least = k < a ? k : a;
      a = k > a ? k : a;
      b = least > b ? least : b;
    };
#pragma unroll
    for (int i = 0; i < PER; ++i) enter(ranked ? (key[i] ? gate_order32((scored ? l[i] : s[i]) + 0.0f) : 0u) : key[i]);
    auto join = [&](unsigned oa, unsigned ob) {
      enter(oa);
      enter(ob);
    };
    if (p.lanes > 0) join(gate_swap<0xB1>(a), gate_swap<0xB1>(b));
    if (p.lanes > 1) join(gate_swap<0x4E>(a), gate_swap<0x4E>(b));
    if (p.lanes > 2) join(gate_swap<0x141>(a), gate_swap<0x141>(b));
    if (p.lanes > 3) join(gate_swap<0x140>(a), gate_swap<0x140>(b));
    if (p.lanes > 4) join(__shfl_xor(a, 16, 64), __shfl_xor(b, 16, 64));
    if (ranked && a && p.group_top > 1 && b) a = gate_order32(gate_value32(a) + gate_value32(b) + 0.0f);
    // The best groups' ranks, down to the last one that is kept, and the next.
    unsigned rank = group < p.groups ? a : 0, last = ~0u;
    const unsigned own = rank;
    int kept = 0;  // (groups of one rank leave together)
    for (int j = 0; j < p.top_groups; ++j) {
      const unsigned m = gate_max32<LANES>(rank);
      const int many = __builtin_popcountll(__ballot(rank == m) >> (lane - li) & all) >> p.lanes;
      if (m && kept < p.top_groups) {
        last = m;
        kept += many;
        rank = rank < m ? rank : 0;
      }
    }
    const unsigned next = gate_max32<LANES>(rank);
    // (A sum of two keys: half a step.)
    close = kept > p.top_groups || (next && (ranked ? unsure(last, next, 0u, 0x1p-23f, 2.0f * bmax) : same(last, next)));
    bool out = own < last;
    if (ranked && !soft && __ballot(close)) {
      // Of the groups of such tokens the keys that may be one of the two largest.
      const float second = b ? gate_value32(b) : -inf;
      const float least = second - (2.0f * err * (__builtin_fabsf(second) + 2.0f * bmax) + 1e-30f);
      unsigned items = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) items |= (key[i] && (scored ? l[i] : s[i]) >= least ? 1u : 0u) << i;
      const bool better =
          gate_group_place<Row>(p, t, close ? items : 0u, group, in, lanes, lane - li) < p.top_groups;
      out = close ? !better : out;
      close = false;
    }
    if (out) {
#pragma unroll
      for (int i = 0; i < PER; ++i) key[i] = 0;
    }
  }
  // The choices in falling order, and one more that the last one must be clear of. Lane j keeps
  // choice j: its key and the lane that has it. (What is done with them is done once, behind.)
  const bool sorted = scored && !soft;
  unsigned best = 0, below = 0, kept = 0;  // below: what this lane's next key is less than
  int from = 0, at = 0;
  auto step = [&](bool first) __attribute__((always_inline)) {
    unsigned m = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = key[i] - below > m ? key[i] - below : m;
    // (Before the first: below is 0 and m the largest key. Where none is left below it, m is a
    // difference to one that is not.)
    m += below;
    m = !first && m >= below ? 0 : m;
    best = gate_max32<LANES>(m);
    below = best;
    if (scored) {  // of several the first; the others' lanes have theirs ahead of them
      from = __builtin_ctzll(__ballot(m == best) >> (lane - li) & all);
      below += li > from;
    }
  };
  for (int j = 0; j <= p.top; ++j) {
    step(j == 0);
    kept = li == j ? best : kept;
    at = li == j ? from : at;
  }
  // Whether lane j's is too close to the one before; in front of the first none is.
  auto doubtful = [&](unsigned a, unsigned b) { return b && (scored ? unsure(a, b, low, 0x1p-19f, bmax) : same(a, b)); };
  const unsigned before = __shfl_up(kept, 1, LANES);
  const uint64_t doubts = __ballot(li > 0 && li <= p.top && doubtful(before, kept)) >> (lane - li) & all;
  bool near = doubts != 0, open = sorted && p.top < LANES && (doubts >> (p.top & 63) & 1);
  if (p.top == LANES)  // (no lane for the one beyond)
    close |= (__ballot(li == LANES - 1 && doubtful(kept, best)) >> (lane - li) & all) != 0;
  // Where 64 bits decide about the last choice, those beyond it, to the first that is clear.
  if (li == p.top && !open) kept = 0;
  for (int j = p.top + 1; j < LANES && __ballot(open); ++j) {
    const unsigned last = best;
    step(false);
    open = open && doubtful(last, best);
    if (li == j && open) {
      kept = best;
      at = from;
    }
  }
  close |= sorted ? open : near;  // (more than a lane each)
  int id = low - (kept & low);
  if (scored) id = (GROUPS ? (at >> p.lanes) * (p.E / p.groups) : 0) + gate_item(id, lanes, GROUPS ? at & (lanes - 1) : at);
  if (!kept) id = -1;
  if (sorted && __ballot(near)) {
    uint64_t exact = kGateMasked;
    if (id >= 0) {
      const double score = 1.0 / (1.0 + exp(-(double)gate_load(Row{}, p.L, t * p.ldl + id)));
      exact = gate_order(score + (double)p.bias[id]);
    }
    int place = id >= 0 ? 0 : li;
#pragma unroll 4
    for (int u = 0; u < LANES; ++u) {
      const int other = __shfl(id, u, LANES);
      const uint64_t k = __shfl(exact, u, LANES);
      place += id >= 0 && other >= 0 && (k > exact || (k == exact && other < id));
    }
    id = __builtin_amdgcn_ds_permute((lane - li + place) << 2, id);
  }
  if (li >= p.top) id = -1;
  // Weights. Renormalised softmax scores are the softmax of the chosen logits.
  const bool chosen = id >= 0;
  const float z = chosen ? gate_load(Row{}, p.L, t * p.ldl + id) : -inf;
  float out = 0.0f;
  if (!soft) {
    out = gate_scores(z).s;
  } else if (p.renorm) {
    const float best = gate_value32(gate_max32<LANES>(chosen ? gate_order32(z) : 0u));
    out = expf(z - best);
  } else {
    out = expf(z - top) / sum;
  }
  out = chosen ? out : 0.0f;
  if (p.renorm) {
    const float total = gate_sum32<LANES>(out);
    close |= total < 1e-30f && gate_max32<LANES>(chosen) != 0u;  // (next to float32's smallest numbers)
    out = chosen ? out / total : 0.0f;
  }
  // Tokens that float32 does not decide go through 64 bits.
  const uint64_t again = __ballot(close || odd);
  if (li < p.top && mine < p.T && (again >> (lane - li) & all) == 0) {
    p.ids[t * p.top + li] = id;
    p.weights[t * p.top + li] = out * p.scale;
  }
#pragma unroll
  for (int u = 0; u < WIDE; ++u) {
    if ((again >> (u * LANES) & all) == 0 || t0 + u >= p.T) continue;
    int found;
    double exact;
    gate_in_64_bits<Row, PER64, GROUPS>(p, t0 + u, lds + w * 2 * 64 * PER64 * GROUPS, found, exact);
    const double total = p.renorm ? gate_wave_sum(exact) : 1.0;
    if (lane < p.top) {
      p.ids[(t0 + u) * p.top + lane] = found;
      p.weights[(t0 + u) * p.top + lane] = gate_weight(p, found, exact, total);
    }
  }
}

// Every token in 64 bits: groups that no power of two of lanes holds.
template <class Row>
__global__ void __launch_bounds__(256) layer_gate_exact_kernel(const GateArgs p) {
  __shared__ uint64_t lds[4 * 2 * 64 * 16];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t t = (int64_t)layer_block(p) * 4 + w;
  if (t >= p.T) return;
  int id;
  double weight;
  gate_in_64_bits<Row, 16, true>(p, t, lds + w * 2 * 64 * 16, id, weight);
  const double total = p.renorm ? gate_wave_sum(weight) : 1.0;
  if (lane < p.top) {
    p.ids[t * p.top + lane] = id;
    p.weights[t * p.top + lane] = gate_weight(p, id, weight, total);
  }
}

constexpr float kGateNoScore = -709.78271484375f;  // exp(-it) is infinity in 64 bits
// With the chosen s_j, their sum S and g_j = scale dw_j:
//   ds_j = g_j, or renormalised (g_j - sum_k g_k s_k / S) / S
//   softmax: dl_e = s_e (ds_e - sum_j ds_j s_j), the sum 0 where renormalised
//   sigmoid: dl_j = s_j (1 - s_j) ds_j, renormalised s_j / S (1 - s_j) (g_j - sum_k g_k s_k / S)
// Renormalised softmax weights need the chosen logits alone: s_j / S is their own
// softmax.
template <class Row, int LANES, int PER>
__global__ void __launch_bounds__(256) layer_gate_grad_kernel(const GateGradArgs p) {
  const int lane = threadIdx.x & 63, li = lane & (LANES - 1);
  const int64_t t = ((int64_t)layer_block(p) * 4 + (threadIdx.x >> 6)) * (64 / LANES) + lane / LANES;
  const bool there = t < p.T;
  const int id = there && li < p.top ? p.ids[t * p.top + li] : -1;
  const float inf = __builtin_inff();
  float l = -inf;
  if ((unsigned)id < (unsigned)p.E) l = gate_load(Row{}, p.L, t * p.ldl + id);
  const bool chosen = l != -inf;  // (a masked one has the score 0, and no gradient)
  const float g = chosen ? p.scale * p.dweights[t * p.top + li] : 0.0f;
  const int size = there ? p.E : 0;
  float s = 0.0f, ds = g, d[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) d[i] = 0.0f;
  if (p.score == GEMM_SCORE_SIGMOID) {
    const GateScore z = gate_scores(l);
    s = chosen ? z.s : 0.0f;
    if (p.renorm) {
      // The shares s / sum have ordinary sizes also where s does not (from -104 on float32 has no
      // number for it), so they are made of scores over exp(low): exp(l - low) / (1 + exp(l)).
      const float top = gate_value32(gate_max32<LANES>(l == l && chosen ? gate_order32(l) : 0u));
      const float low = top < 0.0f ? top : 0.0f;
      const float up = chosen ? (l < 0.0f ? expf(l - low) / (1.0f + z.t) : z.s) : 0.0f;
      const float share = up / gate_sum32<LANES>(up);  // (of a single choice exactly 1, its gradient 0)
      const float mean = gate_sum32<LANES>(chosen ? g * share : 0.0f);
      // Past the last logit whose score is above 0 in 64 bits the weights are 0, and stay so.
      s = top <= kGateNoScore ? 0.0f : share;
      ds = g - mean;
    }
    ds = chosen ? s * z.rest * ds : 0.0f;
  } else if (p.renorm) {
    const bool nan = l != l;
    const float top = gate_value32(gate_max32<LANES>(nan ? 0u : gate_order32(l)));
    s = chosen ? expf(l - top) : 0.0f;
    const float sum = gate_sum32<LANES>(s);
    s = chosen ? s / sum : 0.0f;
    const float mean = gate_sum32<LANES>(g * s);  // (every lane takes part)
    ds = s * (g - mean);
  } else {
    float top = -inf, sum = 0.0f, e[PER];
    gate_load_row<Row, PER>(p.L, t * p.ldl, LANES, li, size, -inf, e);
#pragma unroll
    for (int i = 0; i < PER; ++i) top = e[i] > top ? e[i] : top;
    top = gate_value32(gate_max32<LANES>(gate_order32(top)));
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      e[i] = e[i] == -inf ? 0.0f : expf(e[i] - top);
      sum += e[i];
    }
    sum = gate_sum32<LANES>(sum);
    s = chosen ? expf(l - top) / sum : 0.0f;
    const float mean = gate_sum32<LANES>(g * s);
    ds = g * s;
#pragma unroll
    for (int i = 0; i < PER; ++i) d[i] = sum == 0.0f ? 0.0f : -(e[i] / sum) * mean;
  }
  for (int j = 0; j < p.top; ++j) {
    // Choice j's place: item i of lane `in` of this token's lanes, if it is kept.
    const int from = (lane & ~(LANES - 1)) + j;
    const int at = __shfl(id, from, 64);
    const float v = __shfl(ds, from, 64);
    const int i0 = (at >> 2) / LANES * 4 + (at & 3);
    const bool here = (unsigned)at < (unsigned)size && ((at >> 2) & (LANES - 1)) == li;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (here && i0 == i) d[i] += v;
  }
  gate_store_row<Row, PER>(p.dL, t * p.lddl, LANES, li, size, d);
}

// f(row, lanes, per) with the form of a call: 16 lanes a token where they hold its experts (and a
// choice each), 64 otherwise.
template <class F>
hipError_t gate_for(int rowtype, int form, F f) {
  auto with = [&](auto row) {
    switch (form) {
      case 0: return f(row, LayerConst<16>{}, LayerConst<4>{});
      case 1: return f(row, LayerConst<16>{}, LayerConst<8>{});
      case 2: return f(row, LayerConst<16>{}, LayerConst<16>{});
      case 3: return f(row, LayerConst<64>{}, LayerConst<4>{});
      case 4: return f(row, LayerConst<64>{}, LayerConst<8>{});
      default: return f(row, LayerConst<64>{}, LayerConst<16>{});
    }
  };
  return rowtype == ROW_F32 ? with(GateF32{}) : rowtype == ROW_F16 ? with(TagF16{}) : with(TagBF16{});
}
constexpr int kGateForms = 6;
constexpr int kGateFormLanes[kGateForms] = {16, 16, 16, 64, 64, 64}, kGateFormPer[kGateForms] = {4, 8, 16, 4, 8, 16};
// The first form that holds E experts in so many groups, each in a power of two of lanes
// (log2 of it: lanes), and `top` choices; kGateForms if none does.
int gate_form(int64_t E, int64_t groups, int64_t top, int& lanes) {
  const int64_t size = E / groups;
  for (int f = 0; f < kGateForms; ++f) {
    if (top > kGateFormLanes[f]) continue;
    for (lanes = 0; groups << lanes <= kGateFormLanes[f]; ++lanes)
      if ((int64_t)kGateFormPer[f] << lanes >= size) return f;
  }
  return kGateForms;
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
    if (group_top < 1 || group_top > 2 || (groups > 1 && group_top > size))
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
    while (E > 1 << a.bits) ++a.bits;
    const int form = gate_form(E, groups, top, a.lanes);
    hipStream_t s = static_cast<hipStream_t>(stream);
    if (form == kGateForms) {  // groups that do not fit a wave
      set_path("gate in 64 bits");
      const dim3 grid = layer_grid((T + 3) / 4, 256, a.grid_x);
      const auto k = rowtype == ROW_F32 ? layer_gate_exact_kernel<GateF32> : rowtype == ROW_F16 ? layer_gate_exact_kernel<TagF16> : layer_gate_exact_kernel<TagBF16>;
      return launched(launch_kernel(k, grid, dim3(256), s, a));
    }
    set_path(std::string("gate, ") + (kGateFormLanes[form] == 16 ? "16 lanes a token" : "a wave a token"));
    const int tokens = 4 * 64 / kGateFormLanes[form];
    const dim3 grid = layer_grid((T + tokens - 1) / tokens, 256, a.grid_x);
    return launched(gate_for(rowtype, form, [&](auto row, auto lanes, auto per) {
      constexpr int LANES = decltype(lanes)::value, PER = decltype(per)::value;
      if (a.groups > 1) return launch_kernel(layer_gate_kernel<decltype(row), LANES, PER, true>, grid, dim3(256), s, a);
      return launch_kernel(layer_gate_kernel<decltype(row), LANES, PER, false>, grid, dim3(256), s, a);
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
    int lanes;
    const int form = gate_form(E, 1, top, lanes), tokens = 4 * 64 / kGateFormLanes[form];
    set_path(std::string("gate_grad, ") + (kGateFormLanes[form] == 16 ? "16 lanes a token" : "a wave a token"));
    const dim3 grid = layer_grid((T + tokens - 1) / tokens, 256, a.grid_x);
    return launched(gate_for(rowtype, form, [&](auto row, auto lanes, auto per) {
      return launch_kernel(layer_gate_grad_kernel<decltype(row), decltype(lanes)::value, decltype(per)::value>, grid, dim3(256),
                           static_cast<hipStream_t>(stream), a);
    }));
  });
}

}  // extern "C"
