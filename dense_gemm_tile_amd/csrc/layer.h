// The layer operators' products: what one call carries, how a workgroup finds
// its tile, the activations, and the epilogue.
//
//   dense     Y = act(op(A) @ op(B) + bias) + R
//   by rows   the rows of A and Y are cut into groups by offsets held on the
//             GPU, each with its own B and bias
//   by sum    the summed dimension is cut into groups instead, each with its
//             own Y (the gradient of grouped weights)
#pragma once

#include "gemm_mfma_impl.h"

namespace dgt {

enum LayerMode : int { LAYER_DENSE = 0, LAYER_ROWS = 1, LAYER_SUM = 2 };
enum LayerAct : int { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_ERF = 3, ACT_SILU = 4, ACT_SCALE = 5 };

struct LayerArgs {
  const void* A;
  const void* B;
  const void* bias;  // null: none
  const void* R;     // null: none
  void* Y;
  void* Z;           // null: not kept
  const int* offsets;
  const float* scale;  // ACT_SCALE, of products that are a step of another operator: z *scale
  int64_t lda, ldb, ldr, ldy, ldz;  // elements
  int64_t stride_b;  // by rows: elements from one group's B to the next
  int64_t stride_y;  // by sum: elements from one group's Y (and R) to the next
  int M, N, K;       // by rows: M counts all rows; by sum: K does
  int G, mode, act;
  int out32;         // Y (and R) hold float32, else the operands' 16-bit type
  int whole8;        // N is a multiple of 8
  int a_vw, b_vw;    // staging vector widths of A and B (general kernel)
  int a_direct, b_direct;  // A, B in whole 16-byte pieces (ring kernel)
  int tiles_m, tiles_n;  // of one group (by sum, dense); by rows: tiles_m is not used
  int group_m;
};

// One group's product and one tile of it. Pointers and sizes are uniform.
struct LayerTile {
  const char* A;
  const char* B;
  const char* bias;
  const char* R;
  char* Y;
  char* Z;
  int M, N, K;   // of this group
  int m0, n0;    // the tile's first row and column
};

__device__ __forceinline__ int layer_clamp(int v, int hi) { return v < 0 ? 0 : (v > hi ? hi : v); }
template <class T>
__device__ __forceinline__ T* layer_uniform(T* p) {
  const uint64_t u = (uint64_t)p;
  const unsigned lo = __builtin_amdgcn_readfirstlane((unsigned)u);
  const unsigned hi = __builtin_amdgcn_readfirstlane((unsigned)(u >> 32));
  return (T*)(((uint64_t)hi << 32) | lo);
}

// Rows [first, first + count) of group g, clamped to the call's rows whatever
// the offsets hold.
__device__ __forceinline__ void layer_group(const int* offsets, int g, int rows, int& first,
                                            int& count) {
  first = layer_clamp(offsets[g], rows);
  const int end = layer_clamp(offsets[g + 1], rows);
  count = end > first ? end - first : 0;
}

// Tiles of BM rows that the groups hold in all, and, for a tile index below
// that, its group and its index within the group. Each lane counts the tiles
// of one group of 64; a scan over the wave places them. Every wave of a
// workgroup does this for itself: the offsets stay in its caches, and no LDS
// has to be kept for it.
//
// Offsets that decrease can make groups overlap and their tiles add up past 32
// bits (65535 groups of up to 2^27 tiles). Sums then wrap, as unsigned numbers,
// and a tile finds some group below G or none.
template <int BM>
struct LayerRows {
  __device__ static inline unsigned tiles_of(const LayerArgs& p, int g, int& first, int& count) {
    if (g >= p.G) {
      first = count = 0;
      return 0u;
    }
    layer_group(p.offsets, g, p.M, first, count);
    return (unsigned)(count + BM - 1) / BM;
  }
  __device__ static inline unsigned wave_scan(unsigned v, int lane) {  // inclusive
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const unsigned o = __shfl_up(v, d, 64);
      if (lane >= d) v += o;
    }
    return v;
  }
  __device__ static inline unsigned total(const LayerArgs& p, int lane) {
    unsigned sum = 0;
    for (int g0 = 0; g0 < p.G; g0 += 64) {
      int f, c;
      sum += tiles_of(p, g0 + lane, f, c);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d, 64);
    return __builtin_amdgcn_readfirstlane(sum);
  }
  // t counts tiles with tiles_n column tiles to each row tile. Returns the
  // group, its rows, and the tile's index within the group.
  __device__ static inline int find(const LayerArgs& p, int t, int tiles_n, int lane, int& first,
                                    int& count, int& in) {
    unsigned base = 0;
    for (int g0 = 0; g0 < p.G; g0 += 64) {
      int f, c;
      const unsigned n = tiles_of(p, g0 + lane, f, c);
      const unsigned incl = wave_scan(n, lane);
      const unsigned chunk = __builtin_amdgcn_readlane(incl, 63);
      // The first lane whose inclusive count lies past the tile, if one does (sums
      // that have wrapped may say otherwise). Lanes past the last group count what
      // the last group's lane does, so it is a group's lane.
      uint64_t past = 0;
      if (t < (int)((base + chunk) * (unsigned)tiles_n))
        past = __ballot((int64_t)(int)(base + incl) * tiles_n > t);
      if (past) {
        const int src = __builtin_ctzll(past);
        first = __builtin_amdgcn_readlane(f, src);
        count = __builtin_amdgcn_readlane(c, src);
        const unsigned before = base + (unsigned)__builtin_amdgcn_readlane(incl - n, src);
        in = (int)((unsigned)t - before * (unsigned)tiles_n);
        return g0 + src;
      }
      base += chunk;
    }
    first = count = in = 0;
    return 0;
  }
};

// Tiles of the whole call (an exact count, uniform).
template <int MODE, int BM>
__device__ inline int layer_tiles(const LayerArgs& p, int lane) {
  if constexpr (MODE == LAYER_ROWS) return (int)(LayerRows<BM>::total(p, lane) * (unsigned)p.tiles_n);
  return p.tiles_m * p.tiles_n * (MODE == LAYER_SUM ? p.G : 1);
}

// Tile t (in the order that puts tiles sharing operand panels on one XCD) of
// `total`. Consecutive tiles belong to one group, walked in grouped order.
// The mode is fixed at compile time: with a branch on it at run time this
// compiler left the pointers that the third branch does not change (bias, Z)
// undefined there.
template <int MODE, int BM, int BN>
__device__ inline LayerTile layer_tile(const LayerArgs& p, int t, int total, int lane) {
  LayerTile q;
  const int lid = xcd_remap(t, total);
  const int osz = p.out32 ? 4 : 2;
  int tm, tn;
  q.M = p.M;
  q.N = p.N;
  q.K = p.K;
  q.A = static_cast<const char*>(p.A);
  q.B = static_cast<const char*>(p.B);
  q.bias = static_cast<const char*>(p.bias);
  q.R = static_cast<const char*>(p.R);
  q.Y = static_cast<char*>(p.Y);
  q.Z = static_cast<char*>(p.Z);
  if constexpr (MODE == LAYER_DENSE) {
    grouped_tile(lid, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
  } else if constexpr (MODE == LAYER_ROWS) {
    int first, count, in;
    const int g = LayerRows<BM>::find(p, lid, p.tiles_n, lane, first, count, in);
    // Whatever the offsets hold, the tile lies inside the group, or the group has
    // no rows: every access is masked by its rows.
    int tiles_m = (count + BM - 1) / BM;
    if (in < 0 || in >= (int64_t)tiles_m * p.tiles_n) {
      in = count = 0;
      tiles_m = 1;
    }
    grouped_tile(in, tiles_m, p.tiles_n, p.group_m, tm, tn);
    q.M = count;
    q.A += (int64_t)first * p.lda * 2;
    q.B += (int64_t)g * p.stride_b * 2;
    if (q.bias) q.bias += (int64_t)g * p.N * 2;
    if (q.R) q.R += (int64_t)first * p.ldr * osz;
    q.Y += (int64_t)first * p.ldy * osz;
    if (q.Z) q.Z += (int64_t)first * p.ldz * 2;
  } else {
    const int per = p.tiles_m * p.tiles_n;
    const int g = lid / per;
    grouped_tile(lid - g * per, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
    int first, count;
    layer_group(p.offsets, g, p.K, first, count);
    first = __builtin_amdgcn_readfirstlane(first);
    q.K = __builtin_amdgcn_readfirstlane(count);
    q.A += (int64_t)first * p.lda * 2;
    q.B += (int64_t)first * p.ldb * 2;
    q.bias = nullptr;
    q.Z = nullptr;
    if (q.R) q.R += (int64_t)g * p.stride_y * osz;
    q.Y += (int64_t)g * p.stride_y * osz;
  }
  q.m0 = tm * BM;
  q.n0 = tn * BN;
  return q;
}

// -------------------------------------------------------------- 16-bit types --
__device__ __forceinline__ float layer_f32(TagF16, unsigned short u) {
  return (float)__builtin_bit_cast(_Float16, u);
}
__device__ __forceinline__ float layer_f32(TagBF16, unsigned short u) {
  return __builtin_bit_cast(float, (unsigned)u << 16);
}
// To nearest, ties to even (the hardware conversions round so).
__device__ __forceinline__ unsigned short layer_16(TagF16, float x) {
  return __builtin_bit_cast(unsigned short, (_Float16)x);
}
__device__ __forceinline__ unsigned short layer_16(TagBF16, float x) {
  return __builtin_bit_cast(unsigned short, (__bf16)x);
}
template <class Tag>
__device__ __forceinline__ void layer_unpack8(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    f[2 * d] = layer_f32(Tag{}, (unsigned short)(v[d] & 0xFFFFu));
    f[2 * d + 1] = layer_f32(Tag{}, (unsigned short)(v[d] >> 16));
  }
}
// Two at a time: one instruction for bf16.
typedef float layer_f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 layer_bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 layer_f16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ unsigned layer_pack2(TagF16, float lo, float hi) {
  return __builtin_bit_cast(unsigned, __builtin_convertvector(layer_f32x2{lo, hi}, layer_f16x2));
}
__device__ __forceinline__ unsigned layer_pack2(TagBF16, float lo, float hi) {
  return __builtin_bit_cast(unsigned, __builtin_convertvector(layer_f32x2{lo, hi}, layer_bf16x2));
}
template <class Tag>
__device__ __forceinline__ u32x4 layer_pack8(const float (&f)[8]) {
  u32x4 v;
#pragma unroll
  for (int d = 0; d < 4; ++d) v[d] = layer_pack2(Tag{}, f[2 * d], f[2 * d + 1]);
  return v;
}

// --------------------------------------------------------------- activations --
// 1 / (1 + 2^u), the logistic function of -u ln 2: 2^u overflows to infinity and
// the reciprocal of that is 0, so both ends come out right without a branch.
__device__ __forceinline__ float layer_logistic2(float u) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u));
}
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float layer_sigmoid(float v) { return layer_logistic2(-kLog2e * v); }
constexpr float kGeluA = 1.5957691216057308f;       // 2 sqrt(2 / pi)
constexpr float kGeluB = 0.044715f;

// The normal distribution's function Phi(z) and exp(-z^2 / 2). With x = |z| /
// sqrt(2) and t = 1 / (1 + x / 2), erfc(x) exp(x^2) / t is smooth on t in (0, 1]: a
// polynomial of degree 8 fitted to it for x up to 9.4 by least squares weighted
// toward the largest relative error, 7.4e-8 with these coefficients in exact
// arithmetic. The exponent z^2 / 2 log2(e) is held in two floats, so that the
// exponential keeps its relative accuracy far out: Phi of a negative z is not a
// difference. In float32 Phi is within 4e-7, relative, from -13 on (least
// accurate near -1.6) where the reciprocal and the exponential are rounded
// correctly; the hardware's add their last bit each. (The library's erfc:
// 4096x4096x1024 48 us, 42 so, 32 without an activation.)
struct LayerNormal {
  float phi, e;
};
__device__ __forceinline__ LayerNormal layer_normal(float z) {
  const float c = __builtin_amdgcn_fmed3f(z, -16.0f, 16.0f);  // both are 0 or 1 past that
  constexpr float kHi = 0.7213475108146667f, kLo = 9.629815e-09f;  // log2(e) / 2
  const float h = c * kHi, hl = __builtin_fmaf(c, kLo, __builtin_fmaf(c, kHi, -h));
  const float hi = h * c, lo = __builtin_fmaf(hl, c, __builtin_fmaf(h, c, -hi));
  const float e0 = __builtin_amdgcn_exp2f(-hi);
  const float e = __builtin_fmaf(-0.6931471805599453f * lo, e0, e0);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(__builtin_fabsf(c), 0.3535533905932738f, 1.0f));
  float g = -0.0588473342359066f;
  g = __builtin_fmaf(g, t, 0.2834887206554413f);
  g = __builtin_fmaf(g, t, -0.4849390983581543f);
  g = __builtin_fmaf(g, t, 0.2754654288291931f);
  g = __builtin_fmaf(g, t, -0.024821195751428604f);
  g = __builtin_fmaf(g, t, 0.201917365193367f);
  g = __builtin_fmaf(g, t, 0.24330003559589386f);
  g = __builtin_fmaf(g, t, 0.28234803676605225f);
  g = __builtin_fmaf(g, t, 0.2820879817008972f);
  const float q = 0.5f * t * g * e;  // Phi(-|z|)
  return {c < 0.0f ? q : 1.0f - q, e};
}

// GELU's tanh form, z (1 + tanh(u)) / 2, is z * sigmoid(2 u): no difference
// of nearly equal numbers for negative z.
template <int ACT>
__device__ __forceinline__ float layer_act(float z) {
  if constexpr (ACT == ACT_RELU) return z > 0.0f || z != z ? z : 0.0f;
  if constexpr (ACT == ACT_GELU) {
    const float w = __builtin_fmaf(z * z, -kLog2e * kGeluA * kGeluB, -kLog2e * kGeluA);
    return z * layer_logistic2(z * w);
  }
  if constexpr (ACT == ACT_GELU_ERF) return z * layer_normal(z).phi;
  if constexpr (ACT == ACT_SILU) return z * layer_sigmoid(z);
  return z;
}
// act'(z). Past |z| = 16 GELU's slope is 0 or 1 to float32; the cubic there
// would give infinity times zero.
template <int ACT>
__device__ __forceinline__ float layer_slope(float z) {
  if constexpr (ACT == ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
  if constexpr (ACT == ACT_GELU) {
    const float c = z > 16.0f ? 16.0f : (z < -16.0f ? -16.0f : z);
    const float s = layer_sigmoid(kGeluA * (c + kGeluB * c * c * c));
    return s + c * s * (1.0f - s) * kGeluA * (1.0f + 3.0f * kGeluB * c * c);
  }
  if constexpr (ACT == ACT_GELU_ERF) {
    const LayerNormal n = layer_normal(z);
    const float c = z > 16.0f ? 16.0f : (z < -16.0f ? -16.0f : z);
    return __builtin_fmaf(c * 0.3989422804014327f, n.e, n.phi);
  }
  if constexpr (ACT == ACT_SILU) {
    const float s = layer_sigmoid(z);
    return s * (1.0f + z * (1.0f - s));
  }
  return 1.0f;
}
template <int ACT>
__device__ __forceinline__ void layer_act8_of(float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = layer_act<ACT>(f[e]);
}
__device__ __forceinline__ void layer_scale8(float (&f)[8], float by) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] *= by;
}
__device__ __forceinline__ void layer_act8(float (&f)[8], const LayerArgs& p) {
  switch (p.act) {  // uniform over the launch
    case ACT_RELU: layer_act8_of<ACT_RELU>(f); break;
    case ACT_GELU: layer_act8_of<ACT_GELU>(f); break;
    case ACT_GELU_ERF: layer_act8_of<ACT_GELU_ERF>(f); break;
    case ACT_SILU: layer_act8_of<ACT_SILU>(f); break;
    case ACT_SCALE: layer_scale8(f, *p.scale); break;
    default: break;
  }
}

// ------------------------------------------------------------------ epilogue --
// Row-wise accesses of up to 8 columns of a 16-bit or float32 matrix; nv of
// the 8 lie inside it. Whole pieces go 16 bytes at a time at whatever address
// they have, which this target's memory unit serves: 4096 x 4096 activation
// gradients at an odd pitch 73 us element by element, 31 so; a product of
// 8192x2047x1024 with bias and GELU 58, 42 so.
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
typedef u32x2 u32x2_at2 __attribute__((aligned(2)));
typedef unsigned u32_at2 __attribute__((aligned(2)));
template <class Tag>
__device__ __forceinline__ void layer_load8_16(const char* p, int nv, float (&f)[8]) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (nv == 8) {
    v = *reinterpret_cast<const u32x4_at2*>(p);
  } else {  // 4, 2 and 1 columns: shorter code than one after the other
    u32x2 four = {0u, 0u};
    unsigned two = 0u, one = 0u;
    if (nv & 4) four = *reinterpret_cast<const u32x2_at2*>(p);
    if (nv & 2) two = *reinterpret_cast<const u32_at2*>(p + (nv & 4) * 2);
    if (nv & 1) one = *reinterpret_cast<const unsigned short*>(p + (nv & 6) * 2);
    const unsigned x = nv & 2 ? two : one, y = nv & 2 ? one : 0u;
    v.x = nv & 4 ? four.x : x;
    v.y = nv & 4 ? four.y : y;
    v.z = nv & 4 ? x : 0u;
    v.w = nv & 4 ? y : 0u;
  }
  layer_unpack8<Tag>(v, f);
}
template <class Tag>
__device__ __forceinline__ void layer_store8_16(char* p, int nv, const float (&f)[8]) {
  const u32x4 v = layer_pack8<Tag>(f);
  if (nv == 8) {
    *reinterpret_cast<u32x4_at2*>(p) = v;
  } else {
    const unsigned x = nv & 4 ? v.z : v.x, y = nv & 4 ? v.w : v.y;
    if (nv & 4) *reinterpret_cast<u32x2_at2*>(p) = u32x2{v.x, v.y};
    if (nv & 2) *reinterpret_cast<u32_at2*>(p + (nv & 4) * 2) = x;
    if (nv & 1) *reinterpret_cast<unsigned short*>(p + (nv & 6) * 2) = (unsigned short)(nv & 2 ? y : x);
  }
}
__device__ __forceinline__ void layer_load8_32(const char* p, int nv, float (&f)[8]) {
  const float* s = reinterpret_cast<const float*>(p);
  if (nv == 8) {
    const u32x4_at4* v = reinterpret_cast<const u32x4_at4*>(p);
    const f32x4 lo = __builtin_bit_cast(f32x4, u32x4(v[0])), hi = __builtin_bit_cast(f32x4, u32x4(v[1]));
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = lo[e], f[e + 4] = hi[e];
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = e < nv ? s[e] : 0.0f;
  }
}
__device__ __forceinline__ void layer_store8_32(char* p, int nv, const float (&f)[8]) {
  float* s = reinterpret_cast<float*>(p);
  if (nv == 8) {
    u32x4_at4* v = reinterpret_cast<u32x4_at4*>(p);
    v[0] = __builtin_bit_cast(u32x4, f32x4{f[0], f[1], f[2], f[3]});
    v[1] = __builtin_bit_cast(u32x4, f32x4{f[4], f[5], f[6], f[7]});
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < nv) s[e] = f[e];
  }
}

// Z, activation, residual and Y of 8 columns of one row, from the sums x.
template <class Tag>
__device__ __forceinline__ void layer_finish8(const LayerArgs& p, const LayerTile& q, int r, int c,
                                              int nv, const float (&bias)[8], float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] += bias[e];
  if (q.Z) layer_store8_16<Tag>(q.Z + ((int64_t)r * p.ldz + c) * 2, nv, x);
  layer_act8(x, p);
  if (q.R) {
    float rv[8];
    if (p.out32) layer_load8_32(q.R + ((int64_t)r * p.ldr + c) * 4, nv, rv);
    else layer_load8_16<Tag>(q.R + ((int64_t)r * p.ldr + c) * 2, nv, rv);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] += rv[e];
  }
  if (p.out32) layer_store8_32(q.Y + ((int64_t)r * p.ldy + c) * 4, nv, x);
  else layer_store8_16<Tag>(q.Y + ((int64_t)r * p.ldy + c) * 2, nv, x);
}

// The epilogue of one wave's TM x TN atoms, whose first output is (r0, c0).
// The accumulators of a 16- or 32-wide atom hold 4 rows of one column per
// lane; batches of up to 64 rows go through LDS so that each lane gets 8
// consecutive columns of one row, and a wave's stores of 16-bit outputs are 16
// bytes a lane, whole 128-byte lines where the wave is 64 columns wide. lds: this
// wave's own layer_lds_bytes<C>(); no other wave touches it.
//
// The rows of a batch are finished in a loop that is not unrolled past four
// passes: with all of it unrolled, the epilogue outgrew the instruction cache
// (32768x4096x2048 on 256x256 tiles 419 us, 395 so; with a residual 531 and
// 450).
template <class C>
struct LayerEpi {
  using At = typename C::At;
  static constexpr int W = C::TN * At::N, P = W + 4;  // columns; pitch in floats, 4 apart in banks
  static constexpr int ROWS = C::TM * At::M;
  static constexpr int BATCH = ROWS < 64 ? ROWS : 64;     // rows
  static constexpr int LPR = W / 8, RPP = 64 / LPR;       // lanes a row, rows a pass
  static constexpr int PASSES = BATCH / RPP;
  static constexpr int GROUP = PASSES < 4 ? PASSES : 4;   // passes unrolled
  static_assert(W % 8 == 0 && 64 % LPR == 0 && BATCH % RPP == 0 && PASSES % GROUP == 0 &&
                    ROWS % BATCH == 0 && BATCH % At::M == 0,
                "whole passes");
};
template <class C>
constexpr int layer_lds_bytes() { return LayerEpi<C>::BATCH * LayerEpi<C>::P * 4; }

// LDS written by some lanes of a wave is read by others: LDS operations of one
// wave complete in order, so only the compiler has to keep theirs.
__device__ __forceinline__ void layer_wave_order() {
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
}

// The residual of one group of passes, as it is stored (16-bit: lo alone).
template <int GROUP>
struct LayerGroupR {
  u32x4 lo[GROUP], hi[GROUP];
};
// Requests it for the passes whose first row is r (RPP rows a pass).
template <int GROUP, int RPP>
__device__ __forceinline__ void layer_group_r(LayerGroupR<GROUP>& v, const LayerArgs& p,
                                              const LayerTile& q, int r, int c) {
  if (!q.R || c >= q.N) return;
  const int osz = p.out32 ? 4 : 2;
  const int64_t step = RPP * p.ldr * osz;
  const char* at = q.R + ((int64_t)r * p.ldr + c) * osz;
#pragma unroll
  for (int s = 0; s < GROUP; ++s, at += step) {
    if (r + s * RPP >= q.M) continue;
    v.lo[s] = *reinterpret_cast<const u32x4_at2*>(at);
    if (p.out32) v.hi[s] = *reinterpret_cast<const u32x4_at4*>(at + 16);
  }
}
// The passes of a batch whose first row is r, all of its columns in whole
// 16-byte pieces: lds is this lane's first piece, c its first column. The
// residual is requested a group of passes ahead. (R may be Y: a lane reads each
// of its pieces before it writes it.)
template <class E, class Tag, int ACT>
__device__ __forceinline__ void layer_passes(const LayerArgs& p, const LayerTile& q, int r, int c,
                                             const float* lds, const float (&bias)[8],
                                             LayerGroupR<E::GROUP>& res, float scale) {
  const int osz = p.out32 ? 4 : 2;
  const int64_t ystep = E::RPP * p.ldy * osz, zstep = E::RPP * p.ldz * 2;
  char* y = q.Y + ((int64_t)r * p.ldy + c) * osz;
  char* z = q.Z + ((int64_t)r * p.ldz + c) * 2;
#pragma unroll 1
  for (int g = 0; g < E::PASSES; g += E::GROUP) {
    LayerGroupR<E::GROUP> next;
    if (g + E::GROUP < E::PASSES)
      layer_group_r<E::GROUP, E::RPP>(next, p, q, r + (g + E::GROUP) * E::RPP, c);
#pragma unroll
    for (int s = 0; s < E::GROUP; ++s) {
      const int row = r + (g + s) * E::RPP;
      const float* const from = lds + (g + s) * E::RPP * E::P;
      const f32x4 lo = *reinterpret_cast<const f32x4*>(from);
      const f32x4 hi = *reinterpret_cast<const f32x4*>(from + 4);
      float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] += bias[e];
      if (row < q.M && c < q.N) {
        if (q.Z) *reinterpret_cast<u32x4_at2*>(z) = layer_pack8<Tag>(x);
        if constexpr (ACT == ACT_SCALE) layer_scale8(x, scale);
        else layer_act8_of<ACT>(x);
        if (q.R) {
          float f[8];
          if (p.out32) {
            const f32x4 a = __builtin_bit_cast(f32x4, res.lo[s]), b = __builtin_bit_cast(f32x4, res.hi[s]);
#pragma unroll
            for (int e = 0; e < 4; ++e) f[e] = a[e], f[e + 4] = b[e];
          } else {
            layer_unpack8<Tag>(res.lo[s], f);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] += f[e];
        }
        if (p.out32) layer_store8_32(y, 8, x);
        else *reinterpret_cast<u32x4_at2*>(y) = layer_pack8<Tag>(x);
      }
      y += ystep;
      z += zstep;
    }
    res = next;
  }
}

template <class C, class Tag>
__device__ __forceinline__ void layer_store(typename C::At::acc_t (&acc)[C::TM][C::TN],
                                            const LayerArgs& p, const LayerTile& q, int r0, int c0,
                                            int lane, float* lds) {
  using At = typename C::At;
  using E = LayerEpi<C>;
  constexpr int P = E::P, AR = E::BATCH / At::M;  // atom rows of a batch
  const int cl = 8 * (lane % E::LPR), rl = lane / E::LPR;
  const int c = c0 + cl, nv = q.N - c >= 8 ? 8 : q.N - c;
  float bias[8], scale = 1.0f;
  if (p.act == ACT_SCALE) scale = *p.scale;  // (uniform; read for every row it cost 3 us a 256 x 256 tile)
#pragma unroll
  for (int e = 0; e < 8; ++e) bias[e] = 0.0f;
  if (q.bias && nv > 0) {
    if (p.whole8) layer_unpack8<Tag>(*reinterpret_cast<const u32x4_at2*>(q.bias + (int64_t)c * 2), bias);
    else layer_load8_16<Tag>(q.bias + (int64_t)c * 2, nv, bias);
  }
#pragma unroll
  for (int b = 0; b < C::TM / AR; ++b) {
    const int r = r0 + b * E::BATCH;  // (uniform) the batch's first row
    if (r >= q.M) break;
    LayerGroupR<E::GROUP> res;
    if (p.whole8) layer_group_r<E::GROUP, E::RPP>(res, p, q, r + rl, c);
#pragma unroll
    for (int i = 0; i < AR; ++i)
#pragma unroll
      for (int j = 0; j < C::TN; ++j)
#pragma unroll
        for (int v = 0; v < At::NACC; ++v)
          lds[(i * At::M + At::acc_row(lane, v)) * P + j * At::N + At::acc_col(lane)] =
              acc[b * AR + i][j][v];
    layer_wave_order();
    const float* const from = lds + rl * P + cl;
    if (p.whole8) {
      switch (p.act) {
        case ACT_RELU: layer_passes<E, Tag, ACT_RELU>(p, q, r + rl, c, from, bias, res, scale); break;
        case ACT_GELU: layer_passes<E, Tag, ACT_GELU>(p, q, r + rl, c, from, bias, res, scale); break;
        case ACT_GELU_ERF: layer_passes<E, Tag, ACT_GELU_ERF>(p, q, r + rl, c, from, bias, res, scale); break;
        case ACT_SILU: layer_passes<E, Tag, ACT_SILU>(p, q, r + rl, c, from, bias, res, scale); break;
        case ACT_SCALE: layer_passes<E, Tag, ACT_SCALE>(p, q, r + rl, c, from, bias, res, scale); break;
        default: layer_passes<E, Tag, ACT_NONE>(p, q, r + rl, c, from, bias, res, scale); break;
      }
    } else {
#pragma unroll 1
      for (int s = 0; s < E::PASSES; ++s) {
        const int row = r + s * E::RPP + rl;
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = from[s * E::RPP * P + e];
        if (row < q.M && nv > 0) layer_finish8<Tag>(p, q, row, c, nv, bias, x);
      }
    }
    layer_wave_order();
  }
}

// ----------------------------------------------------------------- launchers --
// Every product kernel is instantiated for the modes and layouts that the
// entry points reach: dense calls in four layouts, by rows with A stored
// [M][K], by sum with both operands stored along the sum. f(mode, ta, tb) gets
// them as integral constants.
template <int V>
struct LayerConst {
  static constexpr int value = V;
};
template <class F>
hipError_t layer_for_layout(const LayerArgs& a, bool ta, bool tb, F f) {
  if (a.mode == LAYER_SUM) return f(LayerConst<LAYER_SUM>{}, LayerConst<1>{}, LayerConst<0>{});
  if (a.mode == LAYER_ROWS)
    return tb ? f(LayerConst<LAYER_ROWS>{}, LayerConst<0>{}, LayerConst<1>{})
              : f(LayerConst<LAYER_ROWS>{}, LayerConst<0>{}, LayerConst<0>{});
  if (!ta)
    return tb ? f(LayerConst<LAYER_DENSE>{}, LayerConst<0>{}, LayerConst<1>{})
              : f(LayerConst<LAYER_DENSE>{}, LayerConst<0>{}, LayerConst<0>{});
  return tb ? f(LayerConst<LAYER_DENSE>{}, LayerConst<1>{}, LayerConst<1>{})
            : f(LayerConst<LAYER_DENSE>{}, LayerConst<1>{}, LayerConst<0>{});
}

// The kernels of the products, each next to its definition. dtype: 0 f16, 1
// bf16. They return the HIP status of the launch.
// tile: 0 128x128, 1 64x64, 2 64x64 with the sum split over four wave groups.
hipError_t launch_layer_general(int dtype, bool ta, bool tb, int tile, const LayerArgs& a,
                                int ntiles, hipStream_t s);
// Operands in whole 16-byte pieces (layer_direct in layer_api.hip). deep: ten
// half-slots of LDS instead of five.
hipError_t launch_layer_pp256(int dtype, bool ta, bool tb, const LayerArgs& a, int ntiles,
                              hipStream_t s);
hipError_t launch_layer_pp128(int dtype, bool ta, bool tb, bool deep, const LayerArgs& a,
                              int ntiles, hipStream_t s);
// Operands not stored along K at any 2-byte alignment, the others in whole 16-byte
// pieces.
hipError_t launch_layer_ring(int dtype, bool ta, bool tb, const LayerArgs& a, int ntiles,
                             hipStream_t s);
// 16 mt x 32 (16 nt) outputs a workgroup. The first: A stored [M][K], B stored
// [N][K], by rows and mt = 1, or (any) dense and by rows at any alignment.
hipError_t launch_layer_skinny(int dtype, bool any, int mt, const LayerArgs& a, int ntiles,
                               hipStream_t s);
hipError_t launch_layer_split(int dtype, bool ta, bool tb, int mt, int nt, const LayerArgs& a, int ntiles,
                              hipStream_t s);

}  // namespace dgt
