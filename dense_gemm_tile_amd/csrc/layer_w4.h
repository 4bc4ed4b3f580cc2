// Products with 4-bit weights: Y = act(A @ W^T + bias) + R, where
//   W[n][k] = s[n][j] (code[n][k] - z[n][j]),  j = k / group.
//
// The matrix cores take 16-bit operands, and a code becomes one without an
// arithmetic operation: its four bits, placed below the leading bit of 16.0, are the
// number 16 + code, exactly, in both types. So for every group
//   sum over k of A[m][k] (code - z) = P - (16 + z) S,  P = sum A (16 + code),  S = sum A,
// P and S from matrix instructions (S against ones), the rest in float32: no weight
// is rounded to 16 bits. 16 and not the type's larger powers of two, since P and
// (16 + z) S cancel by that factor.
//
// A pair of codes k and k + 4 of a 32-bit word goes to one register with one shift
// and one and-or; A's values are brought into that order instead.
#pragma once

#include "layer_split.h"

namespace dgt {

// What a call carries.
struct W4Args {
  LayerArgs a;  // B: codes; ldb, stride_b: bytes
  const void* scales;
  const void* zeros;   // null: 8
  int64_t lds, stride_s;
  int group;
};

// Groups of K values that a call may have: 16 columns of scales and zero points, in LDS beside the
// slices of 8 waves.
constexpr int kW4MaxRuns = 1536;

// The tile that a call took, and whether one launch does not hold so many of it.
struct W4Form {
  int waves, rows, columns;
  bool whole, many;
};

// The launches, a file for each type.
hipError_t launch_w4_f16(const W4Args& p, hipStream_t s, W4Form& form);
hipError_t launch_w4_bf16(const W4Args& p, hipStream_t s, W4Form& form);

namespace {

typedef u32x4 u32x4_at1 __attribute__((aligned(1)));
typedef unsigned u32_at1 __attribute__((aligned(1)));

template <class Tag>
struct W4Type;
template <>
struct W4Type<TagBF16> {
  static constexpr unsigned BASE = 0x41804180u, MASK = 0x00780078u, ONES = 0x3F803F80u;
  static constexpr int AT = 3;  // the place of a code's lowest bit
};
template <>
struct W4Type<TagF16> {
  static constexpr unsigned BASE = 0x4C004C00u, MASK = 0x03C003C0u, ONES = 0x3C003C00u;
  static constexpr int AT = 6;
};

// Eight codes as the 16-bit numbers 16 + code, in the order 0 4 1 5 2 6 3 7.
template <class Tag>
__device__ __forceinline__ u32x4 w4_codes(unsigned q) {
  using T = W4Type<Tag>;
  // (Both constants in registers: one instruction takes no two literals.)
  unsigned mask = T::MASK, base = T::BASE;
  asm("" : "+s"(mask));
  asm("" : "+v"(base));
  u32x4 v;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int right = 4 * j - T::AT;
    v[j] = ((right > 0 ? q >> (right > 0 ? right : 0) : q << (right > 0 ? 0 : -right)) & mask) | base;
  }
  return v;
}
// Eight 16-bit values in that order.
__device__ __forceinline__ u32x4 w4_order(u32x4 x) {
  return u32x4{__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
               __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
}

// A workgroup's tile: its group's rows, weights and outputs. g: the group.
template <int MODE, int BM, int BN>
__device__ __forceinline__ LayerTile w4_tile(const LayerArgs& p, int t, int total, int lane, int& g) {
  LayerTile q;
  const int osz = p.out32 ? 4 : 2, lid = xcd_remap(t, total);
  int tm, tn, first = 0, count = p.M, tiles_m = p.tiles_m, in = lid;
  g = 0;
  if constexpr (MODE == LAYER_ROWS) {
    g = LayerRows<BM>::find(p, lid, p.tiles_n, lane, first, count, in);
    tiles_m = (count + BM - 1) / BM;
    if (in < 0 || in >= (int64_t)tiles_m * p.tiles_n) {  // whatever the offsets hold
      in = count = 0;
      tiles_m = 1;
    }
  }
  grouped_tile(in, tiles_m, p.tiles_n, p.group_m, tm, tn);
  q.A = static_cast<const char*>(p.A) + (int64_t)first * p.lda * 2;
  q.B = static_cast<const char*>(p.B) + (int64_t)g * p.stride_b;
  q.bias = static_cast<const char*>(p.bias);
  if (q.bias) q.bias += (int64_t)g * p.N * 2;
  q.R = static_cast<const char*>(p.R);
  if (q.R) q.R += (int64_t)first * p.ldr * osz;
  q.Y = static_cast<char*>(p.Y) + (int64_t)first * p.ldy * osz;
  q.Z = nullptr;
  q.M = count;
  q.N = p.N;
  q.K = p.K;
  q.m0 = tm * BM;
  q.n0 = tn * BN;
  return q;
}

// Eight values of a row from element k on, zeros past K.
__device__ __forceinline__ u32x4 w4_values(const char* row, int k, int K) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (k + 8 <= K) return *reinterpret_cast<const u32x4_at2*>(row + (int64_t)k * 2);
  if (k >= K) return v;
#pragma unroll
  for (int e = 0; e < 7; ++e)
    if (k + e < K) v[e / 2] |= (unsigned)*reinterpret_cast<const unsigned short*>(row + (int64_t)(k + e) * 2) << (16 * (e % 2));
  return v;
}
// Eight codes of a row from code k (a multiple of 8) on, any value past K.
__device__ __forceinline__ unsigned w4_word(const char* row, int k, int K) {
  if (k + 8 <= K) return *reinterpret_cast<const u32_at1*>(row + k / 2);
  unsigned q = 0;
  if (k >= K) return q;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (k + 2 * e < K) q |= (unsigned)(unsigned char)row[k / 2 + e] << (8 * e);
  return q;
}

// As layer_split.hip does for 16-bit weights: each wave takes slices of 128 K values, every
// KW-th, and loads them straight into LDS of its own, without a barrier; consecutive
// lanes load consecutive bytes. A is the bulk of a slice where there are many rows, so it
// comes in two halves, each asked for again as soon as it has been read; codes and
// scales come a slice ahead of that. (Whole slices of both, two at a time, leave LDS for
// four waves instead of eight: 48x8192x8192 25 us, 19 so.)
//
// A tile has 8 AL rows. In LDS: a half of A as SplitAlong has it; of the codes 16 rows of
// 64 bytes to a KiB, chunk c (32 codes) of row r at chunk c ^ (r >> 2 & 3), so that the
// 4 bytes that each lane reads for 32 K values lie in banks of their own. Rows of A
// past the tile hold anything: they reach only outputs that are not stored.
//
// WHOLE: operands in whole 16-byte pieces. Others, at any pitch and alignment, go through
// registers to the same places in LDS: consecutive lanes still load consecutive bytes, 16 a
// lane wherever they lie, and the last slice's ends element by element. (Fragments
// straight from memory, whose neighbouring lanes lie in different rows, take the address
// units four times as long: 257x1000x1032 16 us, 10 so.)
//
// GRP: K values between which the sums are scaled: 128 or 64 where the group is a multiple of
// it, else 32.

// The scales of a workgroup's columns lie in LDS, in rows of w4_pitch(): loaded where
// they are used they cost as many requests as the codes do (64 experts of 2 rows,
// 2048x2048, groups of 32: 47 us, 41 so).

// Bytes of a column's scales in LDS: whole slices, and an odd number of 8 bytes, so that 16
// columns lie in banks of their own.
__host__ __device__ inline int w4_pitch(int K, int group) {
  const int64_t runs = ((int64_t)(K + 127) / 128 * 128 + group - 1) / group;
  return (int)((runs * 2 + 7) / 8 * 8 | 8);
}
// A wave's part of the slices, and a workgroup's LDS beside the scales. (Rows past the
// tile are read; the waves' sums overlay the slices.)
template <int AL, int NT>
constexpr int w4_wave_lds() { return 2 * AL * 1024 + 2 * NT * 1024; }
template <int AL, int NT, int KW>
constexpr int w4_lds() {
  constexpr int MT = (AL + 1) / 2, USED = KW * w4_wave_lds<AL, NT>() + (2 * MT - AL) * 1024;
  return USED > SplitSum<MT, NT, KW>::LDS_BYTES ? USED : SplitSum<MT, NT, KW>::LDS_BYTES;
}

template <class Tag, int MODE, int AL, int NT, int GRP, bool ZEROS, int KW, bool WHOLE>
__global__ void __launch_bounds__(KW * 64, 2) layer_w4_split_kernel(const W4Args p) {
  using At = SplitAtom;
  constexpr int MT = (AL + 1) / 2, BM = 8 * AL;
  using Sum = SplitSum<MT, NT, KW>;
  using SA = SplitAlong<MT, AL>;
  constexpr int A_HALF = AL * 1024, B_SLICE = NT * 1024, WAVE = w4_wave_lds<AL, NT>();
  constexpr int S = 128 / GRP;  // scales of a column in a slice
  static_assert(w4_lds<AL, NT, KW>() <= 160 * 1024, "gfx950 has 160 KiB of LDS per workgroup");
  __shared__ __attribute__((aligned(1024))) char smem[w4_lds<AL, NT, KW>()];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int total = layer_tiles<MODE, BM>(p.a, lane);
  if ((int)blockIdx.x >= total) return;  // by rows the grid is an upper bound
  int g;
  LayerTile q = w4_tile<MODE, BM, Sum::BN>(p.a, blockIdx.x, total, lane, g);
  if (q.M <= q.m0) return;               // (uniform) no rows, as offsets that decrease can make a tile
  if (q.M > q.m0 + BM) q.M = q.m0 + BM;  // this tile's rows
  const int r16 = lane & 15, oct = lane >> 4;

  const char* const Ab = q.A + (int64_t)q.m0 * p.a.lda * 2;
  const auto ra = make_rsrc_n(Ab, split_records(q.M - q.m0, p.a.lda, q.K));
  const char* const Bb = q.B + (int64_t)q.n0 * p.a.ldb;
  const int rows_b = q.N - q.n0 < Sum::BN ? q.N - q.n0 : Sum::BN;
  const auto rb = make_rsrc_n(Bb, WHOLE ? (unsigned)((rows_b - 1) * (int)p.a.ldb + q.K / 2) : 0u);
  At::acc_t acc[MT][NT], sx[MT], dot[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][n][v] = 0.0f;

  const int KT = (q.K + 127) / 128;
  const int start = split_start(q.n0 / Sum::BN, KT);
  const int NJ = KT > w ? (KT - w + KW - 1) / KW : 0;  // this wave's slices
  extern __shared__ __attribute__((aligned(16))) char scales[];
  const int pitch = w4_pitch(q.K, p.group);
  char* const mine = smem + w * WAVE;
  char* const codes = mine + 2 * A_HALF;
  // The slice that this wave takes j-th; KT, where every load is out of range, past its last.
  auto slice_of = [&](int j) {
    const int s = j * KW + w + start;
    return j >= NJ ? KT : s >= KT ? s - KT : s;
  };
  u32x4 ra_next[WHOLE ? 1 : 2][WHOLE ? 1 : AL], rb_next[WHOLE ? 1 : 2][WHOLE ? 1 : NT];  // (not WHOLE) on their way
  auto request_a = [&](int h, int j) __attribute__((always_inline)) {
    const int at = 2 * slice_of(j) + h;  // slice of 64
    if constexpr (WHOLE) {
      SA::request(ra, (int)(p.a.lda * 2), q.M - q.m0, q.K, at, mine + h * A_HALF, lane);
    } else if (at < 2 * KT) {
      auto from = [&](int i, int& k) {
        const int r = 8 * i + (lane >> 3), row = r < q.M - q.m0 ? r : q.M - q.m0 - 1;  // (a tile has a row)
        k = at * 64 + 8 * ((lane & 7) ^ SA::Op::swz(r));
        return Ab + (int64_t)row * p.a.lda * 2;
      };
      if ((int64_t)at * 64 + 64 <= q.K) {
#pragma unroll
        for (int i = 0; i < AL; ++i) {
          int k;
          const char* const row = from(i, k);
          ra_next[h][i] = *reinterpret_cast<const u32x4_at2*>(row + (int64_t)k * 2);
        }
      } else {
#pragma unroll
        for (int i = 0; i < AL; ++i) {
          int k;
          const char* const row = from(i, k);
          ra_next[h][i] = w4_values(row, k, q.K);
        }
      }
    }
  };
  auto request_b = [&](int d, int j) __attribute__((always_inline)) {
    const int slice = slice_of(j);
    const bool whole = (int64_t)slice * 128 + 128 <= q.K;
    if (!WHOLE && slice >= KT) return;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = 16 * n + (lane >> 2), k = 128 * slice + 32 * ((lane & 3) ^ (r >> 2 & 3));
      if constexpr (WHOLE) {
        const int off = r < rows_b && k < q.K ? r * (int)p.a.ldb + k / 2 : kOutOfRange;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (pp_lds_ptr_t)(codes + d * B_SLICE + n * 1024), 16, off, 0, 0, 0);
      } else {
        const char* const from = Bb + (int64_t)(r < rows_b ? r : rows_b - 1) * p.a.ldb;
        if (whole) {
          rb_next[d][n] = *reinterpret_cast<const u32x4_at1*>(from + k / 2);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) rb_next[d][n][e] = w4_word(from, k + 8 * e, q.K);
        }
      }
    }
  };
  const u32x4 ones = {W4Type<Tag>::ONES, W4Type<Tag>::ONES, W4Type<Tag>::ONES, W4Type<Tag>::ONES};
  const At::acc_t none = {0.0f, 0.0f, 0.0f, 0.0f};
  // Loads are asked for in the order A(j, 0) B(j + 1) A(j, 1) A(j + 1, 0) B(j + 2) ...: after
  // each half of A one of B and one half of A.
  auto landed = [&](int h, int d) __attribute__((always_inline)) {
    if constexpr (WHOLE) {
      layer_fixed_order();
      pp_wait_vm<AL + NT>();
      layer_fixed_order();
    } else {
#pragma unroll
      for (int i = 0; i < AL; ++i) *reinterpret_cast<u32x4*>(mine + h * A_HALF + i * 1024 + lane * 16) = ra_next[h][i];
      if (h == 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
          *reinterpret_cast<u32x4*>(codes + d * B_SLICE + n * 1024 + lane * 16) = rb_next[d][n];
      }
      layer_wave_order();
    }
  };
  auto slice = [&](int d, int j) __attribute__((always_inline)) {
    const int at128 = slice_of(j);
    int run[S];  // of each scale of the slice
#pragma unroll
    for (int u = 0; u < S; ++u)
      run[u] = p.group == GRP ? S * at128 + u : (128 * at128 + GRP * u) / p.group;
    unsigned c[NT][4];
    float s[NT][S], z[NT][S];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      landed(h, d);
      u32x4 x[MT][2];
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < MT; ++i) x[i][m] = SA::read(mine + h * A_HALF, i, m, lane);
      if (h == 0) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int m = 0; m < 4; ++m)
            c[n][m] = *reinterpret_cast<const unsigned*>(codes + d * B_SLICE + n * 1024 + r16 * 64 +
                                                         ((m ^ (r16 >> 2)) << 4) + oct * 4);
#pragma unroll
          for (int u = 0; u < S; ++u) {
            const char* const at = scales + (16 * n + r16) * pitch + run[u] * 2;
            s[n][u] = layer_f32(Tag{}, *reinterpret_cast<const unsigned short*>(at));
            z[n][u] = ZEROS ? 16.0f + layer_f32(Tag{}, *reinterpret_cast<const unsigned short*>(at + Sum::BN * pitch)) : 24.0f;
          }
        }
      }
      if constexpr (WHOLE) pp_wait_lgkm0();  // read before the places are filled again
      layer_fixed_order();
      request_a(h, j + 1);
      if (h == 0) request_b(d, j + 2);
      layer_fixed_order();
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const int at = 2 * h + m, u = at * S / 4;  // 32 K values, and their scale
        const bool first = at * S % 4 == 0, last = (at + 1) * S % 4 == 0;
#pragma unroll
        for (int i = 0; i < MT; ++i) {
          x[i][m] = w4_order(x[i][m]);
          sx[i] = At::mma(Tag{}, x[i][m], ones, first ? none : sx[i]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const u32x4 v = w4_codes<Tag>(c[n][at]);
#pragma unroll
          for (int i = 0; i < MT; ++i) dot[i][n] = At::mma(Tag{}, x[i][m], v, first ? none : dot[i][n]);
        }
        if (last) {
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int v = 0; v < 4; ++v)
                acc[i][n][v] = __builtin_fmaf(s[n][u], __builtin_fmaf(-z[n][u], sx[i][v], dot[i][n][v]), acc[i][n][v]);
        }
      }
    }
  };
  // Columns of scales, then of zero points, in pieces of 8 runs: a thread's first piece is
  // asked for before the first slices. (Columns past N are left out: nothing of theirs is
  // stored.)
  const int runs = (q.K + p.group - 1) / p.group, per = (pitch + 15) / 16;
  const int pieces = per * Sum::BN * (ZEROS ? 2 : 1);
  auto piece = [&](int x) {
    const int row = x / per, r = x - row * per, col = row & (Sum::BN - 1);
    if (x >= pieces || col >= rows_b) return u32x4{0u, 0u, 0u, 0u};
    const void* const from = ZEROS && row >= Sum::BN ? p.zeros : p.scales;
    return w4_values(static_cast<const char*>(from) + ((int64_t)g * p.stride_s + (int64_t)(q.n0 + col) * p.lds) * 2, 8 * r, runs);
  };
  auto keep = [&](int x, u32x4 v) {
    const int row = x / per, r = x - row * per;
    if (x >= pieces) return;
    char* const to = scales + row * pitch + 16 * r;  // (8-byte aligned, an odd number of 8 bytes a row)
    *reinterpret_cast<u32x2*>(to) = u32x2{v.x, v.y};
    if (16 * r + 8 < pitch) *reinterpret_cast<u32x2*>(to + 8) = u32x2{v.z, v.w};
  };
  const u32x4 own = piece(tid);
  layer_fixed_order();
  request_b(0, 0);
  request_a(0, 0);
  request_b(1, 1);
  request_a(1, 0);
  layer_fixed_order();
  keep(tid, own);
  for (int x = tid + KW * 64; x < pieces; x += KW * 64) keep(x, piece(x));
  __syncthreads();
  for (int j = 0; j < NJ; j += 2) {
    slice(0, j);
    if (j + 1 < NJ) slice(1, j + 1);
  }
  // No load is under way when the sums overlay the slices.
  layer_fixed_order();
  pp_wait_vm<0>();
  __syncthreads();
  Sum::template finish<Tag>(acc, p.a, q, smem, tid, w);
}

// ------------------------------------------------------------------ launches --
// Workgroups of tiles of bm x bn: by rows as many as groups of any sizes need.
int64_t w4_grid(LayerArgs& a, int bm, int bn) {
  a.tiles_m = (a.M + bm - 1) / bm;
  a.tiles_n = (a.N + bn - 1) / bn;
  a.group_m = 8;
  const int64_t g = a.mode == LAYER_DENSE ? 1 : a.G < a.M ? a.G : a.M;
  return ((int64_t)a.M + g * (bm - 1)) / bm * a.tiles_n;
}

template <class Tag, int MODE, int AL, int NT, int KW, bool WHOLE = true>
struct W4Split {
  static int64_t scales(const W4Args& p) { return (int64_t)w4_pitch(p.a.K, p.group) * 16 * NT * (p.zeros ? 2 : 1); }
  // Whether so many workgroups fit a CU.
  static bool fits(const W4Args& p, int count = 1) {
    if (AL * NT >= 32 && p.group % 128) return false;  // (with smaller groups such a tile spills)
    return (w4_lds<AL, NT, KW>() + scales(p)) * count <= 160 * 1024;
  }
  static hipError_t launch(W4Args p, hipStream_t s, W4Form& form) {
    const int64_t tiles = w4_grid(p.a, 8 * AL, 16 * NT);
    form = {KW, 8 * AL, 16 * NT, WHOLE, tiles > 0xffffffffll / (KW * 64)};
    if (form.many) return hipErrorInvalidConfiguration;
    const dim3 grid((unsigned)tiles), block(KW * 64);
    auto go = [&](auto grp) {
      constexpr int GRP = decltype(grp)::value;
      const size_t lds = (size_t)scales(p);
      if (p.zeros)
        return launch_kernel_lds(layer_w4_split_kernel<Tag, MODE, AL, NT, GRP, true, KW, WHOLE>, grid, block, lds, s, p);
      return launch_kernel_lds(layer_w4_split_kernel<Tag, MODE, AL, NT, GRP, false, KW, WHOLE>, grid, block, lds, s, p);
    };
    if (p.group % 128 == 0) return go(LayerConst<128>{});
    if constexpr (AL * NT >= 32) return hipErrorInvalidValue;  // (does not fit)
    else if constexpr (WHOLE) return p.group % 64 == 0 ? go(LayerConst<64>{}) : go(LayerConst<32>{});
    else return go(LayerConst<32>{});
  }
};
// Whether operands come in whole 16-byte pieces that 32-bit offsets reach.
bool w4_whole(const W4Args& p) {
  const LayerArgs& a = p.a;
  return a.K % 32 == 0 && (uintptr_t)a.A % 16 == 0 && a.lda % 8 == 0 && (uintptr_t)a.B % 16 == 0 && a.ldb % 16 == 0 &&
         (a.G <= 1 || a.stride_b % 16 == 0) && a.lda < (1 << 23) && a.ldb < (1 << 24);
}
// The first of the forms that fits. (The last, of 16 x 16 tiles, holds the scales of kW4MaxRuns
// groups.)
template <class Form, class... Forms>
hipError_t w4_first(const W4Args& p, hipStream_t s, W4Form& form) {
  if constexpr (sizeof...(Forms) > 0)
    if (!Form::fits(p)) return w4_first<Forms...>(p, s, form);
  return Form::launch(p, s, form);
}
// Tiles, measured (us; f16, waves x rows x columns):
//   1x4096x4096    8x8x16 6.0, 16x8x16 6.3, 4x8x16 7.2
//   8x8192x8192    8x8x32 10.2, 16x8x32 10.7, 4x8x64 22.6
//   48x8192x8192   8x48x32 18.9, 4x48x32 22.8, 8x48x16 28.4
//   64x8192x8192   7x64x32 21.1, 6x64x32 22.3, 6x64x64 (128 tiles) 30.5, 8x32x32 24.2
//   256x4096x4096  6x64x64 19.1, 6x64x32 25.3, 8x32x64 22.1
//   64 experts of 2 rows, 2048x2048: 4x8x64 41, 4x8x32 42, 2x8x64 47, 8x8x64 73; with 8 KiB
//   more of LDS, for two workgroups a CU instead of three, 4x8x64 55
// and through registers:
//   257x1000x1032  4x16x32 9.8, 4x32x16 10.6, 8x48x32 10.5, 4x32x32 11.9, 8x32x32 15.4, 7x64x32 19
//   512x4096x4104  4x32x64 48, 4x32x32 56, 7x64x32 77, 8x32x32 84
//   48x4096x4104   8x32x32 13.2, 8x48x32 16.0, 8x32x16 21.5
template <class Tag, int MODE>
hipError_t launch_rows(const W4Args& p, hipStream_t s, W4Form& form) {
  const LayerArgs& a = p.a;
  // Rows of a group, on average.
  const int64_t rows = MODE == LAYER_ROWS ? ((int64_t)a.M + a.G - 1) / a.G : a.M;
  if (!w4_whole(p)) {
    using R16 = W4Split<Tag, MODE, 2, 1, 8, false>;
    if (rows <= 16) return R16::launch(p, s, form);
    // (Twice the columns, 4x32x64, take 48 us instead of 56, but spill with groups of 32.)
    if (((int64_t)a.M + 31) / 32 * (((int64_t)a.N + 31) / 32) >= 1024)
      return w4_first<W4Split<Tag, MODE, 4, 2, 4, false>, R16>(p, s, form);
    if (a.K >= 2048) return w4_first<W4Split<Tag, MODE, 4, 2, 8, false>, R16>(p, s, form);
    return w4_first<W4Split<Tag, MODE, 2, 2, 4, false>, R16>(p, s, form);
  }
  using Last = W4Split<Tag, MODE, 2, 1, 8>;
  if constexpr (MODE == LAYER_ROWS) {
    using Wide8 = W4Split<Tag, MODE, 1, 4, 4>;
    if (rows <= 8 && Wide8::fits(p, 3)) return Wide8::launch(p, s, form);
    if (rows <= 8) return w4_first<W4Split<Tag, MODE, 1, 2, 4>, Last>(p, s, form);
    if (rows <= 16) return w4_first<W4Split<Tag, MODE, 2, 2, 4>, Last>(p, s, form);
    return w4_first<W4Split<Tag, MODE, 4, 4, 4>, Last>(p, s, form);
  } else {
    if (rows <= 8 && a.N <= 16 * 256) return w4_first<W4Split<Tag, MODE, 1, 1, 8>, Last>(p, s, form);
    if (rows <= 8) return w4_first<W4Split<Tag, MODE, 1, 2, 8>, Last>(p, s, form);
    if (rows <= 16) return w4_first<W4Split<Tag, MODE, 2, 2, 8>, Last>(p, s, form);
    using Slim32 = W4Split<Tag, MODE, 4, 2, 8>;
    if (rows <= 32) return w4_first<Slim32, Last>(p, s, form);
    using Wide64 = W4Split<Tag, MODE, 8, 4, 6>;
    if (((int64_t)a.M + 63) / 64 * (((int64_t)a.N + 63) / 64) >= 256 && Wide64::fits(p)) return Wide64::launch(p, s, form);
    if (rows <= 48) return w4_first<W4Split<Tag, MODE, 6, 2, 8>, Slim32, Last>(p, s, form);
    return w4_first<W4Split<Tag, MODE, 8, 2, 7>, Slim32, Last>(p, s, form);
  }
}

template <class Tag>
hipError_t launch_modes(const W4Args& p, hipStream_t s, W4Form& form) {
  return p.a.mode == LAYER_ROWS ? launch_rows<Tag, LAYER_ROWS>(p, s, form) : launch_rows<Tag, LAYER_DENSE>(p, s, form);
}

}  // namespace
}  // namespace dgt
