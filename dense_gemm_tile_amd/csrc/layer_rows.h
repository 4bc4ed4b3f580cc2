// The layer operators that move rows and ids: launchers, each next to its
// kernels in layer_rows.hip and layer_route.hip. They return the HIP status of
// the first launch that failed.
#pragma once

#include "common.h"

namespace dgt {

// n workgroups as a grid. A launch holds less than 2^32 threads along a
// dimension (and one of more computes a part without an error), so further
// workgroups go along z, the last of them in part past n. grid_x: workgroups of
// one z, which the kernel gets among its arguments (layer_block() in
// layer_rows.hip): the built-in is a hidden argument more for every launch.
inline dim3 layer_grid(int64_t n, unsigned threads, unsigned& grid_x, unsigned y = 1) {
  const int64_t most = ((int64_t{1} << 32) - 1) / threads;
  const int64_t z = (n + most - 1) / most;
  grid_x = (unsigned)((n + z - 1) / z);
  return dim3(grid_x, y, (unsigned)z);
}

// Element types of rows.
enum RowType : int { ROW_F16 = 0, ROW_BF16 = 1, ROW_F32 = 2 };

struct ActGradArgs {
  const int* offsets;  // null: one group of all M rows
  const void* dY;
  const void* Z;       // null: no activation
  void* dZ;            // null: not wanted
  float* db;           // null: not wanted
  float* part;         // partial column sums
  int64_t lddy, ldz, lddz;
  int G, M, N, act;
  int rows;            // act_grad_rows(M, N)
  unsigned grid_x;     // set at the launch (layer_grid), as in the others
};
// Rows that one wave sums by itself (a partial sum is kept for each): 32, fewer
// where that would leave less than 16 waves to a CU. At 4096 x 4096 with GELU,
// 32 rows a wave (4 waves a CU) take 51 us, 4 rows a wave (32) 26 us. Fewer
// than 4 where waves are fewer than SIMDs, as a row then costs its arithmetic's
// latency (76 x 2622: 12 us, 7 so), but not for more than 256 partial sums a
// column, whose joining costs as much (613 x 1536: 9 us, 12 so).
inline int act_grad_rows(int64_t m, int64_t n) {
  const int64_t blocks = (n + 511) / 512;
  int rows = 32;
  while (rows > 4 && (m + rows - 1) / rows * blocks < 16 * 256) rows /= 2;
  while (rows > 1 && (m + rows - 1) / rows <= 128 && (m + rows - 1) / rows * blocks < 4 * 256)
    rows /= 2;
  return rows;
}
// Waves that a call is cut into.
inline int64_t act_grad_waves(int64_t m, int64_t n) {
  const int rows = act_grad_rows(m, n);
  return (m + rows - 1) / rows * ((n + 511) / 512);
}
hipError_t launch_act_grad(int dtype, ActGradArgs a, hipStream_t s);

struct RouteArgs {
  const int* ids;
  int* offsets;
  int* order;
  int* slot;
  int* counts;  // [blocks][E + 1], more than one block only
  int n;        // choices
  int E;
  int blocks, chunk;  // choices per block
};
constexpr int kRouteMaxExperts = 1024;
// Blocks that a call of n choices is cut into, and choices per block.
void route_blocks(int64_t n, int& blocks, int& chunk);
hipError_t launch_route(const RouteArgs& a, hipStream_t s);

struct DispatchArgs {
  const char* X;
  char* Xs;
  const int* slot;
  int64_t ldx, ldxs;  // bytes
  int T, top;
  int64_t bytes;      // of a row
  int piece;          // bytes per access: 16, 8, 4 or 2
  unsigned grid_x;
};
constexpr int kDispatchSpan = 4;  // pieces a lane
inline int64_t dispatch_column_blocks(const DispatchArgs& a) {
  const int64_t span = (int64_t)kDispatchSpan * 64 * a.piece;
  return (a.bytes + span - 1) / span;
}
hipError_t launch_dispatch(DispatchArgs a, hipStream_t s);

struct CombineArgs {
  const void* Ys;
  const int* slot;
  const float* weights;  // null: ones
  const void* R;         // null: none
  void* Y;
  int64_t ldys, ldr, ldy;  // elements
  int T, top, H;
  int piece;  // elements per access
  int once;   // the rows read fill half of the last cache (256 MiB) or more
  unsigned grid_x;
};
// Pieces a lane: two once that leaves 16 waves to a CU.
inline int combine_span(const CombineArgs& a) {
  return a.once || (int64_t)a.T * a.H >= (int64_t)2 * 64 * a.piece * 16 * 256 ? 2 : 1;
}
// Waves that a call's rows are cut into.
inline int64_t combine_waves(const CombineArgs& a) {
  const int64_t span = (int64_t)combine_span(a) * 64 * a.piece;
  return a.T * ((a.H + span - 1) / span);
}
hipError_t launch_combine(int rowtype, const CombineArgs& a, hipStream_t s);

struct CombineGradArgs {
  const void* dY;
  const void* Ys;        // null without dw
  const int* slot;
  const float* weights;  // null: ones
  void* dYs;             // null: not wanted
  float* dw;             // null: not wanted
  int64_t lddy, ldys, lddys;
  int T, top, H;
  int piece;
  unsigned grid_x;
};
hipError_t launch_combine_grad(int rowtype, const CombineGradArgs& a, hipStream_t s);

}  // namespace dgt
