// What one call of the layer norm and of its gradients carries.
#pragma once

#include "layer_rows.h"

namespace dgt {

struct NormArgs {
  const void* X;
  const void* gamma;  // null: ones
  const void* beta;   // null: zeros
  void* Y;
  float* mean;        // null: not wanted
  float* rstd;        // null: not wanted
  int64_t ldx, ldy;   // elements
  float eps;
  int M, N;
  unsigned grid_x;    // set at the launch (layer_grid)
};

struct NormGradArgs {
  const void* dY;
  const void* X;
  const void* gamma;   // null: ones
  const float* mean;
  const float* rstd;
  const void* R;       // null: none
  void* dX;            // null: not wanted
  float* dgamma;       // null: not wanted
  float* dbeta;        // null: not wanted
  float* part;         // [parts][2][N]: partial sums of dgamma and dbeta
  int64_t lddy, ldx, ldr, lddx;
  int M, N;
  int rows, parts;     // rows that one partial sum covers (long rows), and their number
  unsigned grid_x;
};

}  // namespace dgt
