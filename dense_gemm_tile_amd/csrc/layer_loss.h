// What the kernels of the output layer's cross entropy share.
#pragma once

#include "layer.h"
#include "layer_rows.h"

namespace dgt {

// exp(x): the hardware's, of an exponent rounded once (about |x| half steps of the result, and one step).
__device__ __forceinline__ float loss_exp(float x) { return __builtin_amdgcn_exp2f(kLog2e * x); }

// One product of the loss on 256x256 tiles: logits of n vocabulary entries from v0 on (rows) for
// T tokens (columns), and what becomes of them.
struct LossTileArgs {
  const void* W;       // its first row
  const void* X;
  int64_t ldw, ldx;
  int n, T, H;
  int v0;
  int tiles_m, tiles_n, group_m;
  const int* labels;
  int V;
  // Forward.
  float2* parts;       // [tiles_m][T]: a tile's largest logit and sum for each token
  float* target;       // [T]: the label's logit
  // Gradient.
  const float* lse;
  const float* dloss;
  const float* scale;  // dloss is taken relative to it
  void* G;             // n x T8 of the operands' type
  int T8;              // T as a multiple of 8, G's pitch; 0 in the columns from T on
};
// dtype: 0 f16, 1 bf16. Operands in whole 16-byte pieces.
hipError_t launch_loss_tiles(int dtype, bool grad, const LossTileArgs& a, hipStream_t s);

}  // namespace dgt
