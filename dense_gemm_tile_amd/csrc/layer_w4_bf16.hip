// Products of bf16 values with 4-bit weights (layer_w4.h).
#include "layer_w4.h"

namespace dgt {

hipError_t launch_w4_bf16(const W4Args& p, hipStream_t s, W4Form& form) {
  return launch_modes<TagBF16>(p, s, form);
}

}  // namespace dgt
