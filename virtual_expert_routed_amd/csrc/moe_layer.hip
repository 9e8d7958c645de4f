// A whole mixture-of-experts layer for a few tokens: dense weights, and the choice between the
// weight formats.
#include "moe_layer.h"

namespace mol {

hipError_t launch_moe_layer(const LayerArgs& a, bool bf16, hipStream_t st) {
  switch (a.group) {
    case 0: return launch_layer_group<0>(a, bf16, st);
    case 32: return launch_moe_layer_q32(a, bf16, st);
    case 64: return launch_moe_layer_q64(a, bf16, st);
    case 128: return launch_moe_layer_q128(a, bf16, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mol
