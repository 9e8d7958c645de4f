// A whole mixture-of-experts layer for a few tokens: 4-bit weights in groups of 64.
#include "moe_layer.h"

namespace mol {

hipError_t launch_moe_layer_q64(const LayerArgs& a, bool bf16, hipStream_t st) {
  return launch_layer_group<64>(a, bf16, st);
}

}  // namespace mol
