// The base grouped GEMM over 4-bit weights: groups of 32.
#include "moe_q4.h"

namespace mol {

hipError_t launch_q4_gemm_g32(const Q4GemmArgs& a, bool bf16, hipStream_t st) {
  return launch_q4_group<32>(a, bf16, st);
}

}  // namespace mol
