// The base grouped GEMM over 4-bit weights: groups of 128, and the choice between the group sizes.
#include "moe_q4.h"

namespace mol {

hipError_t launch_q4_gemm(const Q4GemmArgs& a, bool bf16, hipStream_t st) {
  switch (a.group) {
    case 32: return launch_q4_gemm_g32(a, bf16, st);
    case 64: return launch_q4_gemm_g64(a, bf16, st);
    case 128: return launch_q4_group<128>(a, bf16, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mol
