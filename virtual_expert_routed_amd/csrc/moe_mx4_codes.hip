// The base grouped GEMM over microscaled 4-bit weights: rows of codes.
#include "moe_mx4.h"

namespace mol {

hipError_t launch_mx4_gemm_codes(const MxGemmArgs& a, bool out_bf16, int form, hipStream_t st) {
  if (out_bf16) {
    switch (form) {
      case kMxSplit: return mx4_launch<kMxRowsCodes, true, 16, 1, 2, 4>(a, false, st);
      case kMxNarrow: return mx4_launch<kMxRowsCodes, true, 16, 1, 4, 1>(a, false, st);
      default: return mx4_launch<kMxRowsCodes, true, 128, 4, 1, 1>(a, true, st);
    }
  }
  switch (form) {
    case kMxSplit: return mx4_launch<kMxRowsCodes, false, 16, 1, 2, 4>(a, false, st);
    case kMxNarrow: return mx4_launch<kMxRowsCodes, false, 16, 1, 4, 1>(a, false, st);
    default: return mx4_launch<kMxRowsCodes, false, 128, 4, 1, 1>(a, true, st);
  }
}

}  // namespace mol
