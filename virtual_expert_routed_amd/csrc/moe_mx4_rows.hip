// The base grouped GEMM over microscaled 4-bit weights: bf16 and fp32 rows, and the choice of the form.
#include "moe_mx4.h"

namespace mol {

hipError_t launch_mx4_gemm_codes(const MxGemmArgs& a, bool out_bf16, int form, hipStream_t st);

hipError_t launch_mx4_gemm(const MxGemmArgs& a, bool bf16, int form, hipStream_t st) {
  if (a.x_scales) return launch_mx4_gemm_codes(a, bf16, form, st);
  if (bf16) {
    switch (form) {
      case kMxSplit: return mx4_launch<kMxRowsBf16, true, 16, 1, 2, 4>(a, false, st);
      case kMxNarrow: return mx4_launch<kMxRowsBf16, true, 16, 1, 4, 1>(a, false, st);
      default: return mx4_launch<kMxRowsBf16, true, 128, 4, 1, 1>(a, true, st);
    }
  }
  switch (form) {
    case kMxSplit: return mx4_launch<kMxRowsF32, false, 16, 1, 1, 4>(a, false, st);
    case kMxNarrow: return mx4_launch<kMxRowsF32, false, 16, 1, 2, 1>(a, false, st);
    default: return mx4_launch<kMxRowsF32, false, 32, 1, 1, 1>(a, true, st);
  }
}

}  // namespace mol
