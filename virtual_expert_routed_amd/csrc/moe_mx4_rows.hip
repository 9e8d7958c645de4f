// The base grouped GEMM over microscaled 4-bit weights: bf16 and fp32 rows, and the choice of the form.
#include "moe_mx4.h"

namespace mol {

hipError_t launch_mx4_gemm_codes(const MxGemmArgs& a, bool out_bf16, int form, hipStream_t st);

hipError_t launch_mx4_gemm(const MxGemmArgs& a, bool bf16, int form, hipStream_t st) {
  if (a.x_scales) return launch_mx4_gemm_codes(a, bf16, form, st);
  if (bf16) {
    switch (form) {
      case kMxSpread: return mx4_narrow<kMxRowsBf16, true, 32, 2, 1, true>(a, st);
      case kMxNarrow: return mx4_narrow<kMxRowsBf16, true, 64, 1, 1, false>(a, st);
      default: return mx4_wide<kMxRowsBf16, true, 128, 2, 1, 8>(a, st);
    }
  }
  switch (form) {
    case kMxSplit: return mx4_narrow<kMxRowsF32, false, 16, 1, 4, true>(a, st);
    case kMxNarrow: return mx4_narrow<kMxRowsF32, false, 32, 1, 1, false>(a, st);
    default: return mx4_wide<kMxRowsF32, false, 32, 1, 1, 4>(a, st);
  }
}

}  // namespace mol
