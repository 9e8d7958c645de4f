// The base grouped GEMM over microscaled 4-bit weights: rows of codes.
#include "moe_mx4.h"

namespace mol {
namespace {

template <bool OBF16>
hipError_t by_form(const MxGemmArgs& a, int form, hipStream_t st) {
  switch (form) {
    case kMxSpread: return mx4_narrow<kMxRowsCodes, OBF16, 64, 1, 1, true>(a, st);
    case kMxNarrow: return mx4_narrow<kMxRowsCodes, OBF16, 64, 1, 1, false>(a, st);
    default: return mx4_wide<kMxRowsCodes, OBF16, 128, 2, 1, 8>(a, st);
  }
}

}  // namespace

hipError_t launch_mx4_gemm_codes(const MxGemmArgs& a, bool out_bf16, int form, hipStream_t st) {
  return out_bf16 ? by_form<true>(a, form, st) : by_form<false>(a, form, st);
}

}  // namespace mol
