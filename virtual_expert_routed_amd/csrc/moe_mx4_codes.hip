// The base grouped GEMM over microscaled 4-bit weights: rows of codes.
#include "moe_mx4_tiles.h"

namespace mol {

hipError_t launch_mx4_gemm_codes(const MxGemmArgs& a, bool out_bf16, int form, hipStream_t st) {
  if (out_bf16) {
    switch (form) {
      case kMxSplit: return mx4_narrow<kMxRowsCodes, true, 16, 2, 4>(a, st);
      case kMxNarrow: return mx4_narrow<kMxRowsCodes, true, 64, 1, 1>(a, st);
      case kMxTiles: return mx4_tiles<true>(a, st);
      default: return mx4_wide<kMxRowsCodes, true, 128, 2, 1, 8>(a, st);
    }
  }
  switch (form) {
    case kMxSplit: return mx4_narrow<kMxRowsCodes, false, 16, 2, 4>(a, st);
    case kMxNarrow: return mx4_narrow<kMxRowsCodes, false, 64, 1, 1>(a, st);
    case kMxTiles: return mx4_tiles<false>(a, st);
    default: return mx4_wide<kMxRowsCodes, false, 128, 2, 1, 8>(a, st);
  }
}

}  // namespace mol
