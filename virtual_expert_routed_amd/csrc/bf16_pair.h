// Two floats as packed bf16, shared by the kernels that store bf16 rows from fp32 sums (not installed).
#pragma once

#include "delta_common.h"

namespace mol {
namespace {

// two floats to packed bf16 (to nearest even), one instruction
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2_t));
}

}  // namespace
}  // namespace mol
