// Microscaled 4-bit floats, shared by the kernels that write and read them (not installed).
//
// A block of 32 consecutive values is 32 codes of 4 bits (sign, two exponent bits, one mantissa bit: 0, 1/2,
// 1, 3/2, 2, 3, 4, 6), two a byte with the even value in the low half, and a scale byte s that stands
// for 2^(s - 127); s = 255 makes the block NaN.
#pragma once

#include "delta_common.h"

namespace mol {
namespace {

typedef float f32x2_t __attribute__((ext_vector_type(2)));

constexpr uint32_t kMxNaN = 255u;  // the scale of a block that is NaN

// The scale as the float that the conversions take: 2^(s - 127), 2^-127 a subnormal, NaN.
__device__ __forceinline__ float mx_scale(uint32_t s) {
  return __uint_as_float(s == 0 ? 0x00400000u : s == kMxNaN ? 0x7fc00000u : s << 23);
}

// Eight codes of a dword times a scale: bf16 (exact: two bits of mantissa, and bf16's subnormals reach
// 2^-133) or fp32; infinite from 2^128 on. A NaN scale makes them NaN.
__device__ __forceinline__ uint4 mx_bf16(uint32_t w, float scale) {
  return make_uint4(
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2)),
      __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3)));
}
__device__ __forceinline__ void mx_f32(uint32_t w, float scale, float (&f)[8]) {
  const f32x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0);
  const f32x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
  const f32x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2);
  const f32x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
  f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
  f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
}

// Eight values over a scale as codes: to the nearest, halves to the even code, beyond 6 to 6.
__device__ __forceinline__ uint32_t mx_encode(const float (&f)[8], float scale) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[0], f[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[2], f[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[4], f[5], scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, f[6], f[7], scale, 3);
}

}  // namespace
}  // namespace mol
