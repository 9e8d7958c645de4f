// A row of router logits in the registers of LPR lanes, VPL consecutive experts a lane, shared by the
// router and the balance loss (not installed). Masked logits (NaN and -infinity) are held as -infinity.
#pragma once

#include "delta_common.h"

namespace mol {
namespace {

constexpr float kMasked = -__builtin_inff();

template <int CTRL>
__device__ __forceinline__ float max_lane(float v) {
  return fmaxf(v, from_lane<CTRL>(v));
}

// the maximum over each group of LPR consecutive lanes, in every lane of the group (the
// butterfly of group_sum)
template <int LPR>
__device__ __forceinline__ float group_max(float v) {
  v = max_lane<0xB1>(v);
  v = max_lane<0x4E>(v);
  v = max_lane<0x141>(v);
  v = max_lane<0x140>(v);
  if constexpr (LPR >= 64) {
    v = fmaxf(v, __int_as_float(__builtin_amdgcn_ds_swizzle(__float_as_int(v), 0x401F)));
    v = fmaxf(v, __shfl_xor(v, 32, 64));
  }
  return v;
}

// exp(l - m) for l <= m; 1 at l == m, infinite m included
__device__ __forceinline__ float exp_below(float l, float m) { return l == m ? 1.f : expf(l - m); }

// Experts [e0, e0 + n), n <= VPL, of the row at src; the rest of the lane's registers are masked.
template <bool BF16, int VPL>
__device__ __forceinline__ void load_row(const char* src, int e0, int n, bool vec, float (&v)[VPL]) {
  constexpr int ESZ = BF16 ? 2 : 4;
  constexpr int VE = 16 / ESZ;
  if (VPL % VE == 0 && vec) {
#pragma unroll
    for (int i = 0; i < VPL; i += VE) {
      if (i + VE <= n) {
        const uint4 w = ld16(src + (int64_t)(e0 + i) * ESZ);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < VE; ++j)
          v[i + j] = !BF16 ? __uint_as_float(u[j % 4]) : j % 2 ? bf16_hi(u[j / 2]) : bf16_lo(u[j / 2]);
      } else {
#pragma unroll
        for (int j = 0; j < VE; ++j) {
          float x = kMasked;
          if (i + j < n) {
            if constexpr (BF16) x = __uint_as_float((uint32_t)((const uint16_t*)src)[e0 + i + j] << 16);
            else x = ((const float*)src)[e0 + i + j];
          }
          v[i + j] = x;
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      float x = kMasked;
      if (i < n) {
        if constexpr (BF16) x = __uint_as_float((uint32_t)((const uint16_t*)src)[e0 + i] << 16);
        else x = ((const float*)src)[e0 + i];
      }
      v[i] = x;
    }
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (v[i] != v[i]) v[i] = kMasked;
}

}  // namespace
}  // namespace mol
