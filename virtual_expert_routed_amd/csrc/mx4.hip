// Rows of numbers to microscaled 4-bit floats and back (mx4.h has the format).
//
// Per block of 32 values v, with m = max |v|:
//   s    = max(floor(log2 m) - 2, -127) + 127      the scale's byte: m / 2^(s - 127) is in [4, 8)
//   code = v / 2^(s - 127) to the nearest of the fifteen values, halves to the even code, beyond 6 to 6
// A block that holds a NaN or an infinity gets s = 255 and codes of zero. With the activation, v is
// SiLU(gate) * up of two halves of a row.
//
// The division is by a power of two and the rounding the hardware's, so codes of given values are
// exact. Those of the activation are the ones of its value in 64 bits: the product is formed in fp32,
// within 2^-18.5 of itself and 2^-149 |up|, and lanes whose codes or scale would be others 2^-18 to either
// side form it again in 64 bits (about one lane in a thousand), as do blocks with an up so large that the
// second term counts: SiLU(gate) is then a number below fp32's normal ones, or 0 in fp32. So do blocks whose
// product leaves fp32's range, which decide in 64 bits whether a value is 2^128 or more.
//
// Bound by bytes. A lane takes eight consecutive values (16 bytes of bf16), four lanes a block; a thread
// has kVecs such vectors in flight. Kernel times (rocprofv3): 196608 rows of 2048 in fp32 (1.6 GB, to codes and
// back) 340 and 328 us, 5.4 and 5.6 TB/s; the activation of 32768 bf16 rows of 2 x 768 27 us over the same rows again
// (4.2 TB/s: eight exponentials, reciprocals and two encodings a lane beside the bytes) and 33 us over three sets in turn,
// which the last-level cache does not hold; back to bf16 10 us (6.3 TB/s); 23 rows of 2048 3 us each way, a launch.
#include "mx4.h"
#include "skinny.h"

namespace mol {
namespace {

constexpr int kVecs = 4;                        // vectors of eight values a thread
constexpr int kChunk = kThreads * kVecs;        // and a workgroup

// Eight elements from a row: wide loads where rows are on 16-byte boundaries.
template <bool BF16>
__device__ __forceinline__ void load8(const char* row, int v, bool vec, float (&f)[8]) {
  constexpr int ESZ = BF16 ? 2 : 4;
  const char* p = row + (int64_t)v * (8 * ESZ);
  if (vec) {
    if constexpr (BF16) {
      const uint4 w = ld16(p);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(u[i]);
        f[2 * i + 1] = bf16_hi(u[i]);
      }
    } else {
      const uint4 a = ld16(p), b = ld16(p + 16);
      const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (BF16) f[i] = __uint_as_float((uint32_t)((const uint16_t*)p)[i] << 16);
      else f[i] = ((const float*)p)[i];
    }
  }
}

// the largest over the four lanes of a block
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xf, 0xf, false));
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xf, 0xf, false));
}

// the scale's byte of a block whose largest |v| has these bits
__device__ __forceinline__ uint32_t scale_of(uint32_t m) {
  return m >= 0x7f800000u ? kMxNaN : (uint32_t)max((int)(m >> 23) - 2, 0);
}

// v = SiLU(g) * u within 2^-18.5 of itself, and what SiLU(g) loses below the normal numbers, up to 2^-149, times |u|. Up to
// |g| = 32 the hardware's exp2 and reciprocal do: the exponent's argument is rounded at 46 (2^-19.5 in all).
__device__ __forceinline__ void silu_mul8(const float (&g)[8], const float (&u)[8], float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(g[j]));
  if (m < 32.f) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = g[j] * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(g[j] * -1.44269502f)) * u[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = silu(g[j]) * u[j];
  }
}

// Whether a lane's ups meet bits that SiLU(g) has lost: 2^-149 |u| is more than 2^-23 of the block's scale, 2^-21 of the
// smallest value that is not 0. Gates of zero lose nothing.
__device__ __forceinline__ bool silu_lost(const float (&g)[8], const float (&u)[8], float unit) {
  bool lost = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) lost |= g[j] != 0.f && fabsf(u[j]) > unit * 0x1p126f;
  return lost;
}

__device__ __forceinline__ bool all_finite(const float (&g)[8], const float (&u)[8]) {
  bool all = true;
#pragma unroll
  for (int j = 0; j < 8; ++j) all &= fabsf(g[j]) < __builtin_inff() && fabsf(u[j]) < __builtin_inff();
  return all;
}

// SiLU(g) * u in 64 bits
__device__ __forceinline__ double silu_mul64(float g, float u) {
  return (double)g / (1.0 + exp(-(double)g)) * (double)u;
}

// A value in 64 bits over 2^(s - 127) as a code.
__device__ __forceinline__ uint32_t encode64(double v, int s) {
  const double y = ldexp(fabs(v), 127 - s);
  const uint32_t c = (y > 0.25) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0);
  return c | (__builtin_signbit(v) ? 8u : 0u);
}

// The codes of vector i once more, from values in 64 bits, and the scale if `scale` (then in a block's four
// lanes together; NaN, as the codes have to find it, if a value is 2^128 or more or none). Reads its values again: kept,
// they would take registers from every lane.
template <bool BF16>
__device__ __forceinline__ void codes64(const MxArgs& a, int i, bool scale, uint32_t& w, uint32_t& s) {
  const int row = fdiv(i, a.f_vpr), k0 = (i - row * a.vpr) * 8;
  auto value = [&](int j) {
    const int64_t at = (int64_t)row * a.ld + k0 + j;
    if constexpr (BF16)
      return silu_mul64(__uint_as_float((uint32_t)((const uint16_t*)a.x)[at] << 16),
                        __uint_as_float((uint32_t)((const uint16_t*)a.x)[at + a.K] << 16));
    else
      return silu_mul64(((const float*)a.x)[at], ((const float*)a.x)[at + a.K]);
  };
  if (scale) {
    double d = 0.0;
#pragma unroll 1
    for (int j = 0; j < 8; ++j) {
      const double v = fabs(value(j));
      d = v < 0x1p128 ? fmax(d, v) : 0x1p128;
    }
    d = fmax(d, __shfl_xor(d, 1, 64));
    d = fmax(d, __shfl_xor(d, 2, 64));
    s = d < 0x1p128 ? (uint32_t)max(ilogb(d) + 125, 0) : kMxNaN;
    if (s == kMxNaN) return;
  }
  w = 0;
#pragma unroll 1
  for (int j = 0; j < 8; ++j) w |= encode64(value(j), (int)s) << (4 * j);
}

template <bool BF16, bool ACT>
__global__ void __launch_bounds__(kThreads) mx4_quantize_kernel(MxArgs a) {
  constexpr int ESZ = BF16 ? 2 : 4;
  const int i0 = (int)blockIdx.x * kChunk + (int)threadIdx.x;
  float f[kVecs][8], g[ACT ? kVecs : 1][8];
#pragma unroll
  for (int t = 0; t < kVecs; ++t) {
    const int i = min(i0 + t * kThreads, a.vecs - 1);  // (a vector of eight values of some row)
    const int row = fdiv(i, a.f_vpr), v = i - row * a.vpr;
    const char* src = (const char*)a.x + (int64_t)row * a.ld * ESZ;
    if constexpr (ACT) {
      load8<BF16>(src, v, a.vec, g[t]);
      load8<BF16>(src + (int64_t)a.K * ESZ, v, a.vec, f[t]);
    } else {
      load8<BF16>(src, v, a.vec, f[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < kVecs; ++t) {
    const int i = i0 + t * kThreads;
    if (i >= a.vecs) break;  // (a block's four lanes go together)
    float v[8];
    if constexpr (ACT) silu_mul8(g[t], f[t], v);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if constexpr (!ACT) v[j] = f[t][j];
      m = max(m, __float_as_uint(v[j]) & 0x7fffffffu);
    }
    m = block_max(m);
    uint32_t s = scale_of(m);
    uint32_t w;
    if constexpr (!ACT) {
      w = mx_encode(v, mx_scale(s));
    } else {
      constexpr float kLess = 1.f - 0x1p-18f, kMore = 1.f + 0x1p-18f;
      float lo[8], hi[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        lo[j] = v[j] * kLess;
        hi[j] = v[j] * kMore;
      }
      const float mf = __uint_as_float(m), unit = mx_scale(s);
      bool other_scale = scale_of(__float_as_uint(mf * kLess)) != scale_of(__float_as_uint(mf * kMore));
      float um = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) um = fmaxf(um, fabsf(f[t][j]));
      if (__builtin_amdgcn_ballot_w64(!(um <= unit * 0x1p126f))) {  // rare, and where the scale is NaN
        if (s == kMxNaN) other_scale |= block_max(!all_finite(g[t], f[t])) == 0;
        else other_scale |= block_max(silu_lost(g[t], f[t], unit)) != 0;
      }
      w = mx_encode(lo, unit);  // (the same as v's, or formed again)
      if (other_scale || (s != kMxNaN && w != mx_encode(hi, unit)))
        codes64<BF16>(a, i, other_scale, w, s);
    }
    if (s == kMxNaN) w = 0;
    ((uint32_t*)a.q)[i] = w;
    if ((threadIdx.x & 3) == 0) a.scales[i >> 2] = (uint8_t)s;
  }
}

// A lane writes 16 bytes, so that a wave's are neighbours: eight values in bf16, four in fp32.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) mx4_dequantize_kernel(MxArgs a) {
  constexpr int V = BF16 ? 8 : 4;  // values a lane
  const int i0 = (int)blockIdx.x * kChunk + (int)threadIdx.x;
  uint32_t w[kVecs], s[kVecs];
#pragma unroll
  for (int t = 0; t < kVecs; ++t) {
    const int i = min(i0 + t * kThreads, a.vecs - 1);
    w[t] = BF16 ? ((const uint32_t*)a.q)[i] : ((const uint16_t*)a.q)[i];
    s[t] = a.scales[i / (kMxValues / V)];
  }
#pragma unroll
  for (int t = 0; t < kVecs; ++t) {
    const int i = i0 + t * kThreads;
    if (i >= a.vecs) break;
    const int row = fdiv(i, a.f_vpr), v = i - row * a.vpr;
    char* dst = (char*)a.out + (int64_t)row * a.ld * (16 / V) + (int64_t)v * 16;
    const float unit = mx_scale(s[t]);
    uint4 b;
    if constexpr (BF16) {
      b = mx_bf16(w[t], unit);
    } else {
      const f32x2_t x = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[t], unit, 0);
      const f32x2_t y = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[t], unit, 1);
      b = make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(y.x), __float_as_uint(y.y));
    }
    if (a.vec) {
      st16_nt(dst, b);
    } else {
      const uint32_t u[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if constexpr (BF16) ((uint16_t*)dst)[j] = (uint16_t)(u[j / 2] >> (16 * (j % 2)));
        else ((uint32_t*)dst)[j] = u[j];
      }
    }
  }
}

int grid_of(const MxArgs& a) { return (int)(((int64_t)a.vecs + kChunk - 1) / kChunk); }

}  // namespace

hipError_t launch_mx4_quantize(const MxArgs& a, bool bf16, bool act, hipStream_t st) {
  const dim3 grid(grid_of(a)), threads(kThreads);
  if (bf16) {
    if (act) hipLaunchKernelGGL((mx4_quantize_kernel<true, true>), grid, threads, 0, st, a);
    else hipLaunchKernelGGL((mx4_quantize_kernel<true, false>), grid, threads, 0, st, a);
  } else {
    if (act) hipLaunchKernelGGL((mx4_quantize_kernel<false, true>), grid, threads, 0, st, a);
    else hipLaunchKernelGGL((mx4_quantize_kernel<false, false>), grid, threads, 0, st, a);
  }
  return hipGetLastError();
}

hipError_t launch_mx4_dequantize(MxArgs a, bool bf16, hipStream_t st) {
  if (!bf16) {  // vectors of four
    a.vpr *= 2;
    a.vecs *= 2;
    a.f_vpr = make_fastdiv((uint32_t)a.vpr);
  }
  const dim3 grid(grid_of(a)), threads(kThreads);
  if (bf16) hipLaunchKernelGGL((mx4_dequantize_kernel<true>), grid, threads, 0, st, a);
  else hipLaunchKernelGGL((mx4_dequantize_kernel<false>), grid, threads, 0, st, a);
  return hipGetLastError();
}

}  // namespace mol
