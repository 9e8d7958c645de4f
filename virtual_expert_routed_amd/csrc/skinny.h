// Products of a few input rows with rows of a large weight matrix, on the matrix cores, shared
// by the 4-bit grouped GEMM and the whole-layer kernels (not installed).
//
//   acc[row, col] = sum_k W[row, k] x[col, k]     16 weight rows, up to 16 T input rows (pairs)
//
// The product is bound by reading W once, so the tile follows W: a 16 x 16 matrix-core tile
// whose A operand is W (each lane loads 16 bytes of one row, a row's four lanes 64 contiguous
// bytes) and whose B operand is x. With one to three pairs most columns of the tile are unused,
// and the matrix cores still run far below their rate at the speed W arrives. Columns are
// independent: nothing in one pair's row (an infinity, a NaN) reaches another pair.
// Lane l holds, of A and of B, row (column) l % 16 and the k's of quad l / 16; of the result,
// column l % 16 and rows 4 (l / 16) + i.
//
// 4-bit weights: two per byte, the even k in the low half; value (q - z) * s with a scale s and a
// zero point z (8 without a table) per group of G consecutive k's. A step takes 128 k's, 16
// bytes a lane, and moves them so that one matrix-core step covers 32 consecutive k's (a 4 x 4
// transpose of dwords between the quads): no group is then split over a step. In bf16, q goes
// into the top mantissa bits of 16.0, which is 16 + q exactly; in fp32, q is converted. The
// products with x are summed per group, and
//   sum_k (q - z) x = sum_k (q + c) x - (c + z) sum_k x,    c = 16 (bf16) or 0 (fp32)
// with sum_k x from one more matrix-core step against ones. Everything after the operands is
// fp32, and the scale is applied once per group.
#pragma once

#include "delta_common.h"

namespace mol {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kTileRows = 16;
constexpr int kTiles = 4;      // tiles of 16 pairs one pass holds
constexpr int kWaves = kThreads / 64;
constexpr int kQ4Chunk = 128;  // k's of one 16-byte load of 4-bit weights by a row's four lanes

// A lane's weight row inside one expert's matrix (uniform over the wave): bytes past the matrix
// read as zero, and so does a row that is not there (off = kOutOfRange).
struct BufRow {
  __amdgpu_buffer_rsrc_t r;
  uint32_t off;
  __device__ __forceinline__ uint4 operator()(uint32_t byte, bool ok) const {
    return buf16(r, ok ? off + byte : kOutOfRange);
  }
};

// A lane's weight row at an address of its own (each lane may have another expert).
struct PtrRow {
  const char* p;
  bool there;
  __device__ __forceinline__ uint4 operator()(uint32_t byte, bool ok) const {
    return ld16_if(p, byte, ok && there);
  }
};

__device__ __forceinline__ f32x4_t mma_bf16(const uint4& a, const uint4& b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                 __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mma_f32(float a, float b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

template <bool BF16>
__device__ __forceinline__ f32x4_t mma16(const uint4& a, const uint4& b, f32x4_t c) {
  if constexpr (BF16) {
    return mma_bf16(a, b, c);
  } else {
    c = mma_f32(__uint_as_float(a.x), __uint_as_float(b.x), c);
    c = mma_f32(__uint_as_float(a.y), __uint_as_float(b.y), c);
    c = mma_f32(__uint_as_float(a.z), __uint_as_float(b.z), c);
    return mma_f32(__uint_as_float(a.w), __uint_as_float(b.w), c);
  }
}

// k's of one load step (16 bytes a lane, four quads) of dense weights
template <bool BF16>
constexpr int kDenseStep = BF16 ? 32 : 16;

// load steps of a row of K: dense, or 4-bit
template <int G, bool BF16>
__device__ __forceinline__ int row_steps(int K) {
  constexpr int step = G ? kQ4Chunk : kDenseStep<BF16>;
  return (K + step - 1) / step;
}

// Dense weights, steps [s0, s1) of the row, for the first nt tiles. U steps of W are in flight.
template <bool BF16, int T, int U, class L>
__device__ __forceinline__ void dense_part(const L& w, const char* const (&xp)[T], int nt, int K,
                                           int s0, int s1, f32x4_t (&acc)[T]) {
  constexpr int ESZ = BF16 ? 2 : 4, VE = 16 / ESZ, STEP = kDenseStep<BF16>;
  const int quad = (threadIdx.x & 63) >> 4;
  for (int s = s0; s < s1; s += U) {
    uint4 wv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s + u) * STEP + quad * VE;
      wv[u] = w((uint32_t)k * ESZ, s + u < s1 && k < K);
    }
#pragma unroll
    for (int t = 0; t < T; ++t) {
      if (t < nt) {
        uint4 xv[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = (s + u) * STEP + quad * VE;
          xv[u] = ld16_if(xp[t], (int64_t)k * ESZ, s + u < s1 && k < K);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) acc[t] = mma16<BF16>(wv[u], xv[u], acc[t]);
      }
    }
  }
}

// The offset that the 4-bit values carry into the products.
template <bool BF16>
constexpr float kQ4Offset = BF16 ? 16.f : 0.f;

// Swaps dwords between the quads: register j of quad q becomes register q of quad j.
__device__ __forceinline__ void transpose_quads(uint32_t (&r)[4]) {
  auto a = __builtin_amdgcn_permlane32_swap(r[0], r[2], false, false);
  auto b = __builtin_amdgcn_permlane32_swap(r[1], r[3], false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  r[0] = c[0];
  r[1] = c[1];
  r[2] = d[0];
  r[3] = d[1];
}

// Eight 4-bit values of a dword as bf16 16 + q, in the order k0 k4 k1 k5 k2 k6 k3 k7.
__device__ __forceinline__ uint4 q4_bf16(uint32_t w) {
  constexpr uint32_t kMask = 0x00780078u, kBase = 0x41804180u;  // 16.0 in both halves
  return make_uint4(((w << 3) & kMask) | kBase, ((w >> 1) & kMask) | kBase,
                    ((w >> 5) & kMask) | kBase, ((w >> 9) & kMask) | kBase);
}
// Eight bf16 of x in the same order.
__device__ __forceinline__ uint4 q4_order(const uint4& x) {
  return make_uint4(__builtin_amdgcn_perm(x.z, x.x, 0x05040100u),
                    __builtin_amdgcn_perm(x.z, x.x, 0x07060302u),
                    __builtin_amdgcn_perm(x.w, x.y, 0x05040100u),
                    __builtin_amdgcn_perm(x.w, x.y, 0x07060302u));
}

// x of one matrix-core step of 32 k's: 8 elements a lane
template <bool BF16>
struct X8 {
  uint4 a, b;  // fp32: elements 0-3 and 4-7; bf16: a alone, in the order of q4_bf16
  __device__ __forceinline__ void load(const char* p, int k, bool ok) {
    if constexpr (BF16) {
      a = q4_order(ld16_if(p, (int64_t)k * 2, ok));
    } else {
      a = ld16_if(p, (int64_t)k * 4, ok);
      b = ld16_if(p, (int64_t)k * 4 + 16, ok);
    }
  }
};

// One step of 32 k's: prod += (c + q) x, sum += x.
template <bool BF16>
__device__ __forceinline__ void q4_step(uint32_t w, const X8<BF16>& x, f32x4_t& prod,
                                        f32x4_t& sum) {
  if constexpr (BF16) {
    prod = mma_bf16(q4_bf16(w), x.a, prod);
    sum = mma_bf16(make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u), x.a, sum);
  } else {
    const uint32_t xs[8] = {x.a.x, x.a.y, x.a.z, x.a.w, x.b.x, x.b.y, x.b.z, x.b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      prod = mma_f32((float)((w >> (4 * j)) & 15u), __uint_as_float(xs[j]), prod);
      sum = mma_f32(1.f, __uint_as_float(xs[j]), sum);
    }
  }
}

// 4-bit weights, chunks [c0, c1) of the row, for the first nt tiles; sc: scale and c + z of
// [group][row] in LDS. K is a multiple of G.
template <int G, bool BF16, int T, int U, class L>
__device__ __forceinline__ void q4_part(const L& w, const char* const (&xp)[T], int nt, int K,
                                        int c0, int c1, const float2* sc, f32x4_t (&acc)[T]) {
  constexpr int SPG = G / 32;  // steps of a group
  const int quad = (threadIdx.x & 63) >> 4;
  for (int c = c0; c < c1; c += U) {
    uint4 wv[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      wv[u] = w((uint32_t)((c + u) * (kQ4Chunk / 2) + quad * 16),
                c + u < c1 && (c + u) * kQ4Chunk + quad * 32 < K);
#pragma unroll
    for (int t = 0; t < T; ++t) {
      if (t < nt) {
        X8<BF16> x[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = (c + u) * kQ4Chunk + j * 32;
            x[u][j].load(xp[t], k + quad * 8, c + u < c1 && k < K);
          }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          uint32_t r[4] = {wv[u].x, wv[u].y, wv[u].z, wv[u].w};
          transpose_quads(r);
#pragma unroll
          for (int g = 0; g < 4 / SPG; ++g) {
            const int k = (c + u) * kQ4Chunk + g * G;
            if (c + u < c1 && k < K) {
              f32x4_t prod = {0.f, 0.f, 0.f, 0.f}, sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int j = 0; j < SPG; ++j) q4_step<BF16>(r[g * SPG + j], x[u][g * SPG + j], prod, sum);
              const float2* s = sc + (k / G) * kTileRows + quad * 4;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 f = s[i];
                acc[t][i] = fmaf(f.x, fmaf(-f.y, sum[i], prod[i]), acc[t][i]);
              }
            }
          }
        }
      }
    }
  }
}

// A wave's part of a pass: steps [s0, s1) of dense or 4-bit rows.
template <int G, bool BF16, int T, class L>
__device__ __forceinline__ void weight_part(const L& w, const char* const (&xp)[T], int nt, int K,
                                            int s0, int s1, const float2* sc, f32x4_t (&acc)[T]) {
  if constexpr (G == 0) dense_part<BF16, T, 8>(w, xp, nt, K, s0, s1, acc);
  else q4_part<G, BF16, T, (T == 1 && BF16 ? 4 : 1)>(w, xp, nt, K, s0, s1, sc, acc);
}

// Scales and zero points of a tile's rows into LDS as [group][row] (scale, c + z); row_at(r) is
// the row's index in the scale table (of ng groups a row), negative for none.
template <bool BF16, class R>
__device__ __forceinline__ void stage_scales(float2* sc, const void* scales, const uint8_t* zeros,
                                             int ng, R row_at) {
  for (int i = threadIdx.x; i < kTileRows * ng; i += kThreads) {
    const int r = i / ng, g = i - r * ng;
    const int64_t row = row_at(r);
    float2 f = make_float2(0.f, 0.f);
    if (row >= 0) {
      const int64_t at = row * ng + g;
      f.x = BF16 ? __uint_as_float((uint32_t)((const uint16_t*)scales)[at] << 16)
                 : ((const float*)scales)[at];
      f.y = kQ4Offset<BF16> + (zeros ? (float)zeros[at] : 8.f);
    }
    sc[g * kTileRows + r] = f;
  }
}

// One pass over a tile of 16 weight rows and the pairs j0 .. j0 + 16 nt - 1 of a list: the four
// waves split the row's steps, their sums meet in LDS (red: kWaves * T * 256 floats), and
// epilogue(j, r, v) gets, on all 256 threads, entry j's value for tile row r. pair_at(j) is the
// pair of entry j, or negative. Ends with red free for the next pass.
template <int G, bool BF16, int T, class L, class P, class F>
__device__ __forceinline__ void tile_pass(const L& w, const void* x, int64_t ld_x,
                                          const FastDiv& row_div, int K, const float2* sc,
                                          P pair_at, int j0, int nt, float* red, F epilogue) {
  constexpr int ESZ = BF16 ? 2 : 4;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const char* xp[T];
  f32x4_t acc[T];
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const int p = t < nt ? pair_at(j0 + t * 16 + col) : -1;
    // an unused column reads some row of x: its results are not used
    xp[t] = (const char*)x + (p >= 0 ? (int64_t)fdiv(p, row_div) * ld_x * ESZ : 0);
    acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  const int steps = row_steps<G, BF16>(K);
  weight_part<G, BF16, T>(w, xp, nt, K, steps * wv / kWaves, steps * (wv + 1) / kWaves, sc, acc);
#pragma unroll
  for (int t = 0; t < T; ++t)
    if (t < nt)
      *reinterpret_cast<f32x4_t*>(red + (wv * T + t) * 256 + col * 16 + quad * 4) = acc[t];
  __syncthreads();
#pragma unroll
  for (int t = 0; t < T; ++t) {
    if (t < nt) {
      float v = 0.f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) v += red[(i * T + t) * 256 + threadIdx.x];
      epilogue(j0 + t * 16 + (int)(threadIdx.x >> 4), (int)(threadIdx.x & 15), v);
    }
  }
  __syncthreads();
}

template <bool BF16>
__device__ __forceinline__ void store_elem(void* out, int64_t i, float v) {
  if constexpr (BF16) ((uint16_t*)out)[i] = f32_to_bf16_rne(v);
  else ((float*)out)[i] = v;
}

}  // namespace
}  // namespace mol
