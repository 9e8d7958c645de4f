// Products of a few input rows with rows of a large weight matrix, on the matrix cores, shared
// by the 4-bit grouped GEMM and the whole-layer kernels (not installed).
//
//   acc[row, col] = sum_k W[row, k] x[col, k]     16 weight rows a wave, up to CW input rows
//
// The product is bound by reading W once, so it is laid out around that stream. Each wave owns
// a tile of 16 weight rows over the whole of K and keeps U loads of W in flight (16 bytes a lane:
// a row's four lanes read 64 contiguous bytes), straight into the A operand of a 16 x 16
// matrix-core tile; W never passes through LDS. The B operand, x, is staged in LDS by the four
// waves together, in the order the lanes read it, for the columns that exist. No sums cross
// waves, and the only barriers are around a stage of x. With one to three pairs most columns
// of the tile are unused, and the matrix cores still run far below their rate at the speed W
// arrives. Columns are independent: nothing in one pair's row (an infinity, a NaN) reaches
// another pair, and a column that is not staged is not read back.
// Lane l holds, of A and of B, row (column) l % 16 and the k's of quad l / 16; of the result,
// column l % 16 and rows 4 (l / 16) + i.
//
// Where x is computed in fp32 (the activation between the two stages), its bf16 form is two
// planes, hi + lo, each multiplied with W: 16 bits of it reach the product instead of 8.
//
// 4-bit weights: two per byte, the even k in the low half; value (q - z) * s with a scale s and a
// zero point z (8 without a table) per group of G consecutive k's. A load takes 128 k's. For G <
// 128 its dwords move between the quads (a 4 x 4 transpose), so that one matrix-core step covers
// 32 consecutive k's and no group is split over a step; for G = 128 the order of x follows the
// loads instead. In bf16, q goes into the top mantissa bits of 16.0, which is 16 + q exactly; in
// fp32, q is converted. The products with x are summed per group, and
//   sum_k (q - z) x = sum_k (q + c) x - (c + z) sum_k x,    c = 16 (bf16) or 0 (fp32)
// with sum_k x formed in fp32 while x is staged. Everything after the operands is fp32, and the
// scale is applied once per group. An infinite x makes both terms infinite, and a large one may take them
// past fp32's range: sums that are not finite at the end are formed again term by term (form_again).
#pragma once

#include "delta_common.h"

namespace mol {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kTileRows = 16;
constexpr int kWaves = kThreads / 64;
constexpr int kItemRows = kWaves * kTileRows;  // weight rows of a tile of each wave
constexpr int kMaxCols = 64;                   // columns of one pass, over the planes of x
constexpr int kXHalf = 16384;                  // bytes of a stage of x, in one of two buffers
constexpr int kQ4Load = 128;                   // k's of one load of 4-bit weights
template <int G>
constexpr int kMaxGroups = G == 128 ? 16 : 32;  // groups whose scales are staged at a time

__device__ __forceinline__ f32x4_t mma_bf16(const uint4& a, const uint4& b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a),
                                                 __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mma_f32(float a, float b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// one 16-byte vector a lane of each operand: 32 k's (bf16) or 16 (fp32)
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

// ---- 4-bit weights ----

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

// ---- x in LDS ----

// One 16-byte vector of x: its planes.
struct XVec {
  uint4 hi, lo;
};

// s + the sum of a vector's elements (bf16: products with 1.0, exact)
template <bool BF16>
__device__ __forceinline__ float vec_sum(const uint4& v, float s) {
  if constexpr (BF16) {
    constexpr uint32_t kOnes = 0x3f803f80u;
    return dot16<true>(v, make_uint4(kOnes, kOnes, kOnes, kOnes), s);
  } else {
    return s + ((__uint_as_float(v.x) + __uint_as_float(v.y)) +
                (__uint_as_float(v.z) + __uint_as_float(v.w)));
  }
}

// VE fp32 values as a vector of x: in bf16 as hi + lo, hi cut off rather than rounded (it cannot
// overflow, and the difference, below 2^-7 of it, is exact) and lo rounded: at most 2^-16 of the
// value is lost. An infinity has no lo.
template <bool BF16>
__device__ __forceinline__ XVec split_vec(const float (&f)[BF16 ? 8 : 4]) {
  if constexpr (BF16) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t u[2], r[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float v = f[2 * i + j];
        u[j] = __float_as_uint(v) & 0xffff0000u;
        r[j] = __builtin_isinf(v) ? 0u : f32_to_bf16_rne(v - __uint_as_float(u[j]));
      }
      h[i] = (u[0] >> 16) | u[1];
      l[i] = r[0] | (r[1] << 16);
    }
    return {make_uint4(h[0], h[1], h[2], h[3]), make_uint4(l[0], l[1], l[2], l[3])};
  } else {
    return {make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                       __float_as_uint(f[3])),
            make_uint4(0, 0, 0, 0)};
  }
}

// The shape of a stream: G the group of 4-bit weights (0: dense), CW columns, NP planes of x, KS
// the waves that share 16 rows and split their k's (1 or kWaves), MULTI whether a row of x takes
// several stages, UM the most loads of W in flight.
template <int G, bool BF16, int CW, int NP, int KS, bool MULTI, int UM>
struct Stream {
  static constexpr int VE = BF16 ? 8 : 4;                 // elements of a vector of x
  static constexpr int KL = G ? kQ4Load : 4 * VE;         // k's of a load of W
  static constexpr int LX = KL / (4 * VE);                // x steps (four vectors) of a load
  static constexpr int XS = kXHalf / (64 * CW * NP);      // x steps of a stage
  static constexpr int GPL = G ? kQ4Load / (G ? G : 1) : 0;  // groups of a load
  static constexpr int CLX = XS / LX;                     // loads of W whose x fits a stage
  static constexpr int CLG = G ? kMaxGroups<G> / (G ? GPL : 1) : CLX;  // and whose scales do
  static constexpr int CL = CLX < CLG ? CLX : CLG;
  static constexpr int Q = CL / KS;                       // of them, one wave's
  // a row of up to this many loads is staged at once, through both buffers
  static constexpr int ONE = G && 2 * CL > CLG ? CLG : 2 * CL;
  static constexpr int U = Q < UM ? Q : UM;               // a round of loads
  static constexpr int T = CW > 16 ? CW / 16 : 1;         // matrix-core tiles of columns
  static constexpr int PERIOD = LX % 4 ? 4 : 1;           // loads between equal x rotations
  static constexpr int PLANE = 2 * XS * 4 * CW;           // 16-byte slots of a plane (both buffers)
  static constexpr int NV = CL * KL / VE;                 // vectors of a column in a stage
  static constexpr int PER = (CW * NV + kThreads - 1) / kThreads;  // a thread's of a whole stage
  static_assert(Q >= 1 && U % PERIOD == 0 && (MULTI ? Q % U == 0 : U <= ONE),
                "a wave's part of a stage is whole rounds of loads");
  static_assert(KS == 1 || T == 1, "split k's: one tile of columns");
  static_assert((NV & (NV - 1)) == 0, "a stage's vectors are told apart by shifts");
};

// The scale and the offset c + z of a group in LDS. bf16: the scale's 16 bits over the offset as fp16
// (integers up to 271: exact), half the LDS of two floats.
template <bool BF16>
struct Q4Scale {
  float2 v;
  __device__ __forceinline__ float scale() const { return v.x; }
  __device__ __forceinline__ float offset() const { return v.y; }
  static __device__ __forceinline__ Q4Scale of(float scale, float offset) {
    return {make_float2(scale, offset)};
  }
};
template <>
struct Q4Scale<true> {
  uint32_t v;
  __device__ __forceinline__ float scale() const { return __uint_as_float(v & 0xffff0000u); }
  __device__ __forceinline__ float offset() const {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)v);
  }
  static __device__ __forceinline__ Q4Scale of(float scale, float offset) {
    return {__float_as_uint(scale) | __builtin_bit_cast(uint16_t, (_Float16)offset)};
  }
};

// Bytes of LDS: x, then sums of x per group and column, then each wave's scales.
template <int G, bool BF16>
struct StreamLds {
  // (a stage of CW columns and NP planes has kXHalf / (64 CW NP) x steps)
  static constexpr int kSums = G ? 2 * (kXHalf / 64 / (BF16 ? 4 : 8)) * (kQ4Load / (G ? G : 1)) * 4 : 0;
  static constexpr int kScales = G ? kWaves * kMaxGroups<G> * kTileRows * (int)sizeof(Q4Scale<BF16>) : 0;
  static constexpr int kBytes = 2 * kXHalf + kSums + kScales;
};

// 16-byte slot of x step `xs` (within the stage), quad, column: columns are rotated by the step
// so that both the staging writes (one column, consecutive k's) and the reads (all columns of a
// step) spread over the banks.
template <int CW>
__device__ __forceinline__ int x_rot(int xs, int quad) {  // has period 4 in xs
  return CW == 4 ? xs & 3 : CW == 8 ? ((xs * 4 + quad) >> 1) & 7 : (xs * 4 + quad) & 15;
}
template <int CW>
__device__ __forceinline__ int x_slot(int xs, int quad, int col) {
  return (xs * 4 + quad) * CW + (col ^ x_rot<CW>(xs, quad));
}

// Puts vector v of column c of a stage into LDS: planes at xs, sums of 4-bit groups at sums. The
// lanes of a group are consecutive, all of them here.
template <class S, int G, bool BF16, int CW, int NP>
__device__ __forceinline__ void put_x(uint4* xs, float* sums, int c, int v, const XVec& x) {
  constexpr int GV = G ? G / S::VE : 1;  // vectors of a group
  int step, quad;
  if constexpr (G == 0) {
    step = v >> 2;
    quad = v & 3;
  } else {
    constexpr int VD = 8 / S::VE;  // vectors of a dword of W (8 k's)
    const int d = v / VD;          // dword of the row
    const int j = G == 128 ? d & 3 : (d >> 2) & 3;
    quad = G == 128 ? (d >> 2) & 3 : d & 3;
    step = ((d >> 4) * 4 + j) * VD + v % VD;
  }
  const int at = x_slot<CW>(step, quad, c);
  if constexpr (G > 0 && BF16) {
    xs[at] = q4_order(x.hi);
    if constexpr (NP == 2) xs[S::PLANE + at] = q4_order(x.lo);
  } else {
    xs[at] = x.hi;
    if constexpr (NP == 2) xs[S::PLANE + at] = x.lo;
  }
  if constexpr (G > 0) {
    float sum = vec_sum<BF16>(x.hi, 0.f);
    if constexpr (NP == 2) sum = vec_sum<BF16>(x.lo, sum);
    sum = group_sum<GV>(sum);
    if ((v & (GV - 1)) == 0) sums[v / GV * CW + c] = sum;
  }
}

// The loads stay where they are issued: used here by all lanes, they cannot sink into the conditions
// of the stores, where each would be waited for on its own.
template <int NP, int N>
__device__ __forceinline__ void arrived(const XVec (&x)[N]) {
#pragma unroll
  for (int b = 0; b < N; ++b) {
    asm volatile("" ::"v"(x[b].hi.x), "v"(x[b].hi.y), "v"(x[b].hi.z), "v"(x[b].hi.w));
    if constexpr (NP == 2)
      asm volatile("" ::"v"(x[b].lo.x), "v"(x[b].lo.y), "v"(x[b].lo.z), "v"(x[b].lo.w));
  }
}

__device__ __forceinline__ uint4 vec_if(const uint4& v, bool ok) {
  return make_uint4(ok ? v.x : 0u, ok ? v.y : 0u, ok ? v.z : 0u, ok ? v.w : 0u);
}
template <int NP>
__device__ __forceinline__ XVec xvec_if(const XVec& x, bool ok) {
  return {vec_if(x.hi, ok), NP == 2 ? vec_if(x.lo, ok) : x.lo};
}

// A whole row of columns [0, ncol), ncol >= 1: src.row(c) is column c's row (c uniform), src(row,
// v) its vector v, an XVec whose lo counts for NP = 2. Units of 64 vectors of one column go round the
// waves, NB of them in flight; every load is issued, on clamped indices, so that no branch
// stands between loads. The row is filled up with zeros to whole rounds of loads (what a load of W
// past the row's end returns, times a stale infinity, would not be zero).
template <class S, int G, bool BF16, int CW, int NP, class Src>
__device__ __forceinline__ void stage_row(uint4* xs, float* sums, const Src& src, int ncol, int K,
                                          int tid) {
  constexpr int NB = NP == 2 ? 2 : 4;
  constexpr int VR = S::KL / S::VE * S::U;  // vectors of a round of loads
  const int vend = K / S::VE, nv = (vend + VR - 1) / VR * VR, nb = (nv + 63) >> 6;
  const int inv = 65536 / nb + 1;  // u / nb = u * inv >> 16 for these units (below 2^12)
  const int units = ncol * nb, lane = tid & 63;
  for (int unit = __builtin_amdgcn_readfirstlane(tid >> 6); unit < units; unit += NB * kWaves) {
    XVec x[NB];
    int c[NB], v[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int u = unit + b * kWaves;
      c[b] = (u * inv) >> 16;
      v[b] = (u - c[b] * nb) * 64 + lane;
      x[b] = src(src.row(min(c[b], ncol - 1)), min(v[b], vend - 1));
    }
    arrived<NP>(x);
#pragma unroll
    for (int b = 0; b < NB; ++b)
      if (c[b] < ncol && v[b] < nv)
        put_x<S, G, BF16, CW, NP>(xs, sums, c[b], v[b], xvec_if<NP>(x[b], v[b] < vend));
  }
}

// One of several stages, on its way through registers while the one before it is at work: vectors
// v0 .. v0 + S::NV - 1 of every column; src.lane_row(c) is column c's row, c of the lane's own.
template <class S, int G, bool BF16, int CW, int NP, class Src>
struct StageRegs {
  XVec x[S::PER];
  __device__ __forceinline__ void load(const Src& src, int ncol, int v0, int vend, int tid) {
#pragma unroll
    for (int b = 0; b < S::PER; ++b) {
      const int i = b * kThreads + tid, c = i / S::NV, v = v0 + i % S::NV;
      x[b] = src(src.lane_row(min(c, ncol - 1)), min(v, vend - 1));
    }
  }
  __device__ __forceinline__ void store(uint4* xs, float* sums, int ncol, int v0, int vend,
                                        int tid) {
    arrived<NP>(x);
#pragma unroll
    for (int b = 0; b < S::PER; ++b) {
      const int i = b * kThreads + tid, c = i / S::NV, v = i % S::NV;
      if (c < ncol)
        put_x<S, G, BF16, CW, NP>(xs, sums, c, v, xvec_if<NP>(x[b], v0 + v < vend));
    }
  }
};

// ---- the stream ----

// Scales and zero points of 4-bit weights.
struct Q4Tables {
  const void* scales;
  const uint8_t* zeros;
  int ng;  // groups of a row
};

// Where a weight row is: its byte offset in the matrix (kOutOfRange: there is none), and its row in
// the scale tables (negative: none).
struct RowAt {
  uint32_t off;
  int64_t srow;
};

// ---- sums that are not finite, term by term ----

// The elements of a vector of x, of its planes together (exact: 16 bits of them at most).
template <bool BF16, int NP>
__device__ __forceinline__ void x_elems(const XVec& x, float (&f)[BF16 ? 8 : 4]) {
  const uint32_t h[4] = {x.hi.x, x.hi.y, x.hi.z, x.hi.w}, l[4] = {x.lo.x, x.lo.y, x.lo.z, x.lo.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16) {
      f[2 * i] = NP == 2 ? bf16_lo(h[i]) + bf16_lo(l[i]) : bf16_lo(h[i]);
      f[2 * i + 1] = NP == 2 ? bf16_hi(h[i]) + bf16_hi(l[i]) : bf16_hi(h[i]);
    } else {
      f[i] = __uint_as_float(h[i]);
    }
  }
}

// Whether the row of x holds a NaN (a wave together).
template <bool BF16, int NP, class Src>
__device__ __forceinline__ bool holds_nan(const Src& src, const char* row, int K, int lane) {
  constexpr int VE = BF16 ? 8 : 4;
  bool nan = false;
  for (int v = lane; v < K / VE; v += 64) {
    float f[VE];
    x_elems<BF16, NP>(src(row, v), f);
#pragma unroll
    for (int i = 0; i < VE; ++i) nan |= f[i] != f[i];
  }
  return __builtin_amdgcn_ballot_w64(nan) != 0;
}

// sum_k W[k] x[k] by a wave, each weight formed first: (q - z) * s of 4-bit ones.
template <int G, bool BF16, int NP, class Src>
__device__ __forceinline__ float sum_of_terms(__amdgpu_buffer_rsrc_t rsrc, const RowAt& at,
                                              const Q4Tables& q, const Src& src, const char* row,
                                              int K, int lane) {
  constexpr int VE = BF16 ? 8 : 4, KU = G ? 32 : VE;  // k's of 16 bytes of W
  float sum = 0.f;
  for (int u = lane; u < K / KU; u += 64) {
    const uint4 wv = buf16(rsrc, at.off + (uint32_t)u * 16u);
    const uint32_t w[4] = {wv.x, wv.y, wv.z, wv.w};
    float s = 0.f, z = 8.f;
    if constexpr (G > 0) {
      const int64_t g = at.srow * q.ng + u * KU / G;
      s = BF16 ? __uint_as_float((uint32_t)((const uint16_t*)q.scales)[g] << 16)
               : ((const float*)q.scales)[g];
      if (q.zeros) z = (float)q.zeros[g];
    }
#pragma unroll
    for (int v = 0; v < KU / VE; ++v) {
      float f[VE];
      x_elems<BF16, NP>(src(row, u * (KU / VE) + v), f);
#pragma unroll
      for (int i = 0; i < VE; ++i) {
        float e;
        if constexpr (G > 0) e = ((float)((w[(v * VE + i) / 8] >> (4 * ((v * VE + i) % 8))) & 15u) - z) * s;
        else if constexpr (BF16) e = i % 2 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
        else e = __uint_as_float(w[i]);
        sum = fmaf(e, f[i], sum);
      }
    }
  }
  return group_sum<64>(sum);
}

// ---- the stream of weight rows ----

// Scales of a stage's groups on their way to LDS: this lane's row (lane % 16), every fourth group.
template <int G, bool BF16>
struct ScaleRegs {
  static constexpr int N = kMaxGroups<G> / 4;
  float s[N], z[N];
  __device__ __forceinline__ void load(const Q4Tables& q, int64_t row, int g0, int gn,
                                       int quad) {
    const int64_t at = (row >= 0 ? row : 0) * q.ng + g0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int g = min(i * 4 + quad, gn - 1);
      s[i] = BF16 ? __uint_as_float((uint32_t)((const uint16_t*)q.scales + at)[g] << 16)
                  : ((const float*)q.scales + at)[g];
      z[i] = 8.f;
    }
    if (q.zeros) {
#pragma unroll
      for (int i = 0; i < N; ++i) z[i] = (float)(q.zeros + at)[min(i * 4 + quad, gn - 1)];
    }
  }
  __device__ __forceinline__ void store(Q4Scale<BF16>* sc, int gn, int lane) const {
#pragma unroll
    for (int i = 0; i < N; ++i)  // groups past the row: a scale of zero
      sc[i * 64 + lane] = Q4Scale<BF16>::of(i * 4 + (lane >> 4) < gn ? s[i] : 0.f,
                                            kQ4Offset<BF16> + z[i]);
  }
};

// Runs one item against ncol columns: this wave's 16 rows, or with KS = kWaves the same rows in
// all waves, which split their k's. me: this lane's row (lane % 16); row_at(i): row i of the 16.
// epilogue(col, acc) gets, on every lane (of wave 0 for KS = kWaves), column col's sums of tile
// rows 4 * quad + i; only columns below ncol and rows that exist are meant. All four waves take
// part in the barriers; on return LDS may still be read by slower waves.
template <int G, bool BF16, int CW, int NP, int KS, bool MULTI, int UM, class Rows, class Src,
          class Epi>
__device__ __forceinline__ void stream_rows(char* lds, __amdgpu_buffer_rsrc_t rsrc,
                                            const RowAt& me, const Rows& row_at,
                                            const Q4Tables& q, const Src& src, int ncol, int K,
                                            bool staged, Epi epilogue) {
  using S = Stream<G, BF16, CW, NP, KS, MULTI, UM>;
  // (opaque to the compiler, which would otherwise compute every variant's addresses ahead of the
  // loop over passes and spill them)
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int loads = (K + S::KL - 1) / S::KL, vend = K / S::VE;
  // loads per stage, and this wave's part of them: one stage is split evenly
  int cl = S::CL, part = S::Q, first = 0;
  if constexpr (!MULTI) {
    part = ((loads + KS - 1) / KS + S::U - 1) / S::U * S::U;
    cl = part * KS;
  }
  if constexpr (KS > 1) first = wv * part;
  // every load is issued: past the row (and for rows that are not there) it reads zeros and
  // moves nothing
  const int k_left = K - quad * (S::KL / 4);  // k's from this lane's part of load 0 on
  const uint32_t lane_off = me.off + (uint32_t)quad * 16u;
  auto load = [&](int l) __attribute__((always_inline)) {
    return buf16(rsrc, l * S::KL < k_left ? lane_off + (uint32_t)l * 64u : kOutOfRange);
  };
  uint4 wr[S::U];
#pragma unroll
  for (int u = 0; u < S::U; ++u) wr[u] = load(first + u);
  f32x4_t acc[S::T];
#pragma unroll
  for (int t = 0; t < S::T; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // this lane's slots of x steps 0-3 (the rotation's period) relative to the step's first slot
  int slot[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) slot[i] = quad * CW + ((col & (CW - 1)) ^ x_rot<CW>(i, quad));
  uint4* const xs = reinterpret_cast<uint4*>(lds);
  float* const sums = reinterpret_cast<float*>(lds + 2 * kXHalf);
  using Scale = Q4Scale<BF16>;
  Scale* const sc = reinterpret_cast<Scale*>(lds + 2 * kXHalf + StreamLds<G, BF16>::kSums) +
                     (KS > 1 ? 0 : wv) * (kMaxGroups<G> * kTileRows);

  // the products of register u, in a round that starts at xb, sumb and scb
  auto products = [&](int u, const uint4* xb, const float* sumb, const Scale* scb)
                      __attribute__((always_inline)) {
    auto x_at = [&](int step, int t, int plane) __attribute__((always_inline)) {  // of the round
      return xb[slot[step & 3] + step * (4 * CW) + t * 16 + plane * S::PLANE];
    };
    if constexpr (G == 0) {
#pragma unroll
      for (int t = 0; t < S::T; ++t)
#pragma unroll
        for (int pl = 0; pl < NP; ++pl) acc[t] = mma16<BF16>(wr[u], x_at(u, t, pl), acc[t]);
    } else {
      constexpr int SPG = G / 32;  // dwords (steps of 32 k's) of a group
      uint32_t r[4] = {wr[u].x, wr[u].y, wr[u].z, wr[u].w};
      if constexpr (G < 128) transpose_quads(r);
#pragma unroll
      for (int g = 0; g < S::GPL; ++g) {
        f32x4_t prod[S::T];
#pragma unroll
        for (int t = 0; t < S::T; ++t) prod[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = g * SPG; j < (g + 1) * SPG; ++j) {
          if constexpr (BF16) {
            const uint4 a = q4_bf16(r[j]);
#pragma unroll
            for (int t = 0; t < S::T; ++t)
#pragma unroll
              for (int pl = 0; pl < NP; ++pl)
                prod[t] = mma_bf16(a, x_at(u * 4 + j, t, pl), prod[t]);
          } else {
#pragma unroll
            for (int t = 0; t < S::T; ++t) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint4 x = x_at((u * 4 + j) * 2 + h, t, 0);
                const uint32_t xe[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  prod[t] = mma_f32((float)((r[j] >> (16 * h + 4 * i)) & 15u),
                                    __uint_as_float(xe[i]), prod[t]);
              }
            }
          }
        }
        struct alignas(16) { Scale row[4]; } f;  // (one or two 16-byte reads)
        __builtin_memcpy(&f, __builtin_assume_aligned(scb + (u * S::GPL + g) * kTileRows, 16), sizeof f);
#pragma unroll
        for (int t = 0; t < S::T; ++t) {
          const float sx = sumb[(u * S::GPL + g) * CW + t * 16];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[t][i] = fmaf(f.row[i].scale(), fmaf(-f.row[i].offset(), sx, prod[t][i]), acc[t][i]);
        }
      }
    }
  };
  // a round: registers' loads b .. b + U - 1 of the stage at xs_, sums_, refilled from load `next` on
  auto round = [&](const uint4* xs_, const float* sums_, int b, int next)
                   __attribute__((always_inline)) {
    // (the offset is opaque to the compiler, which would otherwise keep an address register for
    // every access of the round)
    int o = b;
    asm volatile("" : "+s"(o));
    const uint4* xb = xs_ + o * (S::LX * 4 * CW);
    const float* sumb = sums_ + o * (S::GPL * CW) + (col & (CW - 1));
    const Scale* scb = sc + o * (S::GPL * kTileRows) + quad * 4;
#pragma unroll
    for (int u = 0; u < S::U; ++u) {
      products(u, xb, sumb, scb);
      wr[u] = load(next + u);
    }
  };

  ScaleRegs<G ? G : 32, BF16> regs;
  auto groups_at = [&](int l0) { return min(cl * S::GPL, q.ng - l0 * S::GPL); };
  if constexpr (G > 0) regs.load(q, me.srow, 0, groups_at(0), quad);
  if constexpr (!MULTI) {
    if (!staged) {
      __syncthreads();  // the columns' pairs are written down, and LDS is free
      stage_row<S, G, BF16, CW, NP>(xs, sums, src, ncol, K, tid);
    }
    // (this wave's own part of LDS; KS > 1: all waves write the same values)
    if constexpr (G > 0) regs.store(sc, groups_at(0), lane);
    if (!staged) __syncthreads();
    const int n = min(first + part, loads);
    for (int b = first; b < n; b += S::U)
      round(xs, sums, b, b + S::U < first + part ? b + S::U : loads);
  } else {
    // stages alternate between the two buffers; the next one's x and scales load while one works
    StageRegs<S, G, BF16, CW, NP, Src> stage;
    __syncthreads();  // the columns' pairs are written down, and LDS is free
    stage.load(src, ncol, 0, vend, tid);
    stage.store(xs, sums, ncol, 0, vend, tid);
    int buf = 0;
    for (int l0 = 0; l0 < loads; l0 += S::CL, buf ^= 1) {
      if constexpr (G > 0) regs.store(sc, groups_at(l0), lane);
      __syncthreads();
      const int l1 = l0 + S::CL, v1 = l1 * (S::KL / S::VE);
      const bool more = l1 < loads;
      int t1 = tid;  // (opaque again: addresses are computed anew for each stage, not kept)
      asm volatile("" : "+v"(t1));
      if (more) {
        if constexpr (G > 0) regs.load(q, me.srow, l1 * S::GPL, groups_at(l1), (t1 & 63) >> 4);
        stage.load(src, ncol, v1, vend, t1);
      }
      const uint4* xh = xs + buf * (S::XS * 4 * CW);
      const float* sh = sums + buf * (S::CLX * S::GPL * CW);
#pragma unroll 1
      for (int b = 0; b < S::Q; b += S::U)
        round(xh, sh, first + b, b + S::U < S::Q ? l0 + first + b + S::U : l1 + first);
      if (more)
        stage.store(xs + (buf ^ 1) * (S::XS * 4 * CW), sums + (buf ^ 1) * (S::CLX * S::GPL * CW), ncol,
                    v1, vend, t1);
      // (KS > 1: the waves share the scales, which the next turn stores)
      if constexpr (G > 0 && KS > 1) __syncthreads();
    }
  }
  if constexpr (KS > 1) {
    __syncthreads();
    f32x4_t* red = reinterpret_cast<f32x4_t*>(lds);
    red[wv * 64 + lane] = acc[0];
    __syncthreads();
    if (wv != 0) return;
#pragma unroll
    for (int i = 1; i < kWaves; ++i) acc[0] += red[i * 64 + lane];
  }
#pragma unroll
  for (int t = 0; t < S::T; ++t) epilogue(t * 16 + col, acc[t]);

  // Sums that are not finite once more, each from its terms, and out again over the first: an infinite x, an
  // infinite weight beside a second plane of zeros, or a sum past fp32's range on the way, then gives what
  // the definition gives. Columns whose x holds a NaN are left: all their sums are NaN. Where
  // all is finite the look does not show (4-bit gate/up of 128 tokens 57 us with and without; groups of 32
  // lose up to 3 % to registers in scratch); half of the rows with a NaN 92 us, with an infinity 557.
  if constexpr (G > 0 || NP == 2) {
    bool odd = false;
#pragma unroll
    for (int t = 0; t < S::T; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) odd |= t * 16 + col < ncol && !__builtin_isfinite(acc[t][i]);
    if (!__builtin_amdgcn_ballot_w64(odd)) return;
#pragma unroll 1
    for (int c = 0; c < ncol; ++c) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = acc[0][i];
#pragma unroll
        for (int t = 1; t < S::T; ++t) v[i] = c >> 4 == t ? acc[t][i] : v[i];
      }
      uint32_t rows = 0;  // those of the tile to form again
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t m = __builtin_amdgcn_ballot_w64(!__builtin_isfinite(v[i])) >> (c & 15);
        rows |= ((uint32_t)(m & 1) | (uint32_t)(m >> 16 & 1) << 4 | (uint32_t)(m >> 32 & 1) << 8 |
                 (uint32_t)(m >> 48 & 1) << 12) << i;
      }
      if (rows == 0) continue;
      const char* x = src.row(c);
      if (holds_nan<BF16, NP>(src, x, K, lane)) continue;
#pragma unroll 1
      for (; rows; rows &= rows - 1) {
        const int r = __builtin_ctz(rows);
        const RowAt at = row_at(r);
        if (at.off == kOutOfRange) continue;
        const float sum = sum_of_terms<G, BF16, NP>(rsrc, at, q, src, x, K, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = quad * 4 + i == r ? sum : v[i];
      }
      epilogue(col == (c & 15) ? c : ncol, f32x4_t{v[0], v[1], v[2], v[3]});
    }
  }
}

// The most columns of a pass.
template <int G, bool BF16, int NP, int KS>
constexpr int kPassCols = KS > 1 ? 8 : (G && !BF16) || NP == 2 ? 32 : kMaxCols;

// The stream of a row of K: staged at once where its x fits both buffers, else in several stages.
// Loads of W in flight: as many as the registers allow (4-bit: each load's products take many of
// them; fewer beside the next stage's x), and six where the row has five or six (4-bit down of 23
// tokens in rounds of four and in one of six: K 768, groups of 64 36.5 and 30.1 us, of 128 28.0 and 22.7;
// K 640, groups of 128 25.1 and 20.3).
template <int G, bool BF16, int CW, int NP, int KS, class Rows, class Src, class Epi>
__device__ __forceinline__ void stream_k(char* lds, __amdgpu_buffer_rsrc_t rsrc, const RowAt& me,
                                         const Rows& row_at, const Q4Tables& q, const Src& src,
                                         int ncol, int K, bool staged, Epi epi) {
  constexpr int UM = G == 0 || G == 128 ? 8 : G == 64 ? 4 : 2;
  using S = Stream<G, BF16, CW, NP, KS, false, UM>;
  if constexpr (CW <= 16) {
    if constexpr (G >= 64 && BF16 && KS == 1 && S::ONE >= 6) {
      if (K > 4 * kQ4Load && K <= 6 * kQ4Load) {
        stream_rows<G, BF16, CW, NP, KS, false, 6>(lds, rsrc, me, row_at, q, src, ncol, K, staged, epi);
        return;
      }
    }
    if (K <= S::ONE * S::KL) {
      stream_rows<G, BF16, CW, NP, KS, false, UM>(lds, rsrc, me, row_at, q, src, ncol, K, staged, epi);
      return;
    }
  }
  stream_rows<G, BF16, CW, NP, KS, true, (G ? 2 : 8)>(lds, rsrc, me, row_at, q, src, ncol, K, false,
                                                      epi);
}

// As many columns as the pass has: 4, 8, 16, 32 or 64. A narrow pass leaves room in LDS for longer rows
// of x in one stage; passes of 64 read a weight once where 16 would read it four times (layer of 128
// tokens, popular experts: 308 us with passes of 64 and the second buffer of x, 325 without either).
template <int G, bool BF16, int NP, int KS, class Rows, class Src, class Epi>
__device__ __forceinline__ void stream_cols(char* lds, __amdgpu_buffer_rsrc_t rsrc,
                                            const RowAt& me, const Rows& row_at,
                                            const Q4Tables& q, const Src& src, int ncol, int K,
                                            bool staged, Epi epi) {
  constexpr int MOST = kPassCols<G, BF16, NP, KS>;
  if (ncol <= 4) {
    stream_k<G, BF16, 4, NP, KS>(lds, rsrc, me, row_at, q, src, ncol, K, staged, epi);
  } else if (MOST == 8 || ncol <= 8) {
    stream_k<G, BF16, 8, NP, KS>(lds, rsrc, me, row_at, q, src, ncol, K, staged, epi);
  } else if constexpr (MOST > 8) {
    if (ncol <= 16)
      stream_k<G, BF16, 16, NP, 1>(lds, rsrc, me, row_at, q, src, ncol, K, staged, epi);
    else if (MOST == 32 || ncol <= 32)
      stream_k<G, BF16, 32, NP, 1>(lds, rsrc, me, row_at, q, src, ncol, K, staged, epi);
    else if constexpr (MOST > 32)
      stream_k<G, BF16, 64, NP, 1>(lds, rsrc, me, row_at, q, src, ncol, K, staged, epi);
  }
}

// A work item is `tiles` times 64 rows, 16 a wave and tile, or (KS = kWaves) 16 for all. The first
// row of this wave in the tile that begins at row n0:
template <int KS>
__device__ __forceinline__ int wave_row0(int n0) {
  return KS > 1 ? n0 : n0 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * kTileRows;
}

// bytes of one weight row of K elements
template <int G, bool BF16>
__device__ __forceinline__ int64_t row_bytes(int K) {
  return G ? K / 2 : (int64_t)K * (BF16 ? 2 : 4);
}

// Input rows as they are in memory.
struct RowSrc {
  const char* x;
  int64_t ld_bytes;
  const int* pair;  // of each column (LDS)
  FastDiv row_div;
  __device__ __forceinline__ const char* row(int col) const {
    return x + (int64_t)fdiv(__builtin_amdgcn_readfirstlane(pair[col]), row_div) * ld_bytes;
  }
  __device__ __forceinline__ const char* lane_row(int col) const {
    return x + (int64_t)fdiv(pair[col], row_div) * ld_bytes;
  }
  __device__ __forceinline__ XVec operator()(const char* row, int v) const {
    return {ld16(row + (uint32_t)v * 16u), make_uint4(0, 0, 0, 0)};
  }
};

// The activation h of the pairs, from a row's first byte: bf16 as two planes of I elements, or fp32.
template <bool BF16>
struct PlaneSrc {
  int I;
  __device__ __forceinline__ XVec operator()(const char* row, int v) const {
    const uint4 hi = ld16(row + (uint32_t)v * 16u);
    return {hi, BF16 ? ld16(row + (uint32_t)I * 2u + (uint32_t)v * 16u) : hi};
  }
};

// silu(g) = g / (1 + exp(-g)), within 2^-20 of itself (2^-126 where it is below the normal numbers): the
// hardware's exp2 of t = -g log2(e), corrected by what the product with log2(e) rounds away, and its
// reciprocal. From t = 126 on the 1 is lost beside exp(-g), whose reciprocal leaves the normal numbers before
// g exp(g) does: that is formed from 2^(64 - t), scaled at the end (0 from t = 256 on, NaN at -infinity).
__device__ __forceinline__ float silu(float g) {
  constexpr float kL = 1.44269502f, kLlo = 1.92596303e-8f, kLn2 = 0.693147182f;
  const float t = -g * kL;
  const float lost = fmaf(-g, kLlo, fmaf(-g, kL, -t)) * kLn2;
  const bool far = !(t < 126.f);
  const float e = __builtin_amdgcn_exp2f(far ? 64.f - t : t);
  const float c = fmaf(e, far ? -lost : lost, e);
  const float x = t > -126.f && t < 256.f ? c : far ? 0.f : e;  // (0 and infinity stay as they are)
  return far ? g * x * 0x1p-64f : g * __builtin_amdgcn_rcpf(1.f + x);
}

template <bool BF16>
__device__ __forceinline__ void store_elem(void* out, int64_t i, float v) {
  if constexpr (BF16) ((uint16_t*)out)[i] = f32_to_bf16_rne(v);
  else ((float*)out)[i] = v;
}

}  // namespace
}  // namespace mol
