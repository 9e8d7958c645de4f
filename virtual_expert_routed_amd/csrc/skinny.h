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
// scale is applied once per group.
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
constexpr int kXBytes = 32768;                 // x staged at a time (four workgroups a CU)
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

// One 16-byte vector of x: its planes, and the fp32 sum of its elements (4-bit weights).
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
// overflow, and the difference is exact) and lo rounded: 2^-17 of the value is lost. An infinity
// has no lo.
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
// the waves that share 16 rows and split their k's (1 or kWaves).
template <int G, bool BF16, int CW, int NP, int KS>
struct Stream {
  static constexpr int VE = BF16 ? 8 : 4;                 // elements of a vector of x
  static constexpr int KL = G ? kQ4Load : 4 * VE;         // k's of a load of W
  static constexpr int LX = KL / (4 * VE);                // x steps (four vectors) of a load
  static constexpr int XS = kXBytes / (64 * CW * NP);     // x steps staged at a time
  static constexpr int CLX = XS / LX;                     // loads of W whose x fits a stage
  static constexpr int CLG = G ? kMaxGroups<G> * G / kQ4Load : CLX;  // and whose scales do
  static constexpr int CL = CLX < CLG ? CLX : CLG;
  static constexpr int Q = CL / KS;                       // of them, one wave's
  static constexpr int UM = G == 0 || G == 128 ? 8 : G == 64 ? 4 : 2;
  static constexpr int U = Q < UM ? Q : UM;               // loads of W in flight: a round
  static constexpr int T = CW > 16 ? CW / 16 : 1;         // matrix-core tiles of columns
  static constexpr int PERIOD = LX % 4 ? 4 : 1;           // loads between equal x rotations
  static_assert(Q >= 1 && Q % U == 0 && Q % PERIOD == 0 && U % PERIOD == 0,
                "a wave's part of a stage is whole rounds of loads");
  static_assert(KS == 1 || T == 1, "split k's: one tile of columns");
};

// Bytes of LDS: x, then sums of x per group and column, then each wave's scales.
template <int G>
struct StreamLds {
  static constexpr int kSums = G ? kMaxGroups<G> * 16 * 4 : 0;
  static constexpr int kScales = G ? kWaves * kMaxGroups<G> * kTileRows * 8 : 0;
  static constexpr int kBytes = kXBytes + kSums + kScales;
};

// 16-byte slot of x step `xs` (within the stage), quad, column: columns are rotated by the step
// so that both the staging writes (one column, consecutive k's) and the reads (all columns of a
// step) spread over the banks.
template <int CW>
__device__ __forceinline__ int x_rot(int xs, int quad) {  // has period 4 in xs
  return CW == 8 ? ((xs * 4 + quad) >> 1) & 7 : (xs * 4 + quad) & 15;
}
template <int CW>
__device__ __forceinline__ int x_slot(int xs, int quad, int col) {
  return (xs * 4 + quad) * CW + (col ^ x_rot<CW>(xs, quad));
}

// Stages columns [0, ncol) (ncol >= 1) of x for loads [l0, l0 + cl): src.row(c) is column c's
// row (uniform), src(row, v) its vector v (v < K / VE), an XVec whose lo counts for NP = 2. Units
// of 64 vectors of one column go round the waves, NB of them in flight: load() takes the first
// ones, store() puts them in LDS and goes on with the rest. Every load is issued, on clamped
// indices, so that no branch stands between loads.
template <class S, int G, bool BF16, int CW, int NP, class Src>
struct StageX {
  static constexpr int GV = G ? G / S::VE : 1;  // vectors of a group
  static constexpr int NB = NP == 2 ? 2 : 4;
  static constexpr int VL = S::KL / S::VE;      // vectors of a load
  const Src& src;
  int ncol, lane, v0, vend, nv, nb, inv, unit;
  XVec x[NB];

  __device__ __forceinline__ StageX(const Src& src_, int ncol_, int K, int l0, int cl, int tid)
      : src(src_), ncol(ncol_), lane(tid & 63) {
    v0 = l0 * VL;
    vend = K / S::VE;
    // the row is filled up with zeros to whole rounds of loads (what a load past the row's end
    // returns, times a stale infinity, would not be zero)
    constexpr int VR = VL * S::U;
    nv = min(cl * VL, (vend - v0 + VR - 1) / VR * VR);
    nb = (nv + 63) >> 6;
    inv = 65536 / nb + 1;  // u / nb = u * inv >> 16 for the units of a stage (below 2^12)
    unit = __builtin_amdgcn_readfirstlane(tid >> 6);
  }
  __device__ __forceinline__ int column(int u) const { return (u * inv) >> 16; }
  __device__ __forceinline__ int vector(int u) const {
    return (u - column(u) * nb) * 64 + lane;
  }
  __device__ __forceinline__ void load() {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int u = unit + b * kWaves;
      const int c = column(u), v = v0 + vector(u);
      x[b] = src(src.row(min(c, ncol - 1)), min(v, vend - 1));
    }
  }
  // The loads stay where they are issued: used here by all lanes, they cannot sink into store()'s
  // conditions, where each would be waited for on its own.
  __device__ __forceinline__ void arrived() const {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      asm volatile("" ::"v"(x[b].hi.x), "v"(x[b].hi.y), "v"(x[b].hi.z), "v"(x[b].hi.w));
      if constexpr (NP == 2)
        asm volatile("" ::"v"(x[b].lo.x), "v"(x[b].lo.y), "v"(x[b].lo.z), "v"(x[b].lo.w));
    }
  }
  __device__ __forceinline__ void store(char* lds) {
    uint4* xs = reinterpret_cast<uint4*>(lds);
    float* sums = reinterpret_cast<float*>(lds + kXBytes);
    const int units = ncol * nb;
    for (;;) {
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int u = unit + b * kWaves;
        const int c = column(u), v = vector(u);
        if (c < ncol && v < nv) {
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
          if (v0 + v >= vend) x[b] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
          if constexpr (G > 0 && BF16) {
            xs[at] = q4_order(x[b].hi);
            if constexpr (NP == 2) xs[S::XS * 4 * CW + at] = q4_order(x[b].lo);
          } else {
            xs[at] = x[b].hi;
            if constexpr (NP == 2) xs[S::XS * 4 * CW + at] = x[b].lo;
          }
          if constexpr (G > 0) {  // the lanes of a group are consecutive, all of them here
            float sum = vec_sum<BF16>(x[b].hi, 0.f);
            if constexpr (NP == 2) sum = vec_sum<BF16>(x[b].lo, sum);
            sum = group_sum<GV>(sum);
            if ((v & (GV - 1)) == 0) sums[v / GV * CW + c] = sum;
          }
        }
      }
      unit += NB * kWaves;
      if (unit >= units) break;
      load();
      arrived();
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
  __device__ __forceinline__ void store(float2* sc, int gn, int lane) const {  // scale, (c + z) * scale
#pragma unroll
    for (int i = 0; i < N; ++i) {  // groups past the row: zeros
      const float f = i * 4 + (lane >> 4) < gn ? s[i] : 0.f;
      sc[i * 64 + lane] = make_float2(f, f * (kQ4Offset<BF16> + z[i]));
    }
  }
};

// Runs one item against ncol staged columns: `tiles` tiles of this wave, one after another (KS = 1),
// the same x serving all of them when a row's x fits one stage; with KS = kWaves the waves have
// the same rows and split their k's. off(t): this lane's row of tile t (lane % 16) as a byte
// offset into the matrix, kOutOfRange for none; row_at(t): its row in the scale tables, negative
// for none. epilogue(t, col, acc) gets, on every lane (of wave 0 for KS = kWaves), column
// col's sums of tile rows 4 * quad + i; only columns below ncol and rows that exist are
// meant. All four waves take part in the barriers; on return LDS may still be read by slower
// waves.
template <int G, bool BF16, int CW, int NP, int KS, class Off, class Src, class RowAt, class Epi>
__device__ __forceinline__ void stream_rows(char* lds, __amdgpu_buffer_rsrc_t rsrc, Off off,
                                            int tiles, const Q4Tables& q, RowAt row_at,
                                            const Src& src, int ncol, int K, Epi epilogue) {
  using S = Stream<G, BF16, CW, NP, KS>;
  // (opaque to the compiler, which would otherwise compute every variant's addresses ahead of the
  // loop over passes and spill them)
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int loads = (K + S::KL - 1) / S::KL;
  // loads per stage, and this wave's part of them: one stage is split evenly
  int cl = S::CL, part = S::Q, first = 0;
  const bool one_stage = loads <= S::CL;
  if (one_stage) {
    part = ((loads + KS - 1) / KS + S::U - 1) / S::U * S::U;
    cl = part * KS;
  }
  if constexpr (KS > 1) first = wv * part;
  // every load is issued: past the row (and for rows that are not there) it reads zeros and
  // moves nothing
  const int k_left = K - quad * (S::KL / 4);  // k's from this lane's part of load 0 on
  auto load = [&](uint32_t row_off, int l) {
    return buf16(rsrc, l * S::KL < k_left ? row_off + (uint32_t)quad * 16u + (uint32_t)l * 64u
                                          : kOutOfRange);
  };
  uint32_t here = off(0), next = tiles > 1 ? off(1) : kOutOfRange;
  uint4 wr[S::U];
#pragma unroll
  for (int u = 0; u < S::U; ++u) wr[u] = load(here, first + u);
  f32x4_t acc[S::T];
  // this lane's slots of x steps 0-3 (the rotation's period) relative to the step's first slot
  int slot[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) slot[i] = quad * CW + ((col & (CW - 1)) ^ x_rot<CW>(i, quad));
  const uint4* xs = reinterpret_cast<const uint4*>(lds);
  const float* sums = reinterpret_cast<const float*>(lds + kXBytes) + (col & (CW - 1));
  float2* sc = reinterpret_cast<float2*>(lds + kXBytes + StreamLds<G>::kSums) +
               (KS > 1 ? 0 : wv) * (kMaxGroups<G> * kTileRows);
  constexpr int GPL = G ? kQ4Load / (G ? G : 1) : 0;  // groups of a load

  // the products of register u, in a round that starts at xb, sumb and scb
  auto products = [&](int u, const uint4* xb, const float* sumb, const float2* scb) {
    auto x_at = [&](int step, int t, int plane) {  // step within the round
      return xb[slot[step & 3] + step * (4 * CW) + t * 16 + plane * (S::XS * 4 * CW)];
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
      for (int g = 0; g < GPL; ++g) {
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
        float2 f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = scb[(u * GPL + g) * kTileRows + i];
#pragma unroll
        for (int t = 0; t < S::T; ++t) {
          const float sx = sumb[(u * GPL + g) * CW + t * 16];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[t][i] = fmaf(-f[i].y, sx, fmaf(f[i].x, prod[t][i], acc[t][i]));
        }
      }
    }
  };

  ScaleRegs<G ? G : 32, BF16> regs;
  for (int tile = 0; tile < tiles; ++tile) {
#pragma unroll
    for (int t = 0; t < S::T; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int l0 = 0; l0 < loads; l0 += cl) {
      const int g0 = l0 * GPL, gn = G ? min(cl * GPL, q.ng - g0) : 0;
      if (!one_stage || tile == 0) {
        __syncthreads();
        StageX<S, G, BF16, CW, NP, Src> stage(src, ncol, K, l0, cl, tid);
        if constexpr (G > 0) regs.load(q, row_at(tile), g0, gn, quad);
        stage.load();
        stage.arrived();
        if constexpr (G > 0) regs.store(sc, gn, lane);  // (KS > 1: all waves the same values)
        stage.store(lds);
        __syncthreads();
      } else if constexpr (G > 0) {
        regs.store(sc, gn, lane);  // loaded while the last tile ran; this wave's own part of LDS
      }
      if constexpr (G > 0) {
        if (one_stage && tile + 1 < tiles) regs.load(q, row_at(tile + 1), g0, gn, quad);
      }
      // this wave's loads of the stage, first .. n - 1, in whole rounds
      const int n = min(first + part, loads - l0);
      for (int b = first; b < n; b += S::U) {
        // (the offset is opaque to the compiler, which would otherwise keep an address register
        // for every access of the round)
        int o = b;
        asm volatile("" : "+s"(o));
        const uint4* xb = xs + o * (S::LX * 4 * CW);
        const float* sumb = sums + o * (GPL * CW);
        const float2* scb = sc + o * (GPL * kTileRows) + quad * 4;
        // the registers go on with the next round, the next stage or the next tile
        const bool on = b + S::U < first + part, more = l0 + cl < loads;
        const uint32_t ro = on || more ? here : next;
        const int lo = on ? l0 + b + S::U : more ? l0 + cl + first : first;
#pragma unroll
        for (int u = 0; u < S::U; ++u) {
          products(u, xb, sumb, scb);
          wr[u] = load(ro, lo + u);
        }
      }
    }
    here = next;
    if (tile + 2 < tiles) next = off(tile + 2);
    if constexpr (KS > 1) {
      __syncthreads();
      f32x4_t* red = reinterpret_cast<f32x4_t*>(lds);
      red[wv * 64 + lane] = acc[0];
      __syncthreads();
      if (wv != 0) return;  // (one tile)
#pragma unroll
      for (int i = 1; i < kWaves; ++i) acc[0] += red[i * 64 + lane];
    }
#pragma unroll
    for (int t = 0; t < S::T; ++t) epilogue(tile, t * 16 + col, acc[t]);
  }
}

// The most columns of a pass.
template <int NP, int KS>
constexpr int kPassCols = KS > 1 ? 16 : kMaxCols / NP;

// As many columns as the pass has: 8 (twice the k's per stage), 16, 32 or 64.
template <int G, bool BF16, int NP, int KS, class Off, class Src, class RowAt, class Epi>
__device__ __forceinline__ void stream_cols(char* lds, __amdgpu_buffer_rsrc_t rsrc, Off off,
                                            int tiles, const Q4Tables& q, RowAt row_at,
                                            const Src& src, int ncol, int K, Epi epi) {
  if (ncol <= 8) {
    stream_rows<G, BF16, 8, NP, KS>(lds, rsrc, off, tiles, q, row_at, src, ncol, K, epi);
  } else if (KS > 1 || ncol <= 16) {
    stream_rows<G, BF16, 16, NP, KS>(lds, rsrc, off, tiles, q, row_at, src, ncol, K, epi);
  } else if constexpr (KS == 1) {
    if (NP == 2 || ncol <= 32)
      stream_rows<G, BF16, 32, NP, 1>(lds, rsrc, off, tiles, q, row_at, src, ncol, K, epi);
    else if constexpr (NP == 1)
      stream_rows<G, BF16, 64, NP, 1>(lds, rsrc, off, tiles, q, row_at, src, ncol, K, epi);
  }
}

// Rows of a work item of `tiles` tiles a wave, and the first row of this wave's tile t in an item
// that begins at row n0: a tile's rows are kItemRows apart, or (KS = kWaves) 16 rows for all.
inline int item_rows(bool split, int tiles) { return split ? kTileRows : kItemRows * tiles; }
template <int KS>
__device__ __forceinline__ int tile_row0(int n0, int t) {
  return KS > 1 ? n0
                : n0 + t * kItemRows + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * kTileRows;
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
  __device__ __forceinline__ XVec operator()(const char* row, int v) const {
    return {ld16(row + (uint32_t)v * 16u), make_uint4(0, 0, 0, 0)};
  }
};

// silu(g) = g / (1 + exp(-g)), to about 2^-22: the hardware's exp2 of -g log2(e), corrected by what
// the product with log2(e) rounds away, and its reciprocal.
__device__ __forceinline__ float silu(float g) {
  constexpr float kL = 1.44269502f, kLlo = 1.92596303e-8f, kLn2 = 0.693147182f;
  const float t = -g * kL;
  const float lost = fmaf(-g, kLlo, fmaf(-g, kL, -t)) * kLn2;
  const float e = __builtin_amdgcn_exp2f(t);
  const float x = fabsf(t) < 126.f ? fmaf(e, lost, e) : e;  // (0 and infinity stay as they are)
  return g * __builtin_amdgcn_rcpf(1.f + x);
}

template <bool BF16>
__device__ __forceinline__ void store_elem(void* out, int64_t i, float v) {
  if constexpr (BF16) ((uint16_t*)out)[i] = f32_to_bf16_rne(v);
  else ((float*)out)[i] = v;
}

}  // namespace
}  // namespace mol
