// The base MoE grouped GEMM of a stage over microscaled 4-bit weights (mx4.h has the format):
//   out[p, n] = round( sum_k W[t, n, k] x[p / row_div, k] )
// for every pair p whose base expert t is local; other rows are untouched. x is rows of codes with
// scales of their own, or bf16 or fp32. Routed like the dense grouped GEMM (the aligned blocks of one
// base expert each).
//
// Codes times codes go to the scaled matrix-core product (16 x 16 x 128, both operands 4 bits, a scale
// byte a lane); beside bf16 and fp32 rows the weights are widened to that type in registers, scale
// included, which is exact below 2^128 and infinite from there on (codes at s = 253 and 254). Products and
// sums are fp32, so infinities and NaN of x reach exactly the sums that the formula has them in.
//
// A work item is a span of columns of a routing block (of the wide, spread and split forms; all of the block's of
// the narrow one) and NW times 16 FR weight rows; wave w has 16 FR of them as the A operand, straight from memory into
// registers: lane l holds row l % 16 and whole blocks of 32 k's, which block of a step being free as long as
// x agrees. x goes through LDS for all waves, as it lies in memory: direct-to-LDS loads, whose lanes choose
// their 16 bytes of a row so that the reads of a fragment (16 columns at one place of their rows) spread over
// the banks. Stages of x alternate between two buffers, the next one loading while one is at work; a weight
// register is filled again as soon as it has been used. A row's scales come by 2048 k's (1024 beside bf16
// and fp32 rows) through LDS: a scale byte a lane loaded from memory beside its codes took as many look-ups
// of the L1 as the codes.
//
// Kernel times (rocprofv3) and what bounds them, K 2048 and N 1536 (gate_up) or K 768 and N 2048 (down), top 8 of
// 128 experts, a copy's 4.94 TB/s. First over one set of buffers, which the last-level cache holds a part of, then over three in
// turn:
//   1 token, bf16 rows, gate_up               8.7 and 9.3 us  13.4 MB in 2.7: launch, routing, one latency after another
//   23 tokens, codes, down                   18 us     83 MB of weights, 94 % of the copy's rate
//   128 tokens, zipf, bf16 rows, gate_up     47 and 56 us  200 MB, 86 and 72 %
//   4096 tokens, codes, gate_up             114 and 134 us  1.8 PFLOP/s (the bytes alone: 64)
//   4096 tokens, bf16 rows, down            132 and 155 us  0.78 PFLOP/s of bf16, 70 % of the library's square product
//   16384 tokens, codes, down               272 and 340 us  1.5 PFLOP/s; a third of it the stores of 537 MB
//   4096 tokens, fp32 rows, gate_up        1900 us    108 TFLOP/s, 71 % of the library's square product
// Counters of one launch of the two wide ones over codes: look-ups of the L1 in 65 and 73 % of its cycles, the matrix cores
// busy in 20 and 19 %, waves waiting half their time. W as the A operand costs 64 look-ups a load (16 rows, four
// 16-byte places of each). Both operands through LDS, three stages deep, took as long (129 and 308 us for 4096
// gate_up and 16384 down where this took 130 and 307),
// so the form with fewer barriers stayed; workgroups that stay and take item after item 155 and 363; 256 columns
// an item 138 and 306 against 113 and 275.
//
// Of the result, lane l holds column (pair) l % 16 and rows 4 (l / 16) + i.
#pragma once

#include <type_traits>

#include "bf16_pair.h"
#include "mx4.h"

namespace mol {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

// What stands for k's past a row's end: x reads these zeros.
__device__ const uint4 kMxZeros[1] = {{0u, 0u, 0u, 0u}};

// Shape of a kernel. XF: the rows of x; TC columns a pass; FR times 16 weight rows a wave; SU units a
// stage (and wave); NW waves; KS: the waves share 16 FR rows and split the units (KS = NW), or 1.
template <int XF, int TC, int FR, int SU, int NW, int KS>
struct MxShape {
  static constexpr int THREADS = 64 * NW;
  static constexpr int S = XF == kMxRowsCodes ? 2 : 1;  // blocks a lane has of a unit
  static constexpr int UB = 4 * S;                      // blocks of a unit (four quads)
  static constexpr int XB = UB * kMxValues * (XF == kMxRowsCodes ? 1 : XF == kMxRowsBf16 ? 4 : 8) / 2;
  static constexpr int CH = XB / 16;                    // 16-byte chunks of a row's unit
  static constexpr int LC = CH / 4;                     // and one lane's of them
  static constexpr int T = TC / 16;
  static constexpr int STAGE = SU * KS;                 // units of a stage
  static constexpr int PARTS = TC * XB / 1024;          // direct-to-LDS loads of a unit
  static constexpr int COLS = 64 / CH;                  // columns of one such load
  static constexpr int BYTES = STAGE * TC * XB;         // of a buffer
  static constexpr int ROWS = 16 * FR * (KS > 1 ? 1 : NW);  // of an item
  // units whose scales are staged at a time: those of 2048 k's (1024 beside bf16 or fp32 rows)
  static constexpr int XSU = 8;
  using Scales = typename std::conditional<UB == 8, uint2, uint32_t>::type;  // of one row's unit
  static_assert(CH >= 8 && CH <= 64 && 64 % CH == 0, "a load covers whole columns");
  static_assert(PARTS % NW == 0 || NW % PARTS == 0, "parts go round the waves");
  static_assert(STAGE * PARTS % NW == 0, "every wave has as many loads");
  static_assert(XSU % STAGE == 0, "scales of whole stages");
};

// The 16-byte place of chunk c of column col: an exclusive or with the column, so that 16 columns'
// chunks at one place of their rows lie in different banks (64 of 4 bytes).
template <int CH>
__device__ __forceinline__ int mx_place(int c, int col) {
  return CH == 8 ? c ^ ((col >> 1) & 7) : c ^ (col & 15);
}

// v, opaque to the compiler, which would otherwise compute what follows from it ahead of a loop and keep
// (and spill) it across.
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// Direct-to-LDS load of 16 bytes a lane, lane i's to lds_wave_base + 16 i, hidden from the compiler's count
// of loads in flight: it would wait for the next stage's before it reads this one's. Its arrival is waited
// for by count (mx_wait).
__device__ __forceinline__ void mx_dma16(const void* src, const char* lds_wave_base) {
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)lds_wave_base;
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :
               : "v"(src), "s"(__builtin_amdgcn_readfirstlane(at))
               : "memory");
}
// Waits until at most N of this wave's loads are in flight (the last N issued) and its LDS accesses are done.
template <int N>
__device__ __forceinline__ void mx_wait() {
  static_assert(N < 64, "the counter's range");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(N) : "memory");
}

// V neighbouring outputs of row p from column n on, one store where they are aligned and all there.
template <bool OBF16, int V>
__device__ __forceinline__ void mx_store(const MxGemmArgs& a, int p, int n, const uint32_t (&w)[OBF16 ? V / 2 : V]) {
  constexpr int D = OBF16 ? V / 2 : V;  // dwords: 2 or 4
  const int64_t at = (int64_t)p * a.ld_out + n;
  char* dst = (char*)a.out + at * (OBF16 ? 2 : 4);
  if ((D == 2 ? a.vec8_out : a.vec_out) && n + V <= a.N) {
    if constexpr (D == 2) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else st16_nt(dst, make_uint4(w[0], w[1], w[2], w[3]));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (n + i >= a.N) continue;
      if constexpr (OBF16) ((uint16_t*)dst)[i] = (uint16_t)(w[i / 2] >> (16 * (i % 2)));
      else ((uint32_t*)dst)[i] = w[i];
    }
  }
}

// A lane's sums of column (pair) p, rows n0 + 16 f + 4 quad + i of tile f, F tiles. bf16 tiles go in twos: the
// quads exchange halves, so that a lane has eight neighbouring rows, 16 bytes, and four lanes 64.
template <bool OBF16, int F>
__device__ __forceinline__ void mx_store_tiles(const MxGemmArgs& a, bool there, int p, int n0, int quad,
                                               const f32x4_t (&acc)[F]) {
  if constexpr (OBF16 && F % 2 == 0) {
#pragma unroll
    for (int f = 0; f < F; f += 2) {
      const f32x4_t x = acc[f], y = acc[f + 1];
      const auto lo = __builtin_amdgcn_permlane16_swap(bf16_pair(x[0], x[1]), bf16_pair(y[0], y[1]), false, false);
      const auto hi = __builtin_amdgcn_permlane16_swap(bf16_pair(x[2], x[3]), bf16_pair(y[2], y[3]), false, false);
      const uint32_t w[4] = {lo[0], hi[0], lo[1], hi[1]};
      const int n = n0 + f * 16 + (quad & 1) * 16 + (quad >> 1) * 8;
      if (there && n < a.N) mx_store<true, 8>(a, p, n, w);
    }
  } else {
#pragma unroll
    for (int f = 0; f < F; ++f) {
      const int n = n0 + f * 16 + quad * 4;
      const f32x4_t v = acc[f];
      if (!there || n >= a.N) continue;
      if constexpr (OBF16) {
        const uint32_t w[2] = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
        mx_store<true, 4>(a, p, n, w);
      } else {
        const uint32_t w[4] = {__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
        mx_store<false, 4>(a, p, n, w);
      }
    }
  }
}

// The columns of a pass in LDS: pairs, and the first bytes of their rows of x (row 0's for those that are not there).
template <int TC>
struct MxCols {
  int64_t row[TC];
  int pair[TC];
};

// One pass: the products of an item's weight rows with the ncol real pairs of a block, ncol <= TC.
template <int XF, bool OBF16, int TC, int FR, int SU, int NW, int KS, int TCL>
__device__ __forceinline__ void mx4_pass(const MxGemmArgs& a, char* lds,
                                         typename MxShape<XF, TC, FR, SU, NW, KS>::Scales* wsc,
                                         typename MxShape<XF, TC, FR, SU, NW, KS>::Scales* xsc,
                                         const MxCols<TCL>& cols, int e, int n0, int ncol) {
  using Sh = MxShape<XF, TC, FR, SU, NW, KS>;
  using Scales = typename Sh::Scales;
  constexpr int S = Sh::S, T = Sh::T;
  constexpr bool CODES = XF == kMxRowsCodes;
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int units = (a.blocks + Sh::UB - 1) / Sh::UB;
  const int r0 = n0 + (KS > 1 ? 0 : wv * (16 * FR));
  const int first = KS > 1 ? wv : 0;  // of this wave's units, which are KS apart

  // this lane's weight rows
  const int64_t wbytes = (int64_t)a.N * (a.K / 2);
  const __amdgpu_buffer_rsrc_t w_rsrc = expert_rsrc(a.W + e * wbytes, wbytes);
  uint32_t w_off[FR];
#pragma unroll
  for (int f = 0; f < FR; ++f)  // (rows past the last: it again, not stored)
    w_off[f] = (uint32_t)min(r0 + f * 16 + col, a.N - 1) * (uint32_t)(a.K / 2);
  // block s of the lane's in unit u
  auto load_w = [&](int f, int u, int s, int quad) __attribute__((always_inline)) {
    const int b = u * Sh::UB + quad * S + s;
    return buf16(w_rsrc, b < a.blocks ? w_off[f] + (uint32_t)b * 16u : kOutOfRange);
  };
  // The scales of units [u0, u0 + XSU) of R rows, row r's from row(r) on, zeros (2^-127) past a row's end,
  // where the codes are zeros; all of a row's unit at once where that is one aligned load.
  auto stage_scales = [&](Scales* to, int R, int u0, bool whole, auto row) __attribute__((always_inline)) {
    const int n = min(Sh::XSU, units - u0) * R;
#pragma unroll 1
    for (int i = opaque(tid); i < n; i += Sh::THREADS) {
      const int u = i / R, b = (u0 + u) * Sh::UB;
      const uint8_t* src = row(i - u * R) + b;
      if (whole) {
        to[i] = *reinterpret_cast<const Scales*>(src);
      } else {
        uint64_t v = 0;
#pragma unroll 1
        for (int k = 0; k < Sh::UB && b + k < a.blocks; ++k) v |= (uint64_t)src[k] << (8 * k);
        __builtin_memcpy(&to[i], &v, sizeof(Scales));
      }
    }
  };

  const int row_chunks = a.blocks * (Sh::CH / Sh::UB);
  auto stage_x = [&](int u0, char* buf) __attribute__((always_inline)) {
    const int ln = opaque(lane);
#pragma unroll
    for (int i = 0; i < Sh::STAGE * Sh::PARTS / NW; ++i) {
      const int id = i * NW + wv, u = id / Sh::PARTS, part = id % Sh::PARTS;
      if (part * Sh::COLS >= ncol) continue;
      const int c = part * Sh::COLS + ln / Sh::CH;  // a lane's column, and its chunk of the row
      const int at = (u0 + u) * Sh::CH + mx_place<Sh::CH>(ln % Sh::CH, c);
      const void* src = at < row_chunks ? (const void*)((const char*)a.x + cols.row[c] + (int64_t)at * 16)
                                        : (const void*)kMxZeros;
      mx_dma16(src, buf + u * (TC * Sh::XB) + part * 1024);
    }
  };
  uint4 w[SU][FR][S];
  f32x4_t acc[T][FR];
#pragma unroll
  for (int t = 0; t < T; ++t)
#pragma unroll
    for (int f = 0; f < FR; ++f) acc[t][f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  stage_x(0, lds);
#pragma unroll
  for (int i = 0; i < SU; ++i) {
    const int u = first + i * KS;
#pragma unroll
    for (int f = 0; f < FR; ++f) {
#pragma unroll
      for (int s = 0; s < S; ++s) w[i][f][s] = load_w(f, u, s, quad);
    }
  }

  constexpr int kLoads = SU * FR * S;  // of weights in a stage, all issued after its x
  int buf = 0;
  for (int u0 = 0; u0 < units; u0 += Sh::STAGE, buf ^= 1) {
    if (u0 % Sh::XSU == 0) {  // scales for this stage and those after it
      if (u0 > 0) __syncthreads();
      stage_scales(wsc, Sh::ROWS, u0, a.whole_w, [&](int r) {
        return a.scales + ((int64_t)e * a.N + min(n0 + r, a.N - 1)) * a.blocks;
      });
      if constexpr (CODES)
        stage_scales(xsc, TC, u0, a.whole_x, [&](int c) {
          return a.x_scales + (int64_t)fdiv(cols.pair[min(c, ncol - 1)], a.f_rd) * a.ld_xs;
        });
    }
    // this wave's part of the stage of x has arrived, then everyone's, and the other buffer is free
    if (u0 == 0) mx_wait<0>();  // (the stores of an earlier pass count too)
    else mx_wait<kLoads>();
    __builtin_amdgcn_s_barrier();
    if (u0 + Sh::STAGE < units) stage_x(u0 + Sh::STAGE, lds + (buf ^ 1) * Sh::BYTES);
#pragma unroll
    for (int i = 0; i < SU; ++i) {
      const int u = first + i * KS;  // of the stage
      if (u0 + u >= units) break;
      const char* xu = lds + buf * Sh::BYTES + u * (TC * Sh::XB);
      const int us = (u0 + u) % Sh::XSU, next = u0 + u + Sh::STAGE;
      const int ln = opaque(lane), col = ln & 15, quad = ln >> 4;
      // chunk c of column t * 16 + col (whose place goes by col alone)
      auto x_at = [&](int t, int c) __attribute__((always_inline)) {
        return *reinterpret_cast<const uint4*>(xu + col * Sh::XB + mx_place<Sh::CH>(c, col) * 16 +
                                               t * (16 * Sh::XB));
      };
      // scales of a lane's blocks, one a byte: of weight row f * 16 + col, of column t * 16 + col
      auto scale_w = [&](int f) __attribute__((always_inline)) {
        const Scales* p = wsc + us * Sh::ROWS + (r0 - n0) + f * 16 + col;
        if constexpr (S == 2) return (uint32_t)reinterpret_cast<const uint16_t*>(p)[quad];
        else return (uint32_t)reinterpret_cast<const uint8_t*>(p)[quad];
      };
      auto scale_x = [&](int t) __attribute__((always_inline)) {
        return (uint32_t)reinterpret_cast<const uint16_t*>(xsc + us * TC + t * 16 + col)[quad];
      };
      uint32_t ws[FR];
#pragma unroll
      for (int f = 0; f < FR; ++f) ws[f] = scale_w(f);
      if constexpr (CODES) {
        // fragments of x are read kAhead steps before their products, and no earlier: left to itself
        // the compiler reads all of them first and runs out of registers
        constexpr int Q = S * T, kAhead = T > 1 ? 2 : 1, B = kAhead + 1;
        uint4 xq[B];
        uint32_t xsq[B];
        auto read = [&](int q) __attribute__((always_inline)) {
          xq[q % B] = x_at(q % T, quad * S + q / T);
          xsq[q % B] = scale_x(q % T);
        };
#pragma unroll
        for (int q = 0; q < kAhead; ++q) read(q);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const int s = q / T, t = q % T;
          if (q + kAhead < Q) read(q + kAhead);
          if (t == 0 || t * 16 < ncol) {
            const uint4 x = xq[q % B];
            const i32x8_t xv = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
#pragma unroll
            for (int f = 0; f < FR; ++f) {
              const uint4 v = w[i][f][s];
              const i32x8_t wv8 = {(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
              acc[t][f] = s == 0 ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                       wv8, xv, acc[t][f], 4, 4, 0, (int)ws[f], 0, (int)xsq[q % B])
                                 : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                       wv8, xv, acc[t][f], 4, 4, 1, (int)ws[f], 1, (int)xsq[q % B]);
            }
          }
          if (t == T - 1) {
#pragma unroll
            for (int f = 0; f < FR; ++f) w[i][f][s] = load_w(f, next, s, quad);
          }
          if constexpr (T > 1) __builtin_amdgcn_sched_barrier(0);
        }
      } else {
        float unit[FR];
#pragma unroll
        for (int f = 0; f < FR; ++f) unit[f] = mx_scale(ws[f]);
        constexpr int H = XF == kMxRowsBf16 ? 1 : 2;  // 16-byte vectors of x beside a dword of codes
#pragma unroll
        for (int j = 0; j < 4; ++j) {                 // a dword of codes: eight k's
          uint4 wb[FR];
          float wf[FR][8];
#pragma unroll
          for (int f = 0; f < FR; ++f) {
            const uint4 v = w[i][f][0];
            const uint32_t c = j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
            if constexpr (XF == kMxRowsBf16) wb[f] = mx_bf16(c, unit[f]);
            else mx_f32(c, unit[f], wf[f]);
          }
#pragma unroll
          for (int t = 0; t < T; ++t) {
            uint4 x[H];
#pragma unroll
            for (int h = 0; h < H; ++h) x[h] = x_at(t, quad * Sh::LC + j * H + h);
            if (t > 0 && t * 16 >= ncol) continue;
            if constexpr (XF == kMxRowsBf16) {
#pragma unroll
              for (int f = 0; f < FR; ++f)
                acc[t][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8_t, wb[f]), __builtin_bit_cast(bf16x8_t, x[0]), acc[t][f],
                    0, 0, 0);
            } else {
#pragma unroll
              for (int h = 0; h < H; ++h) {
                const uint32_t xe[4] = {x[h].x, x[h].y, x[h].z, x[h].w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                  for (int f = 0; f < FR; ++f)
                    acc[t][f] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                        wf[f][h * 4 + k], __uint_as_float(xe[k]), acc[t][f], 0, 0, 0);
              }
            }
          }
        }
#pragma unroll
        for (int f = 0; f < FR; ++f) w[i][f][0] = load_w(f, next, 0, quad);
      }
    }
  }

  if constexpr (KS > 1) {  // the waves' sums of one tile
    __syncthreads();
    f32x4_t* red = reinterpret_cast<f32x4_t*>(lds);
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int f = 0; f < FR; ++f) red[((t * FR + f) * NW + wv) * 64 + lane] = acc[t][f];
    __syncthreads();
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
      for (int f = 0; f < FR; ++f) {
        if ((t * FR + f) % NW != wv) continue;
        const f32x4_t* r = red + (t * FR + f) * NW * 64 + lane;
        const f32x4_t v = (r[0] + r[64]) + (r[128] + r[192]);  // (NW = 4)
        const int c = t * 16 + col;
        const f32x4_t one[1] = {v};
        mx_store_tiles<OBF16, 1>(a, c < ncol, cols.pair[c], r0 + f * 16, quad, one);
      }
  } else {
#pragma unroll
    for (int t = 0; t < T; ++t) {
      if (t > 0 && t * 16 >= ncol) break;
      const int c = t * 16 + col;
      mx_store_tiles<OBF16, FR>(a, c < ncol, cols.pair[c], r0, quad, acc[t]);
    }
  }
}

// Bytes of LDS: two buffers of x, the scales of the item's rows and of the columns.
template <int XF, int TC, int FR, int SU, int NW, int KS>
struct MxLds {
  using Sh = MxShape<XF, TC, FR, SU, NW, KS>;
  char x[2 * Sh::BYTES] __attribute__((aligned(16)));
  typename Sh::Scales ws[Sh::XSU * Sh::ROWS];
  typename Sh::Scales xs[XF == kMxRowsCodes ? Sh::XSU * TC : 1];
  MxCols<TC> cols;
};

// The columns of a pass into LDS, p this thread's entry of the block; how many are real pairs, which are
// a prefix of the block.
template <int TC>
__device__ __forceinline__ int put_pairs(MxCols<TC>& cols, int p, const MxGemmArgs& a) {
  if (threadIdx.x < TC) {
    cols.pair[threadIdx.x] = p;
    cols.row[threadIdx.x] = real_pair(p, a.numel) ? (int64_t)fdiv(p, a.f_rd) * a.x_bytes : 0;
  }
  __syncthreads();
  const int lane = threadIdx.x & 63;
  int ncol = 0;
#pragma unroll
  for (int j = 0; j < TC; j += 64)
    ncol += __popcll(__builtin_amdgcn_ballot_w64(j + lane < TC && real_pair(cols.pair[min(j + lane, TC - 1)], a.numel)));
  return ncol;
}

// A few columns a block: an item is a block and 64 weight rows (16 with split k's), whose passes of up to
// TC columns take the buffers in the shape of the columns there are; or, where SPREAD, one such pass.
template <int XF, bool OBF16, int TC, int SU, int KS, bool SPREAD>
__global__ void __launch_bounds__(256, 4) mx4_narrow_kernel(MxGemmArgs a) {
  __shared__ MxLds<XF, TC, 1, SU, 4, KS> lds;
  const int blk = fdiv((int)blockIdx.x, a.f_items);
  int in_blk = (int)blockIdx.x - blk * a.items, first = 0;
  if constexpr (SPREAD) {
    const int span = fdiv(in_blk, a.f_tiles);
    in_blk -= span * (int)a.f_tiles.d;
    first = span * TC;
  }
  const int n0 = in_blk * (KS > 1 ? 16 : 64);
  const int32_t* sorted = a.sorted + (int64_t)blk * a.BM;
  const int tid = threadIdx.x;
  const int npp = *a.npp;
  const int er = a.expert_ids[blk];
  // the first entries with the routing reads (their index stays inside the block)
  int p = tid < TC && tid < a.BM - first ? sorted[first + tid] : a.numel;
  const int nb = npp < 0 ? 0 : fdiv(npp, a.f_bm);
  if (blk >= nb || (unsigned)er >= (unsigned)a.E) return;
  const int e = __builtin_amdgcn_readfirstlane(er);
  for (int j0 = first; j0 < a.BM; j0 += TC) {
    if (j0 > first) {
      p = tid < TC && j0 + tid < a.BM ? sorted[j0 + tid] : a.numel;
      __syncthreads();  // the last pass is done with LDS
    }
    const int ncol = put_pairs<TC>(lds.cols, p, a);
    if (ncol == 0) return;
    auto pass = [&](auto tc) __attribute__((always_inline)) {
      constexpr int C = decltype(tc)::value;
      mx4_pass<XF, OBF16, C, 1, SU * (TC / C), 4, KS>(a, lds.x, lds.ws, lds.xs, lds.cols, e, n0, ncol);
    };
    if constexpr (TC > 16) {
      if (ncol <= 16) pass(std::integral_constant<int, 16>{});
      else if (TC > 32 && ncol <= 32) pass(std::integral_constant<int, 32>{});
      else pass(std::integral_constant<int, TC>{});
    } else {
      pass(std::integral_constant<int, TC>{});
    }
    if (SPREAD || ncol < TC) return;
  }
}

constexpr int kMxChain = 64;  // a wave's lanes, a multiple of what an item takes together

// Many columns an expert: an item is a span of TC columns of a block, or (not of fp32 rows) up to a.merge smaller blocks of
// one expert that together have TC, and 16 FR NW weight rows. The items of the live blocks are a contiguous range for
// each of the eight XCDs (workgroups go round them): neighbouring items share an expert's weights and a block's
// rows in its L2.
template <int XF, bool OBF16, int TC, int FR, int SU, int NW>
__global__ void __launch_bounds__(64 * NW, 4) mx4_wide_kernel(MxGemmArgs a) {
  using Sh = MxShape<XF, TC, FR, SU, NW, 1>;
  __shared__ MxLds<XF, TC, FR, SU, NW, 1> lds;
  const int npp = *a.npp;
  const int nb = npp < 0 ? 0 : min(fdiv(npp, a.f_bm), a.max_blocks);
  // of the items of a.merge neighbouring blocks an XCD has those of the first one for its whole range, then the
  // second's: those that lead (below) lie together more often than not, and their workgroups on all compute units
  const int per_xcd = (int)((((int64_t)nb + a.merge - 1) / a.merge * a.items + 7) >> 3);
  const int local = (int)blockIdx.x >> 3;
  constexpr bool kMerges = XF != kMxRowsF32;
  const int turn = kMerges && a.merge > 1 ? (int)((uint32_t)local / (uint32_t)max(per_xcd, 1)) : 0;
  const int item = ((int)blockIdx.x & 7) * per_xcd + local - turn * per_xcd;
  const int group = fdiv(item, a.f_items);
  const int blk = group * a.merge + turn;
  if (local >= per_xcd * a.merge || blk >= nb) return;
  const int er = a.expert_ids[blk];
  if ((unsigned)er >= (unsigned)a.E) return;
  int width = a.BM;  // columns of the item's blocks
  if (kMerges && a.merge > 1) {
    // A full block and the next one go together where they are one expert's: of a chain of such blocks every
    // a.merge-th, from its first on, leads an item, and its followers leave theirs to it. Chains end before every
    // block whose index is a multiple of kMxChain, so that one look of a wave finds a block's place in its own; it costs
    // one item more for each such end. (Looking back to the first block of an expert grew with the square of its
    // pairs: 65536 pairs of one, K 2048, N 1536, codes at blocks of 16, 32, 64 and 128 1724, 576, 265 and 155 us, so 208,
    // 178, 164 and 156.)
    const int lane = threadIdx.x & 63, at = blk & (kMxChain - 1);
    auto joins = [&](int i) __attribute__((always_inline)) {  // block i with block i + 1, 0 <= i < nb - 1
      return a.expert_ids[i] == er && a.expert_ids[i + 1] == er &&
             real_pair(a.sorted[(int64_t)i * a.BM + a.BM - 1], a.numel);
    };
    const uint64_t begins = __builtin_amdgcn_ballot_w64(lane >= at || !joins(blk - 1 - lane));
    if (__builtin_ctzll(begins) % a.merge) return;  // (lane 63 always votes: at < 64)
    const int i = blk + lane;
    const uint64_t ends = __builtin_amdgcn_ballot_w64(lane >= min(a.merge, kMxChain - at) - 1 || i >= nb - 1 || !joins(i));
    width += __builtin_ctzll(ends) * a.BM;  // (a.merge <= 8)
  }
  const int in_blk = item - group * a.items;
  const int span = fdiv(in_blk, a.f_tiles);  // of the block's spans of columns
  const int n0 = (in_blk - span * (int)a.f_tiles.d) * Sh::ROWS;
  const int j = span * TC + (int)threadIdx.x;
  const int p = threadIdx.x < TC && j < width ? a.sorted[(int64_t)blk * a.BM + j] : a.numel;
  const int ncol = put_pairs<TC>(lds.cols, p, a);
  if (ncol == 0) return;
  mx4_pass<XF, OBF16, TC, FR, SU, NW, 1>(a, lds.x, lds.ws, lds.xs, lds.cols,
                                         __builtin_amdgcn_readfirstlane(er), n0, ncol);
}

template <int XF, bool OBF16, int TC, int SU, int KS, bool SPREAD>
hipError_t mx4_narrow(MxGemmArgs a, hipStream_t st) {
  static_assert(KS == 1 || (KS == 4 && 4096 * TC / 16 <= 2 * MxShape<XF, TC, 1, SU, 4, KS>::BYTES),
                "room for the waves' sums");
  const int32_t tiles = (a.N + (KS > 1 ? 15 : 63)) / (KS > 1 ? 16 : 64);
  a.f_tiles = make_fastdiv((uint32_t)tiles);
  a.items = SPREAD ? tiles * mx_spans(a.BM, TC) : tiles;
  a.f_items = make_fastdiv((uint32_t)a.items);
  hipLaunchKernelGGL((mx4_narrow_kernel<XF, OBF16, TC, SU, KS, SPREAD>), dim3((unsigned)(a.max_blocks * a.items)),
                     dim3(256), 0, st, a);
  return hipGetLastError();
}

template <int XF, bool OBF16, int TC, int FR, int SU, int NW>
hipError_t mx4_wide(MxGemmArgs a, hipStream_t st) {
  using Sh = MxShape<XF, TC, FR, SU, NW, 1>;
  const int32_t tiles = (a.N + Sh::ROWS - 1) / Sh::ROWS;
  a.f_tiles = make_fastdiv((uint32_t)tiles);
  a.items = tiles * mx_spans(a.BM, TC);
  a.merge = mx_merge(a.BM, XF);
  a.f_items = make_fastdiv((uint32_t)a.items);
  // (a range for each XCD, rounded up)
  const int64_t grid = ((int64_t)(a.max_blocks + a.merge - 1) / a.merge * a.items + 7) / 8 * 8 * a.merge;
  hipLaunchKernelGGL((mx4_wide_kernel<XF, OBF16, TC, FR, SU, NW>), dim3((unsigned)grid), dim3(64 * NW), 0,
                     st, a);
  return hipGetLastError();
}

}  // namespace
}  // namespace mol
