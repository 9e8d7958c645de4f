// The base MoE grouped GEMM of a stage over microscaled 4-bit weights (mx4.h has the format):
//   out[p, n] = round( sum_k W[t, n, k] x[p / row_div, k] )
// for every pair p whose base expert t is local; other rows are untouched. x is rows of codes with
// scales of their own, or bf16 or fp32. Routed like the dense grouped GEMM (the aligned blocks of one
// base expert each).
//
// Codes times codes go to the scaled matrix-core product (16 x 16 x 128, both operands 4 bits, a scale
// byte a lane); beside bf16 and fp32 rows the weights are widened to that type in registers, which is
// exact, scale included. Products and sums are fp32, so infinities and NaN of x reach exactly the
// sums that the formula has them in.
//
// A work item is a span of columns of a routing block (a pass of the widest form, all of the block's of the
// narrow ones) and kWaves times 16 FR weight rows; wave w has 16 FR of them as
// the A operand, straight from memory into registers: lane l holds row l % 16 and whole blocks of 32 k's,
// which block of a step being free as long as x agrees. x goes through LDS for all four waves,
// as it lies in memory: direct-to-LDS loads, whose lanes choose their 16 bytes of a row so that the
// reads of a fragment (16 columns at one place of their rows) spread over the banks. Stages of x
// alternate between two buffers, the next one loading while one is at work; a weight register is filled
// again as soon as it has been used.
//
// Of the result, lane l holds column (pair) l % 16 and rows 4 (l / 16) + i.
#pragma once

#include "mx4.h"

namespace mol {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

constexpr int kMxWaves = kThreads / 64;

// What stands for k's past a row's end: x reads these zeros.
__device__ const uint4 kMxZeros[1] = {{0u, 0u, 0u, 0u}};

// Shape of a kernel. XF: the rows of x; TC columns a pass; FR times 16 weight rows a wave; SU units a
// stage (and wave); KS: the waves share 16 FR rows and split the units.
template <int XF, int TC, int FR, int SU, int KS>
struct MxShape {
  static constexpr int S = XF == kMxRowsCodes ? 2 : 1;  // blocks a lane has of a unit
  static constexpr int UB = 4 * S;                      // blocks of a unit (four quads)
  static constexpr int XB = UB * kMxValues * (XF == kMxRowsCodes ? 1 : XF == kMxRowsBf16 ? 4 : 8) / 2;
  static constexpr int CH = XB / 16;                    // 16-byte chunks of a row's unit
  static constexpr int LC = CH / 4;                     // and one lane's of them
  static constexpr int T = TC / 16;
  static constexpr int STAGE = SU * KS;                 // units of a stage
  static constexpr int PARTS = TC * XB / 1024;          // direct-to-LDS loads of a unit
  static constexpr int COLS = 64 / CH;                  // columns of one such load
  static constexpr int NP = PARTS > kMxWaves ? PARTS / kMxWaves : 1;  // a wave's parts
  static constexpr int BYTES = STAGE * TC * XB;         // of a buffer
  static constexpr int ROWS = 16 * FR * (KS > 1 ? 1 : kMxWaves);  // of an item
  static_assert(CH >= 8 && CH <= 64 && 64 % CH == 0, "a load covers whole columns");
  static_assert(PARTS % kMxWaves == 0 || kMxWaves % PARTS == 0, "parts go round the waves");
  static_assert(STAGE * PARTS % kMxWaves == 0, "every wave has as many loads");
};

// The 16-byte place of chunk c of column col: an exclusive or with the column, so that 16 columns'
// chunks at one place of their rows lie in different banks (64 of 4 bytes).
template <int CH>
__device__ __forceinline__ int mx_place(int c, int col) {
  return CH == 8 ? c ^ ((col >> 1) & 7) : c ^ (col & 15);
}

template <bool OBF16>
__device__ __forceinline__ void mx_store(const MxGemmArgs& a, int p, int n, const f32x4_t& v) {
  const int64_t at = (int64_t)p * a.ld_out + n;
  if (a.vec_out && n + 4 <= a.N) {
    if constexpr (OBF16) {
      uint2 w;
      w.x = f32_to_bf16_rne(v[0]) | ((uint32_t)f32_to_bf16_rne(v[1]) << 16);
      w.y = f32_to_bf16_rne(v[2]) | ((uint32_t)f32_to_bf16_rne(v[3]) << 16);
      *reinterpret_cast<uint2*>((uint16_t*)a.out + at) = w;
    } else {
      *reinterpret_cast<float4*>((float*)a.out + at) = make_float4(v[0], v[1], v[2], v[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (n + i >= a.N) continue;
      if constexpr (OBF16) ((uint16_t*)a.out)[at + i] = f32_to_bf16_rne(v[i]);
      else ((float*)a.out)[at + i] = v[i];
    }
  }
}

template <int XF, bool OBF16, int TC, int FR, int SU, int KS>
__global__ void __launch_bounds__(kThreads, 2) mx4_gemm_kernel(MxGemmArgs a) {
  using Sh = MxShape<XF, TC, FR, SU, KS>;
  constexpr int S = Sh::S, T = Sh::T;
  constexpr bool CODES = XF == kMxRowsCodes;
  __shared__ __attribute__((aligned(16))) char lds[2 * Sh::BYTES];
  __shared__ int pair[TC];

  // the items of the live blocks, a contiguous range for each of the eight XCDs (workgroups go round
  // them): neighbouring items share an expert's weights and a block's rows in its L2
  const int npp = *a.npp;
  const int nb = npp < 0 ? 0 : min(fdiv(npp, a.f_bm), a.max_blocks);
  const int per_xcd = (int)(((int64_t)nb * a.items + 7) >> 3);
  const int local = (int)blockIdx.x >> 3;
  const int item = ((int)blockIdx.x & 7) * per_xcd + local;
  const int blk = fdiv(item, a.f_items);
  if (local >= per_xcd || blk >= nb) return;
  const int er = a.expert_ids[blk];
  if ((unsigned)er >= (unsigned)a.E) return;
  const int e = __builtin_amdgcn_readfirstlane(er);
  const int in_blk = item - blk * a.items;
  const int span0 = fdiv(in_blk, a.f_tiles);  // of the block's spans of columns
  const int n0 = (in_blk - span0 * (int)a.f_tiles.d) * Sh::ROWS;

  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int units = (a.blocks + Sh::UB - 1) / Sh::UB;
  const int r0 = n0 + (KS > 1 ? 0 : wv * (16 * FR));
  const int first = KS > 1 ? wv : 0;  // of this wave's units, which are KS apart

  // this lane's weight rows and their scales
  const int64_t wbytes = (int64_t)a.N * (a.K / 2), sbytes = (int64_t)a.N * a.blocks;
  const __amdgpu_buffer_rsrc_t w_rsrc = expert_rsrc(a.W + e * wbytes, wbytes);
  const __amdgpu_buffer_rsrc_t s_rsrc = expert_rsrc(a.scales + e * sbytes, sbytes);
  uint32_t w_off[FR], s_off[FR];
#pragma unroll
  for (int f = 0; f < FR; ++f) {
    const int n = min(r0 + f * 16 + col, a.N - 1);  // (rows past the last: it again, not stored)
    w_off[f] = (uint32_t)n * (uint32_t)(a.K / 2);
    s_off[f] = (uint32_t)n * (uint32_t)a.blocks;
  }
  // the first of a lane's blocks of unit u
  auto block_of = [&](int u) __attribute__((always_inline)) { return u * Sh::UB + quad * S; };
  auto load_w = [&](int f, int u, int s) __attribute__((always_inline)) {
    const int b = block_of(u) + s;
    return buf16(w_rsrc, b < a.blocks ? w_off[f] + (uint32_t)b * 16u : kOutOfRange);
  };
  // the scales of a lane's blocks of a unit, one a byte; 1 past the row (where the codes are zeros)
  auto load_ws = [&](int f, int u) __attribute__((always_inline)) {
    const int b = block_of(u);
    uint32_t v;
    if constexpr (S == 2) {
      if (a.pairs_w) {
        v = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
            s_rsrc, b < a.blocks ? s_off[f] + (uint32_t)b : kOutOfRange, 0, 0);
        return b < a.blocks ? v : 0x7f7fu;
      }
      const uint32_t lo = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
          s_rsrc, b < a.blocks ? s_off[f] + (uint32_t)b : kOutOfRange, 0, 0);
      const uint32_t hi = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
          s_rsrc, b + 1 < a.blocks ? s_off[f] + (uint32_t)b + 1u : kOutOfRange, 0, 0);
      return (b < a.blocks ? lo : 0x7fu) | (b + 1 < a.blocks ? hi : 0x7fu) << 8;
    } else {
      v = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(
          s_rsrc, b < a.blocks ? s_off[f] + (uint32_t)b : kOutOfRange, 0, 0);
      return b < a.blocks ? v : 0x7fu;
    }
  };

  const int32_t* sorted = a.sorted + (int64_t)blk * a.BM;
  const int j_begin = span0 * a.span, j_end = min(a.BM, j_begin + a.span);
  for (int j0 = j_begin; j0 < j_end; j0 += TC) {
    if (j0 > j_begin) __syncthreads();  // the last pass is done with pair and LDS
    for (int j = tid; j < TC; j += kThreads) pair[j] = j0 + j < a.BM ? sorted[j0 + j] : a.numel;
    __syncthreads();
    // the real pairs are a prefix of the block
    int ncol = 0;
#pragma unroll
    for (int j = 0; j < TC; j += 64)
      ncol += __popcll(__builtin_amdgcn_ballot_w64(j + lane < TC && real_pair(pair[min(j + lane, TC - 1)], a.numel)));
    if (ncol == 0) return;

    // this lane's places of x: its column's row in each of the wave's parts of a unit
    const char* x_row[Sh::NP];
    int x_chunk[Sh::NP];
#pragma unroll
    for (int i = 0; i < Sh::NP; ++i) {
      const int part = (i * kMxWaves + wv) % Sh::PARTS;
      const int c = part * Sh::COLS + lane / Sh::CH;
      const int p = pair[min(c, ncol - 1)];  // (columns that are not there: the last one again)
      x_row[i] = (const char*)a.x + (int64_t)fdiv(p, a.f_rd) * a.x_bytes;
      x_chunk[i] = mx_place<Sh::CH>(lane % Sh::CH, c);
    }
    const int row_chunks = a.blocks * (Sh::CH / Sh::UB);
    auto stage_x = [&](int u0, char* buf) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < Sh::STAGE * Sh::PARTS / kMxWaves; ++i) {
        const int id = i * kMxWaves + wv, u = id / Sh::PARTS, part = id % Sh::PARTS;
        if (part * Sh::COLS >= ncol) continue;
        const int at = (u0 + u) * Sh::CH + x_chunk[i % Sh::NP];
        const void* src = at < row_chunks ? (const void*)(x_row[i % Sh::NP] + (int64_t)at * 16)
                                          : (const void*)kMxZeros;
        lds_dma16(src, buf + u * (TC * Sh::XB) + part * 1024);
      }
    };
    // rows of codes: the scales of column t * 16 + col
    uint32_t xs_off[CODES ? T : 1];
    if constexpr (CODES) {
#pragma unroll
      for (int t = 0; t < T; ++t)
        xs_off[t] = (uint32_t)fdiv(pair[min(t * 16 + col, ncol - 1)], a.f_rd) * (uint32_t)a.ld_xs;
    }
    auto load_xs = [&](int t, int u) __attribute__((always_inline)) {
      const int b = block_of(u);
      const uint8_t* src = a.x_scales + (size_t)(xs_off[CODES ? t : 0] + (uint32_t)min(b, a.blocks - 1));
      uint32_t v;
      if (a.pairs_x) {
        v = *(const uint16_t*)(b < a.blocks ? src : a.x_scales);
        return b < a.blocks ? v : 0x7f7fu;
      }
      const uint32_t lo = src[0], hi = src[b + 1 < a.blocks ? 1 : 0];
      return (b < a.blocks ? lo : 0x7fu) | (b + 1 < a.blocks ? hi : 0x7fu) << 8;
    };

    uint4 w[SU][FR][S];
    uint32_t ws[SU][FR], xs[SU][CODES ? T : 1];
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
        for (int s = 0; s < S; ++s) w[i][f][s] = load_w(f, u, s);
        ws[i][f] = load_ws(f, u);
      }
      if constexpr (CODES) {
#pragma unroll
        for (int t = 0; t < T; ++t) xs[i][t] = load_xs(t, u);
      }
    }

    int buf = 0;
    for (int u0 = 0; u0 < units; u0 += Sh::STAGE, buf ^= 1) {
      __builtin_amdgcn_s_waitcnt(0);  // this wave's part of the stage of x has arrived,
      __syncthreads();                // everyone's, and the other buffer is no longer read
      if (u0 + Sh::STAGE < units) stage_x(u0 + Sh::STAGE, lds + (buf ^ 1) * Sh::BYTES);
#pragma unroll
      for (int i = 0; i < SU; ++i) {
        const int u = first + i * KS;  // of the stage
        if (u0 + u >= units) break;
        const char* xu = lds + buf * Sh::BYTES + u * (TC * Sh::XB);
        auto x_at = [&](int t, int c) __attribute__((always_inline)) {  // chunk c of column t * 16 + col
          const int cc = t * 16 + col;
          return *reinterpret_cast<const uint4*>(xu + cc * Sh::XB + mx_place<Sh::CH>(c, cc) * 16);
        };
        if constexpr (CODES) {
#pragma unroll
          for (int s = 0; s < S; ++s) {
#pragma unroll
            for (int t = 0; t < T; ++t) {
              if (t > 0 && t * 16 >= ncol) break;
              const uint4 x = x_at(t, quad * S + s);
              const i32x8_t xv = {(int)x.x, (int)x.y, (int)x.z, (int)x.w, 0, 0, 0, 0};
#pragma unroll
              for (int f = 0; f < FR; ++f) {
                const uint4 v = w[i][f][s];
                const i32x8_t wv8 = {(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
                acc[t][f] = s == 0 ? __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                         wv8, xv, acc[t][f], 4, 4, 0, (int)ws[i][f], 0, (int)xs[i][t])
                                   : __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                                         wv8, xv, acc[t][f], 4, 4, 1, (int)ws[i][f], 1, (int)xs[i][t]);
              }
            }
          }
        } else {
          float unit[FR];
#pragma unroll
          for (int f = 0; f < FR; ++f) unit[f] = mx_scale(ws[i][f]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {  // a dword of codes: eight k's
            if constexpr (XF == kMxRowsBf16) {
              uint4 wb[FR];
#pragma unroll
              for (int f = 0; f < FR; ++f) {
                const uint4 v = w[i][f][0];
                wb[f] = mx_bf16(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w, unit[f]);
              }
#pragma unroll
              for (int t = 0; t < T; ++t) {
                if (t > 0 && t * 16 >= ncol) break;
                const bf16x8_t x = __builtin_bit_cast(bf16x8_t, x_at(t, quad * Sh::LC + j));
#pragma unroll
                for (int f = 0; f < FR; ++f)
                  acc[t][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                      __builtin_bit_cast(bf16x8_t, wb[f]), x, acc[t][f], 0, 0, 0);
              }
            } else {
              float wf[FR][8];
#pragma unroll
              for (int f = 0; f < FR; ++f) {
                const uint4 v = w[i][f][0];
                mx_f32(j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w, unit[f], wf[f]);
              }
#pragma unroll
              for (int t = 0; t < T; ++t) {
                if (t > 0 && t * 16 >= ncol) break;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint4 x = x_at(t, quad * Sh::LC + j * 2 + h);
                  const uint32_t xe[4] = {x.x, x.y, x.z, x.w};
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
        }
        const int next = u0 + u + Sh::STAGE;
#pragma unroll
        for (int f = 0; f < FR; ++f) {
#pragma unroll
          for (int s = 0; s < S; ++s) w[i][f][s] = load_w(f, next, s);
          ws[i][f] = load_ws(f, next);
        }
        if constexpr (CODES) {
#pragma unroll
          for (int t = 0; t < T; ++t) xs[i][t] = load_xs(t, next);
        }
      }
    }

    if constexpr (KS > 1) {  // the waves' sums of one tile
      __syncthreads();
      f32x4_t* red = reinterpret_cast<f32x4_t*>(lds);
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int f = 0; f < FR; ++f) red[((t * FR + f) * kMxWaves + wv) * 64 + lane] = acc[t][f];
      __syncthreads();
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int f = 0; f < FR; ++f) {
          if ((t * FR + f) % kMxWaves != wv) continue;
          const f32x4_t* r = red + (t * FR + f) * kMxWaves * 64 + lane;
          const f32x4_t v = (r[0] + r[64]) + (r[128] + r[192]);
          const int c = t * 16 + col;
          const int n = r0 + f * 16 + quad * 4;
          if (c < ncol && n < a.N) mx_store<OBF16>(a, pair[c], n, v);
        }
    } else {
#pragma unroll
      for (int t = 0; t < T; ++t) {
        const int c = t * 16 + col;
        if (c >= ncol) continue;
        const int p = pair[c];
#pragma unroll
        for (int f = 0; f < FR; ++f) {
          const int n = r0 + f * 16 + quad * 4;
          if (n < a.N) mx_store<OBF16>(a, p, n, acc[t][f]);
        }
      }
    }
    if (ncol < TC) return;
  }
}

template <int XF, bool OBF16, int TC, int FR, int SU, int KS>
hipError_t mx4_launch(MxGemmArgs a, bool wide, hipStream_t st) {
  using Sh = MxShape<XF, TC, FR, SU, KS>;
  static_assert(KS == 1 || TC / 16 * FR * kMxWaves * 1024 <= 2 * Sh::BYTES, "room for the waves' sums");
  const int32_t tiles = (a.N + Sh::ROWS - 1) / Sh::ROWS;
  a.f_tiles = make_fastdiv((uint32_t)tiles);
  a.span = wide ? TC : a.BM;
  a.items = tiles * ((a.BM + a.span - 1) / a.span);
  a.f_items = make_fastdiv((uint32_t)a.items);
  // (a range for each XCD, rounded up)
  const int64_t grid = ((int64_t)a.max_blocks * a.items + 7) / 8 * 8;
  hipLaunchKernelGGL((mx4_gemm_kernel<XF, OBF16, TC, FR, SU, KS>), dim3((unsigned)grid), dim3(kThreads), 0,
                     st, a);
  return hipGetLastError();
}

}  // namespace
}  // namespace mol
