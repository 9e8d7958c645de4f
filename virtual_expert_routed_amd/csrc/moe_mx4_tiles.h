// The wide form of the product over rows of codes whose scales lie on 4-byte boundaries (K a multiple of 128):
// 128 columns of a routing block and 256 weight rows a workgroup of eight waves, 64 of each a wave.
//
// Both operands go through LDS, by direct-to-LDS loads. A lane that loads its operand itself has the place that the
// matrix core gives it, 16 lanes in 16 rows, and the L1 looks up a line for every lane (as the first wide form did:
// the look-ups alone took 63 % of its time); four lanes that load the 64 bytes of a row together need one.
//
// A stage is 128 k's: 64 bytes of each of the 384 rows, and every second stage the scales of two. Three stages
// are in LDS at a time: one at work, two on their way. The 16-byte place of chunk c of a row r is c ^ (r / 4 % 4), so that
// 16 rows' chunks at one k lie in different banks (64 of 4 bytes).
#pragma once

#include "moe_mx4.h"

namespace mol {
namespace {

struct MxTiles {
  static constexpr int TC = 128, RN = 256, ROWS = TC + RN;
  static constexpr int STAGES = 3, STAGE = ROWS * 64;  // bytes of a stage
  char codes[STAGES][STAGE] __attribute__((aligned(16)));
  uint32_t scales[2][ROWS * 2];  // of two stages: two dwords a row, columns first
  MxCols<TC> cols;
};
static_assert(2 * sizeof(MxTiles) <= 163840, "two workgroups a CU");

// 4 bytes a lane, as mx_dma16.
__device__ __forceinline__ void mx_dma4(const void* src, const void* lds_wave_base) {
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const char*)lds_wave_base;
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off"
               :
               : "v"(src), "s"(__builtin_amdgcn_readfirstlane(at))
               : "memory");
}

template <bool OBF16>
__global__ void __launch_bounds__(512, 4) mx4_tiles_kernel(MxGemmArgs a) {
  constexpr int TC = MxTiles::TC, RN = MxTiles::RN;
  __shared__ MxTiles lds;
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
  const int span = fdiv(in_blk, a.f_tiles);
  const int tile0 = (in_blk - span * (int)a.f_tiles.d) * a.run;  // of `tiles` tiles of weight rows
  const int tiles = min(a.run, (a.N + RN - 1) / RN - tile0);
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int j = span * TC + tid;
  const int p = tid < TC && j < a.BM ? a.sorted[(int64_t)blk * a.BM + j] : a.numel;
  const int ncol = put_pairs<TC>(lds.cols, p, a);
  if (ncol == 0) return;

  const int units = a.blocks >> 2;
  const int half = a.K / 2;  // bytes of a weight row
  const char* W = (const char*)a.W + (int64_t)e * a.N * half;
  const uint8_t* ws = a.scales + (int64_t)e * a.N * a.blocks;
  int sc_to = 0, sc_at = MxTiles::ROWS * 2;  // places of the next scales to load, and of those at work
  // The loads of stage u of the tile from row n0 on: 16 columns and twice 16 weight rows a wave, and from an even u on
  // the scales of 2 * 32 rows (12 such loads, four of them twice: as many for every wave). Stages are counted
  // through the tiles: g.
  auto issue = [&](int g, int u, int n0) __attribute__((always_inline)) {
    char* to = lds.codes[g % MxTiles::STAGES];
    const int ln = opaque(lane), r = ln >> 2, at = u * 64 + ((ln & 3) ^ (r >> 2 & 3)) * 16;
    mx_dma16((const char*)a.x + lds.cols.row[wv * 16 + r] + at, to + wv * 1024);
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // (rows past the last: it again, not stored)
      const int n = min(n0 + (wv * 2 + h) * 16 + r, a.N - 1);
      mx_dma16(W + (uint32_t)n * (uint32_t)half + at, to + TC * 64 + (wv * 2 + h) * 1024);
    }
    if (u % 2 == 0) {
      const int sr = ln >> 1, sb = min(u + (ln & 1), units - 1) * 4;
      uint32_t* sto = lds.scales[0] + sc_to;
      const int c = (wv & 3) * 32 + sr;
      mx_dma4(a.x_scales + (int64_t)fdiv(lds.cols.pair[min(c, ncol - 1)], a.f_rd) * a.ld_xs + sb, sto + (wv & 3) * 64);
      const int n = min(n0 + wv * 32 + sr, a.N - 1);
      mx_dma4(ws + (int64_t)n * a.blocks + sb, sto + (TC / 32 + wv) * 64);
      sc_to ^= MxTiles::ROWS * 2;  // (the two places of scales alternate)
    }
  };
  const int wn = wv & 3, wc = wv >> 2;
  f32x4_t acc[4][4];
  auto clear = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int f = 0; f < 4; ++f) acc[t][f] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  };
  clear();
  const int stages = tiles * units;
  int n0 = tile0 * RN, u = 0;       // of the stage at work
  int nl = n0, ul = 0;              // of the next stage to load
  int later = 0;                    // loads of the stage after the one at work
  auto load = [&](int g) __attribute__((always_inline)) {
    issue(g, ul, nl);
    later = ul % 2 == 0 ? 5 : 3;
    if (++ul == units) {
      ul = 0;
      nl += RN;
    }
  };
  load(0);
  later = 0;
  if (stages > 1) load(1);
  for (int g = 0; g < stages; ++g) {
    // stage g has arrived, this wave's part and then everyone's; the one after it may be on its way
    if (later == 0) mx_wait<0>();
    else if (later == 3) mx_wait<3>();
    else mx_wait<5>();
    __builtin_amdgcn_s_barrier();
    later = 0;
    if (g + 2 < stages) load(g + 2);  // (over stage g - 1, which all waves are done with)
    if (u % 2 == 0) sc_at ^= MxTiles::ROWS * 2;
    if (wc * 64 < ncol) {
      const int ln = opaque(lane), r = ln & 15, quad = ln >> 4;
      const char* x = lds.codes[g % MxTiles::STAGES] + (wc * 64 + r) * 64 + (quad ^ (r >> 2)) * 16;
      const char* w = x + (TC + wn * 64 - wc * 64) * 64;
      const uint8_t* xs = (const uint8_t*)(lds.scales[0] + sc_at + (wc * 64 + r) * 2 + u % 2) + quad;
      const uint8_t* wsc = xs + (TC + wn * 64 - wc * 64) * 8;
      i32x8_t wf[4];
      int wsf[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const uint4 v = *reinterpret_cast<const uint4*>(w + f * 1024);
        wf[f] = i32x8_t{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
        wsf[f] = wsc[f * 128];
      }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint4 v = *reinterpret_cast<const uint4*>(x + t * 1024);
        const i32x8_t xf = {(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0};
        const int xsf = xs[t * 128];
#pragma unroll
        for (int f = 0; f < 4; ++f)
          acc[t][f] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[f], xf, acc[t][f], 4, 4, 0, wsf[f], 0, xsf);
      }
    }
    if (++u == units) {
      if (wc * 64 < ncol) {
        const int ln = opaque(lane);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int c = wc * 64 + t * 16 + (ln & 15);
          mx_store_tiles<OBF16, 4>(a, c < ncol, lds.cols.pair[c], n0 + wn * 64, ln >> 4, acc[t]);
        }
        clear();
      }
      u = 0;
      n0 += RN;
    }
  }
}

template <bool OBF16>
hipError_t mx4_tiles(MxGemmArgs a, hipStream_t st) {
  const int32_t tiles = (a.N + MxTiles::RN - 1) / MxTiles::RN;
  const int32_t spans = (a.BM + MxTiles::TC - 1) / MxTiles::TC;
  a.run = 1;
  while (a.run < 4 && (int64_t)a.max_blocks * spans * tiles >= 2 * a.run * 2048) a.run *= 2;
  const int32_t runs = (tiles + a.run - 1) / a.run;
  a.f_tiles = make_fastdiv((uint32_t)runs);
  a.items = runs * ((a.BM + MxTiles::TC - 1) / MxTiles::TC);
  a.f_items = make_fastdiv((uint32_t)a.items);
  // (a range for each XCD, rounded up)
  const int64_t grid = ((int64_t)a.max_blocks * a.items + 7) / 8 * 8;
  hipLaunchKernelGGL((mx4_tiles_kernel<OBF16>), dim3((unsigned)grid), dim3(512), 0, st, a);
  return hipGetLastError();
}

}  // namespace
}  // namespace mol
