// A whole mixture-of-experts layer for a few tokens. Per pair p = (token m, slot k) with base
// expert t in [0, E), and l the token's adapter slot:
//   g, u = Wg_t x_m (+ c_l Bg (Ag x_m)),  Wu_t x_m (+ c_l Bu (Au x_m))
//   h_p  = silu(g) * u
//   y_m  = round( sum_k w_mk (Wd_t h_p (+ c_l Bd (Ad h_p))) )
// Everything between x and y is fp32; where h is an operand of a bf16 product it is two bf16
// planes (16 bits of it), so y carries one rounding to bf16.
//
// Launches: gate/up, down, and the combine (with adapters the activation too); without adapters,
// and for very few tokens, down and the combine are one (moe_layer_direct.hip). No launch routes: a
// workgroup finds its pairs among the M * topk ids itself, which is cheaper than a launch.
//
// Gate/up and down stream weight rows (skinny.h): a work item is 64 rows of one expert or more, for
// all the pairs that use it (16 rows and split k's where 64 make too few items). Up to E pairs the
// items are per pair, and a pair whose expert an earlier pair has exits; beyond, per expert (128
// experts, top-8, queued calls per pair and per expert: 1 token 21.1 and 31.9 us, 4 tokens 60 and 76, 8
// tokens 100 and 107, 16 tokens 150 and 152). The adapters run beside the base product, in the same
// launch: an item per virtual expert forms s = A x for its pairs, keeps it in LDS and writes c B s as
// fp32 rows, which the activation (then a launch of its own) and the combine add to the base rows. Their
// latency (a dependent chain over a few hundred KiB) hides behind the base product's stream, so these
// items come first in the grid; as launches of their own before each stage they took 13 and 6 us more at 23
// tokens, 59 and 23 at 128.
//
// Bound by the stream of weights out of HBM. bf16, 128 experts, hidden 2048, inter 768, top-8:
//   1 token, no adapters      gate/up 13.3 us (50 MB, 3.8 TB/s), direct down 7.9
//   23 tokens, rank 32 of 8   gate/up 122 us (660 MB, 5.4 TB/s), down 65 (340 MB, 5.2), act 4.8,
//                             combine 4.8
//   128 tokens, rank 32 of 16 gate/up 192 us, down 109, act 6.5, combine 5.5
// 4-bit base weights, 23 tokens: gate/up 55 us, down 35 (230 + 90 MB with the adapters: bound like
// the 4-bit product, by the latency of items and the unpacking; groups of 32 spill registers there too).
#pragma once

#include <algorithm>

#include "mol.h"
#include "skinny.h"

namespace mol {
namespace {

// base expert of pair p, or -1
__device__ __forceinline__ int pair_expert(const LayerArgs& a, int p) {
  const int t = a.ids[p];
  return (unsigned)t < (unsigned)a.E ? t : -1;
}

// rank of the adapter of pair p's token (0: none), and its slot
__device__ __forceinline__ int pair_rank(const LayerArgs& a, int p, int& slot) {
  const int l = a.lora[fdiv(p, a.f_topk)];
  slot = (unsigned)l < (unsigned)a.S ? l : 0;
  const int rl = a.ranks ? a.ranks[slot] : a.r;
  return slot != l ? 0 : rl < 0 ? 0 : rl > a.r ? a.r : rl;
}

// the matrix that pair p uses: its base expert, or (VIRT) its virtual expert; -1 for none
template <bool VIRT>
__device__ __forceinline__ int pair_key(const LayerArgs& a, int p) {
  const int t = pair_expert(a, p);
  if constexpr (!VIRT) return t;
  int l;
  const int rank = pair_rank(a, p, l);
  return t < 0 || rank == 0 ? -1 : t + l * a.E;
}

// The pairs of a matrix, in ascending order, those of rank j0 .. j0 + kMaxCols - 1 among them (LDS).
struct PairList {
  int pair[kMaxCols];
  int hits[kWaves];
};
// The matrix of a work item (negative: nothing to do), how many pairs use it and the first of them.
struct PairsOf {
  int key;
  int total;
  int first;
};

// Up to this many every wave looks through all ids itself, without a barrier: eight loads in flight
// (one token: 21.3 us a layer, against 23.1 with quarters and barriers).
constexpr int kFewPairs = 512;

// Fills the list. key: t, or (VIRT) t + l E; the caller knows that slot l has a rank. All loads of a
// batch of ids are in flight together. Up to kFewPairs there is no barrier: each wave finds the pairs,
// wave 0 writes them down, and the list may be read after the caller's next barrier. Beyond, each
// wave looks through a quarter of a batch, and the list may be read on return.
template <bool VIRT>
__device__ __forceinline__ PairsOf list_pairs(const LayerArgs& a, int key, int j0, PairList& list) {
  constexpr int NB = kFewPairs / 64;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = VIRT ? key / a.E : 0, t = VIRT ? key - l * a.E : key;
  const bool few = a.numel <= kFewPairs;
  PairsOf found{key, 0, 0};
  for (int i0 = 0; i0 < a.numel; i0 += kWaves * kFewPairs) {
    // this wave's ids: whole 64s, contiguous, as even as that allows
    const int left = min(a.numel - i0, kWaves * kFewPairs);
    const int per = few ? (left + 63) / 64 : (left + kThreads - 1) / kThreads;  // 64s a wave
    const int base = few ? 0 : i0 + wv * per * 64;
    int id[NB], sl[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int i = min(base + b * 64 + lane, a.numel - 1);
      id[b] = a.ids[i];
      if constexpr (VIRT) sl[b] = a.lora[fdiv(i, a.f_topk)];
    }
    uint64_t m[NB];
    int mine = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const bool hit = b < per && base + b * 64 + lane < a.numel && id[b] == t &&
                       (!VIRT || sl[b] == l);
      m[b] = __builtin_amdgcn_ballot_w64(hit);
      mine += __popcll(m[b]);
    }
    int at = found.total, before = found.total;
    if (few) {
      found.total = mine;
    } else {
      if (lane == 0) list.hits[wv] = mine;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const int h = list.hits[w];
        at += w < wv ? h : 0;
        found.total += h;
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if ((m[b] >> lane) & 1) {
        const int r = at + __popcll(m[b] & ((1ull << lane) - 1)) - j0;
        if (r >= 0 && r < kMaxCols && (!few || wv == 0)) list.pair[r] = base + b * 64 + lane;
      }
      if (few && at == 0 && m[b]) found.first = b * 64 + __builtin_ctzll(m[b]);
      at += __popcll(m[b]);
    }
    if (!few) {
      __syncthreads();
      if (before == 0 && found.total > 0 && j0 == 0) found.first = list.pair[0];
    }
  }
  return found;
}

// The matrix of this work item and its pairs. By pair (slot = a pair): an earlier pair with the same
// matrix takes it.
template <bool VIRT>
__device__ __forceinline__ PairsOf find_pairs(const LayerArgs& a, int slot, bool by_pair,
                                              PairList& list) {
  int key = slot;
  if (by_pair) {
    key = pair_key<VIRT>(a, slot);
  } else if constexpr (VIRT) {
    const int l = slot / a.E;
    if (a.ranks && a.ranks[l] <= 0) key = -1;
  }
  key = __builtin_amdgcn_readfirstlane(key);
  if (key < 0) return {-1, 0, 0};
  PairsOf found = list_pairs<VIRT>(a, key, 0, list);
  if (found.total == 0 || (by_pair && found.first != slot)) found.key = -1;
  return found;
}

// h of the pairs.
template <bool BF16>
struct HSrc {
  const LayerArgs& a;
  const int* pair;  // of each column (LDS)
  __device__ __forceinline__ const char* row(int col) const {
    return (const char*)a.h + (int64_t)__builtin_amdgcn_readfirstlane(pair[col]) * a.I * 4;
  }
  __device__ __forceinline__ const char* lane_row(int col) const {
    return (const char*)a.h + (int64_t)pair[col] * a.I * 4;
  }
  __device__ __forceinline__ XVec operator()(const char* row, int v) const {
    return PlaneSrc<BF16>{a.I}(row, v);
  }
};

// The activation on its own, where the adapters' part has to be added first: h of pair blockIdx.y from
// its base rows g, u and the adapters' part of them.
template <bool BF16>
__global__ void __launch_bounds__(64) layer_act_kernel(LayerArgs a) {
  constexpr int VE = BF16 ? 8 : 4;
  const int p = (int)blockIdx.y, v = (int)blockIdx.x * 64 + (int)threadIdx.x;
  if (pair_expert(a, p) < 0 || v * VE >= a.I) return;
  int l;
  const bool add = pair_rank(a, p, l) > 0;
  const float* gu = a.gu + (int64_t)p * 2 * a.I + v * VE;
  const float* d = (add ? a.rank_gu.d : a.gu) + (int64_t)p * 2 * a.I + v * VE;
  float h[VE];
#pragma unroll
  for (int q = 0; q < VE; q += 4) {
    const f32x4_t g = *reinterpret_cast<const f32x4_t*>(gu + q);
    const f32x4_t u = *reinterpret_cast<const f32x4_t*>(gu + a.I + q);
    const f32x4_t dg = *reinterpret_cast<const f32x4_t*>(d + q);
    const f32x4_t du = *reinterpret_cast<const f32x4_t*>(d + a.I + q);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      h[q + i] = silu(add ? g[i] + dg[i] : g[i]) * (add ? u[i] + du[i] : u[i]);
  }
  const XVec s = split_vec<BF16>(h);
  char* o = (char*)a.h + (int64_t)p * a.I * 4 + v * 16;
  *reinterpret_cast<uint4*>(o) = s.hi;
  if constexpr (BF16) *reinterpret_cast<uint4*>(o + a.I * 2) = s.lo;
}

// The adapter part of one stage for the pairs of virtual expert v, rank rl (> 0):
//   d[p, g w + n] = c sum_{j < rl} B_v[g w + n, j] s[p, g r + j],  s[p] = A_v (input row of p)
// over `slices` slices of w rows. s stays in LDS (cols x R floats behind the stream's part). Rows
// of A and elements of B past the slot's rank are not read.
template <bool BF16, int NP, class Src>
__device__ __forceinline__ void rank_part(const LayerArgs& a, const RankPart& rp, PairList& list,
                                          char* lds, const PairsOf& of, const Src& src) {
  constexpr int ESZ = BF16 ? 2 : 4, VE = 16 / ESZ, KL = 4 * VE, COLS = 16;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  int slot;
  const int v = of.key, total = of.total;
  const int rl = __builtin_amdgcn_readfirstlane(pair_rank(a, of.first, slot));
  const float scale = a.scale[slot];
  const int R = rp.slices * a.r, w = rp.N / rp.slices;
  float* s = reinterpret_cast<float*>(lds + StreamLds<0, BF16>::kBytes);
  const int64_t abytes = (int64_t)R * rp.K * ESZ, bbytes = (int64_t)rp.N * a.r * ESZ;
  const __amdgpu_buffer_rsrc_t ra = expert_rsrc((const char*)rp.A + (int64_t)v * abytes, abytes);
  const __amdgpu_buffer_rsrc_t rb = expert_rsrc((const char*)rp.B + (int64_t)v * bbytes, bbytes);
  auto in_rank = [&](int row) { return row < R && row % a.r < rl; };
  for (int j0 = 0; j0 < total; j0 += COLS) {
    if (j0 > 0) {
      __syncthreads();
      list_pairs<true>(a, v, j0, list);
    }
    const int ncol = min(COLS, total - j0);
    for (int r0 = 0; r0 < R; r0 += kItemRows) {
      const int row0 = wave_row0<1>(r0);
      auto row_at = [&](int i) {
        const int row = row0 + i;
        return RowAt{in_rank(row) ? (uint32_t)row * (uint32_t)(rp.K * ESZ) : kOutOfRange, -1};
      };
      auto keep = [&](int c, const f32x4_t& acc) {
        if (c >= ncol) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = row0 + quad * 4 + i;
          if (at < R) s[c * R + at] = in_rank(at) ? acc[i] : 0.f;
        }
      };
      if (ncol <= 4)
        stream_k<0, BF16, 4, NP, 1>(lds, ra, row_at(col), row_at, Q4Tables{}, src, ncol, rp.K, r0 > 0,
                                    keep);
      else
        stream_k<0, BF16, 16, NP, 1>(lds, ra, row_at(col), row_at, Q4Tables{}, src, ncol, rp.K,
                                     r0 > 0, keep);
    }
    __syncthreads();
    // B s: the operand rows of B are 16 bytes of rank a lane and step, s in two planes (bf16)
    constexpr int NT = 4;  // tiles in flight
    const int p = col < ncol ? list.pair[col] : 0;
    const float* sc = s + (col < ncol ? col : 0) * R;
    for (int g = 0; g < rp.slices; ++g) {
      for (int t0 = wv; t0 * kTileRows < w; t0 += NT * kWaves) {
        f32x4_t acc[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        for (int k0 = 0; k0 < rl; k0 += KL) {
          const int k = k0 + quad * VE;
          uint4 b[NT];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const int n = (t0 + t * kWaves) * kTileRows + col;
            b[t] = buf16(rb, n < w && k < rl ? (uint32_t)((g * w + n) * a.r + k) * ESZ
                                             : kOutOfRange);
          }
          float f[VE];
#pragma unroll
          for (int j = 0; j < VE; ++j) f[j] = k + j < rl ? sc[g * a.r + k + j] : 0.f;
          const XVec sv = split_vec<BF16>(f);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            const uint4 bk = keep_first<BF16>(b[t], rl - k);
            acc[t] = mma16<BF16>(bk, sv.hi, acc[t]);
            if constexpr (BF16) acc[t] = mma16<BF16>(bk, sv.lo, acc[t]);
          }
        }
        // An infinite element of B gives NaN beside a second plane of zeros: sums that are not finite once
        // more, term by term (where s holds a NaN they all are, and stay).
        bool odd = false;
        if constexpr (BF16) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) odd |= col < ncol && !__builtin_isfinite(acc[t][i]);
        }
        if (odd) {
          bool nan = false;
          for (int k = 0; k < rl; ++k) nan |= sc[g * a.r + k] != sc[g * a.r + k];
          const uint16_t* B = (const uint16_t*)rp.B + (int64_t)v * rp.N * a.r;
#pragma unroll 1
          for (int j = 0; j < 4 * NT && !nan; ++j) {
            const int n = (t0 + (j >> 2) * kWaves) * kTileRows + quad * 4 + (j & 3);
            float sum = 0.f;
            for (int k = 0; n < w && k < rl; ++k)
              sum = fmaf(bf16_lo(B[(g * w + n) * a.r + k]), sc[g * a.r + k], sum);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc[t][i] = t * 4 + i == j && !__builtin_isfinite(acc[t][i]) ? sum : acc[t][i];
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int n = (t0 + t * kWaves) * kTileRows + quad * 4;
          if (col < ncol && n < w) {  // w is a multiple of 4
            acc[t] *= scale;
            *reinterpret_cast<f32x4_t*>(rp.d + (int64_t)p * rp.N + g * w + n) = acc[t];
          }
        }
      }
    }
  }
}

template <int G, bool BF16, bool LORA, int KS>
__global__ void __launch_bounds__(kThreads, G == 0 || G == 128 ? 4 : 3) gate_up_kernel(LayerArgs a) {
  __shared__ PairList list;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const RowSrc src{(const char*)a.x, a.ld_x * (BF16 ? 2 : 4), list.pair, a.f_topk};
  int b = (int)blockIdx.x;
  if constexpr (LORA) {
    if (b < a.rank_slots) {
      const PairsOf of = find_pairs<true>(a, b, a.rank_by_pair, list);
      if (of.key >= 0) rank_part<BF16, 1>(a, a.rank_gu, list, lds, of, src);
      return;
    }
    b -= a.rank_slots;
  }
  const int slot = fdiv(b, a.f_gu_items);
  const int n0 = (b - slot * a.gu_items) * (KS > 1 ? kTileRows : kItemRows * a.gu_tiles);
  const PairsOf of = find_pairs<false>(a, slot, a.by_pair, list);
  const int e = of.key, total = of.total;
  if (e < 0) return;
  const int lane = threadIdx.x & 63, quad = lane >> 4;
  const int64_t rb = row_bytes<G, BF16>(a.H), wbytes = 2 * a.I * rb;
  const __amdgpu_buffer_rsrc_t rsrc = expert_rsrc((const char*)a.W_gu + (int64_t)e * wbytes, wbytes);
  const Q4Tables q{a.sc_gu, a.z_gu, G ? a.H / (G ? G : 1) : 0};
  for (int j0 = 0; j0 < total; j0 += kPassCols<G, BF16, 1, KS>) {
    if (j0 > 0) {
      __syncthreads();
      list_pairs<false>(a, e, j0, list);
    }
    const int ncol = min(kPassCols<G, BF16, 1, KS>, total - j0);
#pragma unroll 1
    for (int t = 0; t < (KS > 1 ? 1 : a.gu_tiles); ++t) {
      // With adapters the tile is 16 consecutive rows of gate and up; without, 8 gate rows and
      // their up rows, the two of a column in one lane: rows 4 q, 4 q + 1 are gate columns i0 + 2 q,
      // + 1 and rows 4 q + 2, 4 q + 3 the same up columns (i0 half of the tile's first row).
      const int r0 = wave_row0<KS>(n0 + t * kItemRows);
      auto row_at = [&](int r) {
        int n;
        if constexpr (LORA) {
          n = r0 + r < 2 * a.I ? r0 + r : -1;
        } else {
          const int i = r0 / 2 + (r >> 2) * 2 + (r & 1);
          n = i < a.I ? ((r & 2) ? a.I : 0) + i : -1;
        }
        return n >= 0 ? RowAt{(uint32_t)(n * rb), (int64_t)e * 2 * a.I + n} : RowAt{kOutOfRange, -1};
      };
      stream_cols<G, BF16, 1, KS>(
          lds, rsrc, row_at(lane & 15), row_at, q, src, ncol, a.H, t > 0,
          [&](int c, const f32x4_t& acc) {
            if (c >= ncol) return;
            const int64_t p = list.pair[c];
            if constexpr (LORA) {
              const int at = r0 + quad * 4;  // 2 I is a multiple of 4
              if (at < 2 * a.I) *reinterpret_cast<f32x4_t*>(a.gu + p * 2 * a.I + at) = acc;
            } else {
              const int i = r0 / 2 + quad * 2;  // I is a multiple of 2
              if (i >= a.I) return;
              float h[2];
#pragma unroll
              for (int j = 0; j < 2; ++j) h[j] = silu(acc[j]) * acc[2 + j];
              if constexpr (BF16) {
                const float f[8] = {h[0], h[1], 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                const XVec s = split_vec<true>(f);
                uint16_t* o = (uint16_t*)a.h + p * 2 * a.I + i;
                *reinterpret_cast<uint32_t*>(o) = s.hi.x;
                *reinterpret_cast<uint32_t*>(o + a.I) = s.lo.x;
              } else {
                *reinterpret_cast<float2*>((float*)a.h + p * a.I + i) = make_float2(h[0], h[1]);
              }
            }
          });
    }
  }
}

template <int G, bool BF16, bool LORA, int KS>
__global__ void __launch_bounds__(kThreads, G == 0 || G == 128 ? 4 : 3) down_kernel(LayerArgs a) {
  constexpr int NP = BF16 ? 2 : 1;
  __shared__ PairList list;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const HSrc<BF16> src{a, list.pair};
  int b = (int)blockIdx.x;
  if constexpr (LORA) {
    if (b < a.rank_slots) {
      const PairsOf of = find_pairs<true>(a, b, a.rank_by_pair, list);
      if (of.key >= 0) rank_part<BF16, NP>(a, a.rank_dn, list, lds, of, src);
      return;
    }
    b -= a.rank_slots;
  }
  const int slot = fdiv(b, a.f_dn_items);
  const int n0 = (b - slot * a.dn_items) * (KS > 1 ? kTileRows : kItemRows * a.dn_tiles);
  const PairsOf of = find_pairs<false>(a, slot, a.by_pair, list);
  const int e = of.key, total = of.total;
  if (e < 0) return;
  const int lane = threadIdx.x & 63, quad = lane >> 4;
  const int64_t rb = row_bytes<G, BF16>(a.I), wbytes = a.H * rb;
  const __amdgpu_buffer_rsrc_t rsrc = expert_rsrc((const char*)a.W_dn + (int64_t)e * wbytes, wbytes);
  const Q4Tables q{a.sc_dn, a.z_dn, G ? a.I / (G ? G : 1) : 0};
  for (int j0 = 0; j0 < total; j0 += kPassCols<G, BF16, NP, KS>) {
    if (j0 > 0) {
      __syncthreads();
      list_pairs<false>(a, e, j0, list);
    }
    const int ncol = min(kPassCols<G, BF16, NP, KS>, total - j0);
#pragma unroll 1
    for (int t = 0; t < (KS > 1 ? 1 : a.dn_tiles); ++t) {
      const int r0 = wave_row0<KS>(n0 + t * kItemRows);
      auto row_at = [&](int i) {
        const int n = r0 + i;
        return n < a.H ? RowAt{(uint32_t)(n * rb), (int64_t)e * a.H + n} : RowAt{kOutOfRange, -1};
      };
      stream_cols<G, BF16, NP, KS>(
          lds, rsrc, row_at(lane & 15), row_at, q, src, ncol, a.I, t > 0,
          [&](int c, const f32x4_t& acc) {
            const int at = r0 + quad * 4;  // H is a multiple of 4
            if (c < ncol && at < a.H)
              *reinterpret_cast<f32x4_t*>(a.z + (int64_t)list.pair[c] * a.H + at) = acc;
          });
    }
  }
}

// y[m, n] = sum over the token's pairs of their weighted rows (and the adapters'), four columns
// a thread, token blockIdx.y
template <bool BF16, bool LORA>
__global__ void __launch_bounds__(64) layer_combine_kernel(LayerArgs a) {
  const int m = (int)blockIdx.y, n = ((int)blockIdx.x * 64 + (int)threadIdx.x) * 4;
  if (n >= a.H) return;
  bool add = false;
  if constexpr (LORA) {
    int l;
    add = pair_rank(a, m * a.topk, l) > 0;
  }
  f32x4_t y = {0.f, 0.f, 0.f, 0.f};
  constexpr int NB = 8;  // pairs in flight; every load is issued, unused ones on the token's first
  for (int k0 = 0; k0 < a.topk; k0 += NB) {
    f32x4_t v[NB], d[NB];
    float w[NB];
    bool there[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int p = m * a.topk + min(k0 + b, a.topk - 1);
      there[b] = k0 + b < a.topk && pair_expert(a, p) >= 0;
      w[b] = a.weights[p];
      v[b] = *reinterpret_cast<const f32x4_t*>(a.z + (int64_t)p * a.H + n);
      if constexpr (LORA) d[b] = *reinterpret_cast<const f32x4_t*>(a.rank_dn.d + (int64_t)p * a.H + n);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float x = LORA && add ? v[b][j] + d[b][j] : v[b][j];
        y[j] = there[b] ? fmaf(w[b], x, y[j]) : y[j];
      }
    }
  }
  const int64_t o = (int64_t)m * a.ld_y + n;
#pragma unroll
  for (int j = 0; j < 4; ++j) store_elem<BF16>(a.y, o + j, y[j]);
}

template <int G, bool BF16, bool LORA, int KS>
void launch_gate_up(const LayerArgs& a, int grid, size_t lds, hipStream_t st) {
  hipLaunchKernelGGL((gate_up_kernel<G, BF16, LORA, KS>), dim3(grid), dim3(kThreads), lds, st, a);
}
template <int G, bool BF16, bool LORA, int KS>
void launch_down(const LayerArgs& a, int grid, size_t lds, hipStream_t st) {
  hipLaunchKernelGGL((down_kernel<G, BF16, LORA, KS>), dim3(grid), dim3(kThreads), lds, st, a);
}

template <int G, bool BF16, bool LORA>
hipError_t layer(const LayerArgs& a, hipStream_t st) {
  const int rank = LORA ? a.rank_slots : 0;
  // the stream's LDS; behind a dense one's, s of an adapter item (16 columns)
  auto lds = [&](int R) {
    const size_t s = LORA ? (size_t)StreamLds<0, BF16>::kBytes + 16 * (size_t)R * sizeof(float) : 0;
    return std::max<size_t>(StreamLds<G, BF16>::kBytes, s);
  };
  const int gu = rank + a.slots * a.gu_items, dn = rank + a.slots * a.dn_items;
  const size_t lds_gu = lds(2 * a.r), lds_dn = lds(a.r);
  if (a.gu_split) launch_gate_up<G, BF16, LORA, kWaves>(a, gu, lds_gu, st);
  else launch_gate_up<G, BF16, LORA, 1>(a, gu, lds_gu, st);
  hipError_t r = hipGetLastError();
  if (r != hipSuccess) return r;
  if (!LORA && a.direct) return launch_moe_layer_direct(a, BF16, st);
  if constexpr (LORA) {
    constexpr int VE = BF16 ? 8 : 4;
    hipLaunchKernelGGL((layer_act_kernel<BF16>), dim3((a.I / VE + 63) / 64, a.numel), dim3(64), 0, st,
                       a);
    if ((r = hipGetLastError()) != hipSuccess) return r;
  }
  if (a.dn_split) launch_down<G, BF16, LORA, kWaves>(a, dn, lds_dn, st);
  else launch_down<G, BF16, LORA, 1>(a, dn, lds_dn, st);
  if ((r = hipGetLastError()) != hipSuccess) return r;
  hipLaunchKernelGGL((layer_combine_kernel<BF16, LORA>), dim3((a.H / 4 + 63) / 64, a.M), dim3(64), 0,
                     st, a);
  return hipGetLastError();
}

}  // namespace

// The layer over weights of group G: one translation unit each.
template <int G>
hipError_t launch_layer_group(const LayerArgs& a, bool bf16, hipStream_t st) {
  if (a.lora) return bf16 ? layer<G, true, true>(a, st) : layer<G, false, true>(a, st);
  return bf16 ? layer<G, true, false>(a, st) : layer<G, false, false>(a, st);
}

}  // namespace mol
