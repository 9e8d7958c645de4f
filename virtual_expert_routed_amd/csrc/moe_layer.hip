// A whole mixture-of-experts layer for a few tokens. Per pair p = (token m, slot k) with base
// expert t in [0, E), and l the token's adapter slot:
//   g, u = Wg_t x_m (+ c_l Bg (Ag x_m)),  Wu_t x_m (+ c_l Bu (Au x_m))
//   h_p  = silu(g) * u
//   y_m  = round( sum_k w_mk (Wd_t h_p (+ c_l Bd (Ad h_p))) )
// Everything between x and y is fp32; where h is an operand of a bf16 product it is two bf16
// planes (16 bits of it), so y carries one rounding to bf16.
//
// Launches: gate/up, down, and the combine; without adapters, and for few tokens, down and the
// combine are one (moe_layer_direct.hip). No launch routes: a workgroup finds its pairs among the M
// * topk ids itself, which is cheaper than a launch.
//
// Gate/up and down stream weight rows (skinny.h): a work item is 64 rows of one expert for all the
// pairs that use it (16 rows and split k's where 64 make too few items). Up to E pairs the
// items are per pair, and a pair whose expert an earlier pair has exits; beyond, per expert.
// The adapters run beside the base product, in the same launch: an item per virtual expert forms
// s = A x for its pairs, keeps it in LDS and writes c B s as fp32 rows, which the next launch
// adds to the base rows where it reads them. Their latency (a dependent chain over a few hundred KiB)
// hides behind the base product's stream, so these items come first in the grid.
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

// The pairs of a matrix, in ascending order, those of rank j0 .. j0 + kMaxCols - 1 among them.
struct PairList {
  int pair[kMaxCols];
  int total;  // of the matrix
  int first;  // the first of them (j0 = 0)
};
template <bool VIRT>
__device__ __forceinline__ void list_pairs(const LayerArgs& a, int key, int j0, PairList& list) {
  if (threadIdx.x < 64) {
    constexpr int NB = VIRT ? 2 : 4;  // ids in flight
    int n = 0;
    for (int i0 = 0; i0 < a.numel; i0 += 64 * NB) {
      int k[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b)
        k[b] = pair_key<VIRT>(a, min(i0 + b * 64 + (int)threadIdx.x, a.numel - 1));
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int i = i0 + b * 64 + (int)threadIdx.x;
        const bool hit = i < a.numel && k[b] == key;
        const uint64_t m = __builtin_amdgcn_ballot_w64(hit);
        const int at = n + __popcll(m & ((1ull << threadIdx.x) - 1)) - j0;
        if (hit && at >= 0 && at < kMaxCols) list.pair[at] = i;
        if (hit && at + j0 == 0) list.first = i;
        n += __popcll(m);
      }
    }
    if (threadIdx.x == 0) list.total = n;
  }
  __syncthreads();
}

// The matrix of this work item and its pairs; negative for a workgroup with nothing to do. By pair
// (slot = a pair): an earlier pair with the same matrix takes it.
template <bool VIRT>
__device__ __forceinline__ int find_pairs(const LayerArgs& a, int slot, bool by_pair,
                                          PairList& list) {
  const int key = __builtin_amdgcn_readfirstlane(by_pair ? pair_key<VIRT>(a, slot) : slot);
  if (key < 0) return -1;
  list_pairs<VIRT>(a, key, 0, list);
  return list.total == 0 || (by_pair && list.first != slot) ? -1 : key;
}

// h of the pairs, from where the gate/up launch left it: without adapters, h itself (bf16: the two
// planes); with them, the base rows g, u and the adapters' part of them, both fp32.
template <bool BF16, bool LORA>
struct HSrc {
  static constexpr int VE = BF16 ? 8 : 4;
  const LayerArgs& a;
  const int* pair;  // of each column (LDS)
  struct Row {
    const char* p;
    const char* d;
    bool add;
  };
  __device__ __forceinline__ Row row(int col) const {
    const int p = __builtin_amdgcn_readfirstlane(pair[col]);
    if constexpr (LORA) {
      int l;
      const bool add = pair_rank(a, p, l) > 0;
      const int64_t at = (int64_t)p * 2 * a.I * 4;
      return {(const char*)a.gu + at, (const char*)(add ? a.d1 : a.gu) + at, add};
    } else {
      return {(const char*)a.h + (int64_t)p * a.I * (BF16 ? 4 : 4), nullptr, false};
    }
  }
  __device__ __forceinline__ XVec operator()(const Row& r, int v) const {
    if constexpr (!LORA) {
      const uint4 hi = ld16(r.p + (uint32_t)v * 16u);
      return {hi, BF16 ? ld16(r.p + (uint32_t)a.I * 2u + (uint32_t)v * 16u) : hi};
    } else {
      float h[VE];
#pragma unroll
      for (int q = 0; q < VE / 4; ++q) {
        const uint32_t at = (uint32_t)(v * VE + q * 4) * 4u, up = at + (uint32_t)a.I * 4u;
        const uint4 g4 = ld16(r.p + at), u4 = ld16(r.p + up);
        const uint4 dg = ld16(r.d + at), du = ld16(r.d + up);
        const uint32_t gw[4] = {g4.x, g4.y, g4.z, g4.w}, uw[4] = {u4.x, u4.y, u4.z, u4.w};
        const uint32_t dgw[4] = {dg.x, dg.y, dg.z, dg.w}, duw[4] = {du.x, du.y, du.z, du.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float g = __uint_as_float(gw[i]) + (r.add ? __uint_as_float(dgw[i]) : 0.f);
          const float u = __uint_as_float(uw[i]) + (r.add ? __uint_as_float(duw[i]) : 0.f);
          h[q * 4 + i] = g / (1.f + expf(-g)) * u;
        }
      }
      return split_vec<BF16>(h);
    }
  }
};

// The adapter part of one stage for the pairs of virtual expert v, rank rl (> 0):
//   d[p, g w + n] = c sum_{j < rl} B_v[g w + n, j] s[p, g r + j],  s[p] = A_v (input row of p)
// over `slices` slices of w rows. s stays in LDS (cols x R floats behind the stream's part). Rows
// of A and elements of B past the slot's rank are not read.
template <bool BF16, int NP, class Src>
__device__ __forceinline__ void rank_part(const LayerArgs& a, const RankPart& rp, PairList& list,
                                          char* lds, int v, const Src& src) {
  constexpr int ESZ = BF16 ? 2 : 4, VE = 16 / ESZ, KL = 4 * VE, COLS = 16;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  int slot;
  const int rl = __builtin_amdgcn_readfirstlane(pair_rank(a, list.first, slot));
  const float scale = a.scale[slot];
  const int R = rp.slices * a.r, w = rp.N / rp.slices;
  float* s = reinterpret_cast<float*>(lds + StreamLds<0>::kBytes);
  const int64_t abytes = (int64_t)R * rp.K * ESZ, bbytes = (int64_t)rp.N * a.r * ESZ;
  const __amdgpu_buffer_rsrc_t ra = expert_rsrc((const char*)rp.A + (int64_t)v * abytes, abytes);
  const __amdgpu_buffer_rsrc_t rb = expert_rsrc((const char*)rp.B + (int64_t)v * bbytes, bbytes);
  auto in_rank = [&](int row) { return row < R && row % a.r < rl; };
  const int total = list.total;
  for (int j0 = 0; j0 < total; j0 += COLS) {
    if (j0 > 0) {
      __syncthreads();
      list_pairs<true>(a, v, j0, list);
    }
    const int ncol = min(COLS, total - j0);
    for (int r0 = 0; r0 < R; r0 += kItemRows) {
      const int row0 = r0 + wv * kTileRows, row = row0 + col;
      const WeightRows wr{ra, in_rank(row) ? (uint32_t)row * (uint32_t)(rp.K * ESZ) : kOutOfRange};
      auto keep = [&](int c, const f32x4_t& acc) {
        if (c >= ncol) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = row0 + quad * 4 + i;
          if (at < R) s[c * R + at] = in_rank(at) ? acc[i] : 0.f;
        }
      };
      auto none = [](int) { return (int64_t)-1; };
      if (ncol <= 8)
        stream_rows<0, BF16, 8, NP, 1>(lds, wr, Q4Tables{}, none, row0 < R, src, ncol, rp.K, keep);
      else
        stream_rows<0, BF16, 16, NP, 1>(lds, wr, Q4Tables{}, none, row0 < R, src, ncol, rp.K, keep);
    }
    __syncthreads();
    // B s: the operand rows of B are 16 bytes of rank a lane and step, s in two planes (bf16)
    constexpr int NK = MOL_MAX_RANK_BYTES / 64;  // steps of a rank
    const int p = col < ncol ? list.pair[col] : 0;
    for (int g = 0; g < rp.slices; ++g) {
      XVec sv[NK];
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const int k = i * KL + quad * VE;
        float f[VE];
#pragma unroll
        for (int j = 0; j < VE; ++j)
          f[j] = col < ncol && k + j < rl ? s[col * R + g * a.r + k + j] : 0.f;
        sv[i] = split_vec<BF16>(f);
      }
      constexpr int NT = 4;  // tiles in flight
      for (int t0 = wv; t0 * kTileRows < w; t0 += NT * kWaves) {
        uint4 b[NT][NK];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int n = (t0 + t * kWaves) * kTileRows + col;
          const uint32_t off = n < w ? (uint32_t)((g * w + n) * a.r) * ESZ : kOutOfRange;
#pragma unroll
          for (int i = 0; i < NK; ++i) {
            const int k = i * KL + quad * VE;
            if (i * KL < a.r) b[t][i] = buf16(rb, k < rl ? off + (uint32_t)k * ESZ : kOutOfRange);
          }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int n = (t0 + t * kWaves) * kTileRows + quad * 4;
          f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < NK; ++i) {
            if (i * KL < a.r) {
              const int k = i * KL + quad * VE;
              const uint4 bk = keep_first<BF16>(b[t][i], rl - k);
              acc = mma16<BF16>(bk, sv[i].hi, acc);
              if constexpr (BF16) acc = mma16<BF16>(bk, sv[i].lo, acc);
            }
          }
          if (col < ncol && n < w) {  // w is a multiple of 4
            acc *= scale;
            *reinterpret_cast<f32x4_t*>(rp.d + (int64_t)p * rp.N + g * w + n) = acc;
          }
        }
      }
    }
  }
}

template <int G, bool BF16, bool LORA, int KS>
__global__ void __launch_bounds__(kThreads, 3) gate_up_kernel(LayerArgs a) {
  __shared__ PairList list;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const RowSrc src{(const char*)a.x, a.ld_x * (BF16 ? 2 : 4), list.pair, a.f_topk};
  int b = (int)blockIdx.x;
  if constexpr (LORA) {
    if (b < a.rank_slots) {
      const int v = find_pairs<true>(a, b, a.rank_by_pair, list);
      if (v >= 0) rank_part<BF16, 1>(a, a.rank_gu, list, lds, v, src);
      return;
    }
    b -= a.rank_slots;
  }
  constexpr int ROWS = kItemRowsOf<KS>;
  const int slot = fdiv(b, a.f_gu_items);
  const int item = b - slot * a.gu_items;
  const int e = find_pairs<false>(a, slot, a.by_pair, list);
  if (e < 0) return;
  const int lane = threadIdx.x & 63, quad = lane >> 4;
  // With adapters the tile is 16 consecutive rows of gate and up; without, 8 gate rows and their
  // up rows, the two of a column in one lane: rows 4 q, 4 q + 1 are gate columns i0 + 2 q, + 1 and
  // rows 4 q + 2, 4 q + 3 the same up columns.
  const int r0 = wave_row0<KS>(item * ROWS);
  const int i0 = r0 / 2;
  auto row_of = [&](int r) {
    if constexpr (LORA) return r0 + r < 2 * a.I ? r0 + r : -1;
    const int i = i0 + (r >> 2) * 2 + (r & 1);
    return i < a.I ? ((r & 2) ? a.I : 0) + i : -1;
  };
  const int64_t rb = row_bytes<G, BF16>(a.H), wbytes = 2 * a.I * rb;
  const int n = row_of(lane & 15);
  const WeightRows w{expert_rsrc((const char*)a.W_gu + (int64_t)e * wbytes, wbytes),
                     n >= 0 ? (uint32_t)(n * rb) : kOutOfRange};
  const Q4Tables q{a.sc_gu, a.z_gu, G ? a.H / (G ? G : 1) : 0};
  auto row_at = [&](int r) {
    const int m = row_of(r);
    return m >= 0 ? (int64_t)e * 2 * a.I + m : (int64_t)-1;
  };
  const int total = list.total;
  for (int j0 = 0; j0 < total; j0 += kPassCols<1, KS>) {
    if (j0 > 0) {
      __syncthreads();
      list_pairs<false>(a, e, j0, list);
    }
    const int ncol = min(kPassCols<1, KS>, total - j0);
    stream_cols<G, BF16, 1, KS>(lds, w, q, row_at, r0 < 2 * a.I, src, ncol, a.H,
                                [&](int c, const f32x4_t& acc) {
      if (c >= ncol) return;
      const int64_t p = list.pair[c];
      if constexpr (LORA) {
        const int at = r0 + quad * 4;  // 2 I is a multiple of 4
        if (at < 2 * a.I) *reinterpret_cast<f32x4_t*>(a.gu + p * 2 * a.I + at) = acc;
      } else {
        const int i = i0 + quad * 2;  // I is a multiple of 2
        if (i >= a.I) return;
        float h[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) h[j] = acc[j] / (1.f + expf(-acc[j])) * acc[2 + j];
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

template <int G, bool BF16, bool LORA, int KS>
__global__ void __launch_bounds__(kThreads, 3) down_kernel(LayerArgs a) {
  constexpr int NP = BF16 ? 2 : 1;
  __shared__ PairList list;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const HSrc<BF16, LORA> src{a, list.pair};
  int b = (int)blockIdx.x;
  if constexpr (LORA) {
    if (b < a.rank_slots) {
      const int v = find_pairs<true>(a, b, a.rank_by_pair, list);
      if (v >= 0) rank_part<BF16, NP>(a, a.rank_dn, list, lds, v, src);
      return;
    }
    b -= a.rank_slots;
  }
  constexpr int ROWS = kItemRowsOf<KS>;
  const int slot = fdiv(b, a.f_dn_items);
  const int item = b - slot * a.dn_items;
  const int e = find_pairs<false>(a, slot, a.by_pair, list);
  if (e < 0) return;
  const int lane = threadIdx.x & 63, quad = lane >> 4;
  const int r0 = wave_row0<KS>(item * ROWS);
  const int64_t rb = row_bytes<G, BF16>(a.I), wbytes = a.H * rb;
  const int n = r0 + (lane & 15);
  const WeightRows w{expert_rsrc((const char*)a.W_dn + (int64_t)e * wbytes, wbytes),
                     n < a.H ? (uint32_t)(n * rb) : kOutOfRange};
  const Q4Tables q{a.sc_dn, a.z_dn, G ? a.I / (G ? G : 1) : 0};
  auto row_at = [&](int r) { return r0 + r < a.H ? (int64_t)e * a.H + r0 + r : (int64_t)-1; };
  const int total = list.total;
  for (int j0 = 0; j0 < total; j0 += kPassCols<NP, KS>) {
    if (j0 > 0) {
      __syncthreads();
      list_pairs<false>(a, e, j0, list);
    }
    const int ncol = min(kPassCols<NP, KS>, total - j0);
    stream_cols<G, BF16, NP, KS>(lds, w, q, row_at, r0 < a.H, src, ncol, a.I,
                                 [&](int c, const f32x4_t& acc) {
      const int at = r0 + quad * 4;  // H is a multiple of 4
      if (c < ncol && at < a.H)
        *reinterpret_cast<f32x4_t*>(a.z + (int64_t)list.pair[c] * a.H + at) = acc;
    });
  }
}

// y[m, n] = sum over the token's pairs of their weighted rows (and the adapters'), four columns
// a thread
template <bool BF16, bool LORA>
__global__ void __launch_bounds__(kThreads) layer_combine_kernel(LayerArgs a) {
  const int groups = a.H / 4;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (int64_t)a.M * groups) return;
  const int m = (int)(i / groups), n = (int)(i - (int64_t)m * groups) * 4;
  bool add = false;
  if constexpr (LORA) {
    int l;
    add = pair_rank(a, m * a.topk, l) > 0;
  }
  f32x4_t y = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < a.topk; ++k) {
    const int p = m * a.topk + k;
    if (pair_expert(a, p) < 0) continue;
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(a.z + (int64_t)p * a.H + n);
    if (LORA && add) v += *reinterpret_cast<const f32x4_t*>(a.rank_dn.d + (int64_t)p * a.H + n);
    const float w = a.weights[p];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = fmaf(w, v[j], y[j]);
  }
  const int64_t o = (int64_t)m * a.ld_y + n;
#pragma unroll
  for (int j = 0; j < 4; ++j) store_elem<BF16>(a.y, o + j, y[j]);
}

template <int G, bool BF16, bool LORA>
hipError_t layer(const LayerArgs& a, hipStream_t st) {
  const int rank = LORA ? a.rank_slots : 0;
  // the stream's LDS; behind a dense one's, s of an adapter item (16 columns)
  auto lds = [&](int R) {
    const size_t s = LORA ? (size_t)StreamLds<0>::kBytes + 16 * (size_t)R * sizeof(float) : 0;
    return std::max<size_t>(StreamLds<G>::kBytes, s);
  };
  const dim3 gu(rank + a.slots * a.gu_items);
  if (a.gu_split)
    hipLaunchKernelGGL((gate_up_kernel<G, BF16, LORA, kWaves>), gu, dim3(kThreads), lds(2 * a.r), st, a);
  else
    hipLaunchKernelGGL((gate_up_kernel<G, BF16, LORA, 1>), gu, dim3(kThreads), lds(2 * a.r), st, a);
  hipError_t r = hipGetLastError();
  if (r != hipSuccess) return r;
  if (!LORA && a.direct) return launch_moe_layer_direct(a, BF16, st);
  const dim3 dn(rank + a.slots * a.dn_items);
  if (a.dn_split)
    hipLaunchKernelGGL((down_kernel<G, BF16, LORA, kWaves>), dn, dim3(kThreads), lds(a.r), st, a);
  else
    hipLaunchKernelGGL((down_kernel<G, BF16, LORA, 1>), dn, dim3(kThreads), lds(a.r), st, a);
  if ((r = hipGetLastError()) != hipSuccess) return r;
  const int64_t threads = (int64_t)a.M * (a.H / 4);
  hipLaunchKernelGGL((layer_combine_kernel<BF16, LORA>),
                     dim3((int)((threads + kThreads - 1) / kThreads)), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

template <int G>
hipError_t by_type(const LayerArgs& a, bool bf16, hipStream_t st) {
  if (a.lora) return bf16 ? layer<G, true, true>(a, st) : layer<G, false, true>(a, st);
  return bf16 ? layer<G, true, false>(a, st) : layer<G, false, false>(a, st);
}

}  // namespace

int moe_layer_item_rows(bool split) { return split ? kTileRows : kItemRows; }

hipError_t launch_moe_layer(const LayerArgs& a, bool bf16, hipStream_t st) {
  switch (a.group) {
    case 0: return by_type<0>(a, bf16, st);
    case 32: return by_type<32>(a, bf16, st);
    case 64: return by_type<64>(a, bf16, st);
    case 128: return by_type<128>(a, bf16, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mol
