// A whole mixture-of-experts layer for a few tokens. Per pair p = (token m, slot k) with base
// expert t in [0, E), and l the token's adapter slot:
//   g, u = Wg_t x_m (+ c_l Bg (Ag x_m)),  Wu_t x_m (+ c_l Bu (Au x_m))
//   h_p  = round(silu(g) * u)             the operand of the next product, in x's type
//   y_m  = round( sum_k w_mk (Wd_t h_p (+ c_l Bd (Ad h_p))) )
// Sums, g, u and everything else are fp32; h and y are the only values rounded to fewer bits.
//
// Launches: gate/up with the activation, then down with the combine; with adapters, the rank
// products (A x) before the first and (A h) before the second; and for many tokens the combine
// on its own (below). No launch routes: a workgroup finds its pairs among the M * topk ids itself,
// which is cheaper than a launch.
//
// Gate/up, and the rank products: a work item is 16 weight rows of one matrix (8 gate rows and
// their 8 up rows, so that the activation stays in the item) for all the pairs that use it. Up to
// E pairs, the items are per pair, and a pair whose expert an earlier pair has exits; beyond, per
// expert.
// Down, direct (few tokens): a work item is NR output columns of one token over all its pairs.
// The 16 tile rows are NR columns of 16 / NR experts, whose h rows are the tile's columns: the
// diagonal blocks of the product are the wanted sums, every loaded weight is used, and the
// weighted sum over the pairs ends in the item. Items of a column group are neighbours on one XCD,
// so an expert that several tokens share is read from that XCD's L2 again.
// Down, grouped (more tokens): items as in gate/up write each pair's weighted fp32 row, and the
// combine adds a token's rows.
#include "skinny.h"

namespace mol {
namespace {

constexpr int kXcds = 8;

// base expert of pair p, or -1
__device__ __forceinline__ int pair_expert(const LayerArgs& a, int p) {
  const int t = a.ids[p];
  return (unsigned)t < (unsigned)a.E ? t : -1;
}

// adapter slot of pair p if it has one with a rank, or -1; its rank
__device__ __forceinline__ int pair_slot(const LayerArgs& a, int p, int& rank) {
  const int l = a.lora[fdiv(p, a.f_topk)];
  rank = 0;
  if ((unsigned)l >= (unsigned)a.S) return -1;
  const int rl = a.ranks ? a.ranks[l] : a.r;
  rank = rl < 0 ? 0 : (rl > a.r ? a.r : rl);
  return rank > 0 ? l : -1;
}

// the matrix that pair p uses: its base expert, or (VIRT) its virtual expert; -1 for none
template <bool VIRT>
__device__ __forceinline__ int pair_key(const LayerArgs& a, int p) {
  const int t = pair_expert(a, p);
  if constexpr (!VIRT) return t;
  int rank;
  const int l = pair_slot(a, p, rank);
  return t < 0 || l < 0 ? -1 : t + l * a.E;
}

// The pairs of this workgroup's matrix, in ascending order: key and count, or count 0 for a
// workgroup with nothing to do. By pair (slot = a pair): an earlier pair with the key takes it.
struct PairList {
  uint16_t pair[kLayerMaxPairs];
  int count;
};
template <bool VIRT>
__device__ __forceinline__ int find_pairs(const LayerArgs& a, int slot, bool by_pair,
                                          PairList& list) {
  const int key =
      __builtin_amdgcn_readfirstlane(by_pair ? pair_key<VIRT>(a, slot) : slot);
  if (key < 0) return -1;
  if (threadIdx.x < 64) {
    int n = 0;
    for (int i0 = 0; i0 < a.numel; i0 += 64) {
      const int i = i0 + (int)threadIdx.x;
      const bool hit = i < a.numel && pair_key<VIRT>(a, i < a.numel ? i : 0) == key;
      const uint64_t m = __builtin_amdgcn_ballot_w64(hit);
      if (hit) list.pair[n + __popcll(m & ((1ull << threadIdx.x) - 1))] = (uint16_t)i;
      n += __popcll(m);
    }
    if (threadIdx.x == 0) list.count = n;
  }
  __syncthreads();
  return list.count == 0 || (by_pair && list.pair[0] != slot) ? -1 : key;
}

// <B row, s row> over the first rl ranks: B 16-byte vectors of the pair's adapter, s fp32
template <bool BF16>
__device__ __forceinline__ float rank_dot(const void* B, int64_t row, int r, int rl,
                                          const float* s) {
  constexpr int VE = BF16 ? 8 : 4;
  const char* b = (const char*)B + row * r * (BF16 ? 2 : 4);
  float d = 0.f;
  for (int j = 0; j < rl; j += VE) {
    uint4 v = ld16(b + j * (BF16 ? 2 : 4));
    if (rl < j + VE) v = keep_first<BF16>(v, rl - j);
    d = dot16_s<BF16>(v, s + j, d);
  }
  return d;
}

// s[p, i] = <A_v[i], row of p> of the pairs with an adapter; zero past the slot's rank, whose
// weights are not read. Rows per matrix: `rows` (a multiple of r); input row p / row_div.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) layer_shrink_kernel(LayerArgs a, ShrinkPart sp) {
  __shared__ PairList list;
  __shared__ float red[kWaves * kTiles * 256];
  const int slot = fdiv((int)blockIdx.x, sp.f_tiles);
  const int n0 = ((int)blockIdx.x - slot * sp.tiles) * kTileRows;
  const int v = find_pairs<true>(a, slot, sp.by_pair, list);
  if (v < 0) return;
  int rl;
  pair_slot(a, list.pair[0], rl);
  constexpr int ESZ = BF16 ? 2 : 4;
  const int n = n0 + (int)(threadIdx.x & 15);
  auto in_rank = [&](int row) { return row < sp.rows && row % a.r < rl; };
  const int64_t wbytes = (int64_t)sp.rows * sp.K * ESZ;
  const BufRow w{expert_rsrc((const char*)sp.A + (int64_t)v * wbytes, wbytes),
                 in_rank(n) ? (uint32_t)n * (uint32_t)(sp.K * ESZ) : kOutOfRange};
  auto entry = [&](int j) { return j < list.count ? (int)list.pair[j] : -1; };
  auto store = [&](int j, int r, float x) {
    const int p = entry(j);
    if (p >= 0 && n0 + r < sp.rows)
      sp.s[(int64_t)p * sp.rows + n0 + r] = in_rank(n0 + r) ? x : 0.f;
  };
  for (int j0 = 0; j0 < list.count; j0 += 16 * kTiles) {
    const int nt = min(kTiles, (list.count - j0 + 15) / 16);
    if (nt == 1)
      tile_pass<0, BF16, 1>(w, sp.x, sp.ld_x, sp.f_rd, sp.K, nullptr, entry, j0, 1, red, store);
    else
      tile_pass<0, BF16, kTiles>(w, sp.x, sp.ld_x, sp.f_rd, sp.K, nullptr, entry, j0, nt, red,
                                 store);
  }
}

// bytes of one weight row of K elements
template <int G, bool BF16>
__device__ __forceinline__ int64_t row_bytes(int K) {
  return G ? K / 2 : (int64_t)K * (BF16 ? 2 : 4);
}

template <int G, bool BF16>
__global__ void __launch_bounds__(kThreads) gate_up_kernel(LayerArgs a) {
  __shared__ PairList list;
  __shared__ float red[kWaves * kTiles * 256];
  extern __shared__ __attribute__((aligned(16))) float2 sc[];
  constexpr int HALF = kTileRows / 2;
  const int slot = fdiv((int)blockIdx.x, a.f_gu_tiles);
  const int i0 = ((int)blockIdx.x - slot * a.gu_tiles) * HALF;
  const int e = find_pairs<false>(a, slot, a.by_pair, list);
  if (e < 0) return;
  // tile rows 0-7: gate columns i0.., rows 8-15: the same up columns
  auto row_of = [&](int r) { return i0 + (r & (HALF - 1)) < a.I ? (r < HALF ? 0 : a.I) + i0 + (r & (HALF - 1)) : -1; };
  if constexpr (G > 0) {
    stage_scales<BF16>(sc, a.sc_gu, a.z_gu, a.H / G, [&](int r) {
      const int n = row_of(r);
      return n >= 0 ? (int64_t)e * 2 * a.I + n : (int64_t)-1;
    });
    __syncthreads();
  }
  const int64_t rb = row_bytes<G, BF16>(a.H), wbytes = 2 * a.I * rb;
  const int n = row_of(threadIdx.x & 15);
  const BufRow w{expert_rsrc((const char*)a.W_gu + (int64_t)e * wbytes, wbytes),
                 n >= 0 ? (uint32_t)(n * rb) : kOutOfRange};
  auto entry = [&](int j) { return j < list.count ? (int)list.pair[j] : -1; };
  auto store = [&](int j, int r, float v) {
    const int p = entry(j);
    const int row = row_of(r);
    if (a.lora && p >= 0 && row >= 0) {
      int rl;
      const int l = pair_slot(a, p, rl);
      if (l >= 0)
        v = fmaf(a.scale[l],
                 rank_dot<BF16>(a.B_gu, ((int64_t)e + (int64_t)l * a.E) * 2 * a.I + row, a.r, rl,
                                a.s1 + (int64_t)p * 2 * a.r + (r < HALF ? 0 : a.r)),
                 v);
    }
    const float up = __shfl_down(v, HALF, 16);
    if (p >= 0 && r < HALF && row >= 0)
      store_elem<BF16>(a.h, (int64_t)p * a.I + i0 + r, v / (1.f + expf(-v)) * up);
  };
  for (int j0 = 0; j0 < list.count; j0 += 16 * kTiles) {
    const int nt = min(kTiles, (list.count - j0 + 15) / 16);
    if (nt == 1)
      tile_pass<G, BF16, 1>(w, a.x, a.ld_x, a.f_topk, a.H, sc, entry, j0, 1, red, store);
    else
      tile_pass<G, BF16, kTiles>(w, a.x, a.ld_x, a.f_topk, a.H, sc, entry, j0, nt, red, store);
  }
}

// one pair's adapter part of output column n, times its slot's scale
template <bool BF16>
__device__ __forceinline__ float down_delta(const LayerArgs& a, int p, int e, int n) {
  int rl;
  const int l = pair_slot(a, p, rl);
  if (l < 0) return 0.f;
  return a.scale[l] * rank_dot<BF16>(a.B_dn, ((int64_t)e + (int64_t)l * a.E) * a.H + n, a.r, rl,
                                     a.s2 + (int64_t)p * a.r);
}

template <int G, bool BF16>
__global__ void __launch_bounds__(kThreads) down_grouped_kernel(LayerArgs a) {
  __shared__ PairList list;
  __shared__ float red[kWaves * kTiles * 256];
  extern __shared__ __attribute__((aligned(16))) float2 sc[];
  const int slot = fdiv((int)blockIdx.x, a.f_dn_tiles);
  const int n0 = ((int)blockIdx.x - slot * a.dn_tiles) * kTileRows;
  const int e = find_pairs<false>(a, slot, a.by_pair, list);
  if (e < 0) return;
  if constexpr (G > 0) {
    stage_scales<BF16>(sc, a.sc_dn, a.z_dn, a.I / G, [&](int r) {
      return n0 + r < a.H ? (int64_t)e * a.H + n0 + r : (int64_t)-1;
    });
    __syncthreads();
  }
  const int64_t rb = row_bytes<G, BF16>(a.I), wbytes = a.H * rb;
  const int n = n0 + (int)(threadIdx.x & 15);
  const BufRow w{expert_rsrc((const char*)a.W_dn + (int64_t)e * wbytes, wbytes),
                 n < a.H ? (uint32_t)(n * rb) : kOutOfRange};
  auto entry = [&](int j) { return j < list.count ? (int)list.pair[j] : -1; };
  auto store = [&](int j, int r, float v) {
    const int p = entry(j);
    if (p < 0 || n0 + r >= a.H) return;
    if (a.lora) v += down_delta<BF16>(a, p, e, n0 + r);
    a.z[(int64_t)p * a.H + n0 + r] = a.weights[p] * v;
  };
  for (int j0 = 0; j0 < list.count; j0 += 16 * kTiles) {
    const int nt = min(kTiles, (list.count - j0 + 15) / 16);
    if (nt == 1)
      tile_pass<G, BF16, 1>(w, a.h, a.I, a.f_one, a.I, sc, entry, j0, 1, red, store);
    else
      tile_pass<G, BF16, kTiles>(w, a.h, a.I, a.f_one, a.I, sc, entry, j0, nt, red, store);
  }
}

// y[m, n] = sum over the token's pairs of their weighted rows, four columns a thread
template <bool BF16>
__global__ void __launch_bounds__(kThreads) layer_combine_kernel(LayerArgs a) {
  const int groups = a.H / 4;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (int64_t)a.M * groups) return;
  const int m = (int)(i / groups), n = (int)(i - (int64_t)m * groups) * 4;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < a.topk; ++k) {
    const int p = m * a.topk + k;
    if (pair_expert(a, p) < 0) continue;
    const float4 v = *reinterpret_cast<const float4*>(a.z + (int64_t)p * a.H + n);
    y.x += v.x;
    y.y += v.y;
    y.z += v.z;
    y.w += v.w;
  }
  const int64_t o = (int64_t)m * a.ld_y + n;
  store_elem<BF16>(a.y, o, y.x);
  store_elem<BF16>(a.y, o + 1, y.y);
  store_elem<BF16>(a.y, o + 2, y.z);
  store_elem<BF16>(a.y, o + 3, y.w);
}

// Down with the combine for one token and NR columns: groups of KK = 16 / NR of its pairs.
template <int G, bool BF16, int NR>
__global__ void __launch_bounds__(kThreads) down_direct_kernel(LayerArgs a) {
  constexpr int KK = kTileRows / NR;
  __shared__ float red[kWaves * kTileRows];
  __shared__ float delta[kLayerMaxTopk * NR];
  extern __shared__ __attribute__((aligned(16))) float2 sc[];
  // blocks go round the XCDs: the tokens of a column group share one
  const int xcd = (int)blockIdx.x % kXcds, i = (int)blockIdx.x / kXcds;
  const int cg = fdiv(i, a.f_m);
  const int m = i - cg * a.M;
  const int n0 = (cg * kXcds + xcd) * NR;
  if (n0 >= a.H) return;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int p0 = m * a.topk;
  const int64_t rb = row_bytes<G, BF16>(a.I);
  constexpr int ESZ = BF16 ? 2 : 4;
  if (a.lora) {
    for (int t = threadIdx.x; t < a.topk * NR; t += kThreads) {
      const int p = p0 + t / NR, n = n0 + t % NR;
      const int e = pair_expert(a, p);
      delta[t] = e >= 0 && n < a.H ? a.weights[p] * down_delta<BF16>(a, p, e, n) : 0.f;
    }
  }
  const int ng = G ? a.I / (G ? G : 1) : 0;
  const int groups = (a.topk + KK - 1) / KK;
  const int steps = row_steps<G, BF16>(a.I);
  f32x4_t tot = {0.f, 0.f, 0.f, 0.f};
  for (int g = 0; g < groups; ++g) {
    // tile row r: column n0 + r % NR of pair g * KK + r / NR
    auto expert_of = [&](int kk) {
      const int k = g * KK + kk;
      return k < a.topk ? pair_expert(a, p0 + k) : -1;
    };
    if constexpr (G > 0) {
      if (g > 0) __syncthreads();
      stage_scales<BF16>(sc, a.sc_dn, a.z_dn, ng, [&](int r) {
        const int e = expert_of(r / NR), n = n0 + r % NR;
        return e >= 0 && n < a.H ? (int64_t)e * a.H + n : (int64_t)-1;
      });
      __syncthreads();
    }
    const int e = expert_of(col / NR), n = n0 + col % NR;
    const bool there = e >= 0 && n < a.H;
    const PtrRow w{(const char*)a.W_dn + (there ? ((int64_t)e * a.H + n) * rb : 0), there};
    // tile column c: the h row of pair g * KK + c (columns past the last repeat one)
    const int kx = g * KK + (col < KK ? col : 0);
    const int px = expert_of(col < KK ? col : 0) >= 0 ? p0 + kx : -1;
    // (a pair without an expert has no h: its column reads pair 0's and is not used)
    const char* const xp[1] = {(const char*)a.h + (px >= 0 ? (int64_t)px * a.I * ESZ : 0)};
    f32x4_t acc[1] = {{0.f, 0.f, 0.f, 0.f}};
    weight_part<G, BF16, 1>(w, xp, 1, a.I, steps * wv / kWaves, steps * (wv + 1) / kWaves, sc, acc);
    // the wanted lanes: column = the pair of their rows
    const int kw = g * KK + quad * 4 / NR;
    const bool mine = kw < a.topk && expert_of(quad * 4 / NR) >= 0;
    const float wt = mine ? a.weights[p0 + kw] : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) tot[j] = mine ? fmaf(wt, acc[0][j], tot[j]) : tot[j];
  }
  if (col == quad * 4 / NR) *reinterpret_cast<f32x4_t*>(red + wv * kTileRows + quad * 4) = tot;
  __syncthreads();
  if ((int)threadIdx.x < NR && n0 + (int)threadIdx.x < a.H) {
    float y = 0.f;
#pragma unroll
    for (int kk = 0; kk < KK; ++kk)
#pragma unroll
      for (int s = 0; s < kWaves; ++s) y += red[s * kTileRows + kk * NR + threadIdx.x];
    if (a.lora)
      for (int k = 0; k < a.topk; ++k) y += delta[k * NR + threadIdx.x];
    store_elem<BF16>(a.y, (int64_t)m * a.ld_y + n0 + threadIdx.x, y);
  }
}

template <int G, bool BF16, int NR>
hipError_t launch_direct(const LayerArgs& a, size_t lds, hipStream_t st) {
  const int cgs = (a.H + NR - 1) / NR;
  const int per_xcd = (cgs + kXcds - 1) / kXcds;
  hipLaunchKernelGGL((down_direct_kernel<G, BF16, NR>), dim3(per_xcd * a.M * kXcds),
                     dim3(kThreads), lds, st, a);
  return hipGetLastError();
}

template <bool BF16>
hipError_t launch_rank(const LayerArgs& a, const ShrinkPart& sp, hipStream_t st) {
  hipLaunchKernelGGL((layer_shrink_kernel<BF16>), dim3(sp.slots * sp.tiles), dim3(kThreads), 0, st,
                     a, sp);
  return hipGetLastError();
}

template <int G, bool BF16>
hipError_t layer(const LayerArgs& a, const ShrinkPart& sp1, const ShrinkPart& sp2,
                 hipStream_t st) {
  const size_t tile = kTileRows * sizeof(float2);
  const size_t lds_gu = G ? (size_t)(a.H / (G ? G : 1)) * tile : 0;
  const size_t lds_dn = G ? (size_t)(a.I / (G ? G : 1)) * tile : 0;
  hipError_t r = hipSuccess;
  if (a.lora && (r = launch_rank<BF16>(a, sp1, st)) != hipSuccess) return r;
  hipLaunchKernelGGL((gate_up_kernel<G, BF16>), dim3(a.slots * a.gu_tiles), dim3(kThreads), lds_gu,
                     st, a);
  if ((r = hipGetLastError()) != hipSuccess) return r;
  if (a.lora && (r = launch_rank<BF16>(a, sp2, st)) != hipSuccess) return r;
  if (a.direct) {
    // as many experts in a tile as the token has, up to four
    if (a.topk == 1) return launch_direct<G, BF16, 16>(a, lds_dn, st);
    if (a.topk == 2) return launch_direct<G, BF16, 8>(a, lds_dn, st);
    return launch_direct<G, BF16, 4>(a, lds_dn, st);
  }
  hipLaunchKernelGGL((down_grouped_kernel<G, BF16>), dim3(a.slots * a.dn_tiles), dim3(kThreads),
                     lds_dn, st, a);
  if ((r = hipGetLastError()) != hipSuccess) return r;
  const int64_t threads = (int64_t)a.M * (a.H / 4);
  hipLaunchKernelGGL((layer_combine_kernel<BF16>), dim3((int)((threads + kThreads - 1) / kThreads)),
                     dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

template <bool BF16>
hipError_t by_group(const LayerArgs& a, const ShrinkPart& sp1, const ShrinkPart& sp2,
                    hipStream_t st) {
  switch (a.group) {
    case 0: return layer<0, BF16>(a, sp1, sp2, st);
    case 32: return layer<32, BF16>(a, sp1, sp2, st);
    case 64: return layer<64, BF16>(a, sp1, sp2, st);
    case 128: return layer<128, BF16>(a, sp1, sp2, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_moe_layer(const LayerArgs& a, const ShrinkPart& sp1, const ShrinkPart& sp2,
                            bool bf16, hipStream_t st) {
  return bf16 ? by_group<true>(a, sp1, sp2, st) : by_group<false>(a, sp1, sp2, st);
}

}  // namespace mol
