// The down stage of a whole layer with the combine, for very few tokens without adapters:
//   y_m = round( sum_k w_mk Wd_t h_p ),  p = m * topk + k, t the pair's expert
// A work item is NR output columns of one token over all its pairs. The 16 rows of a
// matrix-core tile are NR columns of 16 / NR experts, whose h rows are the tile's columns: the diagonal
// blocks of the product are the wanted sums, every loaded weight is used, and the weighted sum
// over the pairs ends in the item, so neither the pairs' rows nor a combine launch are needed.
// An expert that several tokens share is read once by each of them; items of a column group are
// neighbours on one XCD, so most of that comes from its L2. Per token rather than per expert: for one
// token that saves a launch and a pass over the pairs' rows.
//
// Bound by the latency of its one round of loads: 7.9 us for one token (top-8, hidden 2048, inter 768
// in bf16: 25 MB, 3.2 TB/s). Twelve loads of weights and twelve of h in flight a lane are all of a
// wave's share there.
#include "skinny.h"

namespace mol {
namespace {

constexpr int kXcds = 8;

template <int G, bool BF16, int NR>
__global__ void __launch_bounds__(kThreads) down_direct_kernel(LayerArgs a) {
  constexpr int KK = kTileRows / NR;         // pairs of a tile
  constexpr int NP = BF16 ? 2 : 1;           // planes of h: columns kk and KK + kk
  constexpr int ESZ = BF16 ? 2 : 4, VE = 16 / ESZ;
  constexpr int KL = G ? kQ4Load : 4 * VE, U = G ? 2 : 12;
  __shared__ float red[kWaves * kTileRows * NP];
  const int xcd = (int)blockIdx.x % kXcds, i = (int)blockIdx.x / kXcds;
  const int cg = fdiv(i, a.f_m);
  const int m = i - cg * a.M;
  const int n0 = (cg * kXcds + xcd) * NR;
  if (n0 >= a.H) return;
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, quad = lane >> 4;
  const int p0 = m * a.topk;
  const int64_t rb = row_bytes<G, BF16>(a.I);
  const int groups = (a.topk + KK - 1) / KK;
  // waves: up to four groups of pairs at a time, the rest of the waves split the k's
  const int gw = groups >= 4 ? 4 : groups >= 2 ? 2 : 1, kw = kWaves / gw;
  const int loads = (a.I + KL - 1) / KL;
  const int part = (loads + kw - 1) / kw;
  const int l0 = wv / gw * part, l1 = min(l0 + part, loads);
  const int ng = G ? a.I / (G ? G : 1) : 0;
  auto expert_of = [&](int k) {  // of the token's pair k, or -1
    const int t = a.ids[p0 + min(k, a.topk - 1)];
    return k < a.topk && (unsigned)t < (unsigned)a.E ? t : -1;
  };
  f32x4_t tot = {0.f, 0.f, 0.f, 0.f};
  for (int g = wv % gw; g < groups; g += gw) {
    // tile row r: column n0 + r % NR of pair g * KK + r / NR
    const int e = expert_of(g * KK + col / NR), n = n0 + col % NR;
    const bool there = e >= 0 && n < a.H;
    const int64_t row = there ? (int64_t)e * a.H + n : 0;
    const char* wp = (const char*)a.W_dn + row * rb;
    // tile column c: plane c / KK of the h row of pair g * KK + c % KK (of a pair without an expert,
    // or past the last: pair 0's, unused)
    const int kx = g * KK + col % KK;
    const int px = col < NP * KK && expert_of(kx) >= 0 ? p0 + kx : 0;
    const int plane = col < NP * KK ? col / KK : 0;
    const char* xp = (const char*)a.h + ((int64_t)px * NP + plane) * a.I * ESZ;
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    for (int l = l0; l < l1; l += U) {
      uint4 w[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = (l + u) * KL + quad * (KL / 4);
        w[u] = ld16_if(wp, G ? k / 2 : (int64_t)k * ESZ, there && l + u < l1 && k < a.I);
      }
      if constexpr (G == 0) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = (l + u) * KL + quad * VE;
          x[u] = ld16_if(xp, (int64_t)k * ESZ, l + u < l1 && k < a.I);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) acc = mma16<BF16>(w[u], x[u], acc);
      } else {
        constexpr int SPG = G / 32;
        uint4 x[U][4][BF16 ? 1 : 2];
        float sc[U][4 / SPG][4], zc[U][4 / SPG][4];
        // scales of the result's rows: column n0 + (4 quad + i) % NR of pair g * KK + quad * 4 / NR
        const int es = expert_of(g * KK + quad * 4 / NR);
#pragma unroll
        for (int u = 0; u < U; ++u) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = (l + u) * KL + j * 32 + quad * 8;
            const bool ok = l + u < l1 && k < a.I;
            x[u][j][0] = ld16_if(xp, (int64_t)k * ESZ, ok);
            if constexpr (!BF16) x[u][j][1] = ld16_if(xp, (int64_t)k * ESZ + 16, ok);
          }
#pragma unroll
          for (int h = 0; h < 4 / SPG; ++h) {
            const int gi = ((l + u) * KL) / G + h;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int ns = n0 + (quad * 4 + j) % NR;
              const bool ok = es >= 0 && ns < a.H && l + u < l1 && gi < ng;
              const int64_t at = ok ? ((int64_t)es * a.H + ns) * ng + gi : 0;
              const float s = BF16 ? __uint_as_float((uint32_t)((const uint16_t*)a.sc_dn)[at] << 16)
                                   : ((const float*)a.sc_dn)[at];
              sc[u][h][j] = ok ? s : 0.f;
              zc[u][h][j] = kQ4Offset<BF16> + (a.z_dn ? (float)a.z_dn[at] : 8.f);
            }
          }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          uint32_t r[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
          transpose_quads(r);
#pragma unroll
          for (int h = 0; h < 4 / SPG; ++h) {
            f32x4_t prod = {0.f, 0.f, 0.f, 0.f}, sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int j = h * SPG; j < (h + 1) * SPG; ++j) {
              if constexpr (BF16) {
                const uint4 xo = q4_order(x[u][j][0]);
                constexpr uint32_t kOnes = 0x3f803f80u;
                prod = mma_bf16(q4_bf16(r[j]), xo, prod);
                sum = mma_bf16(make_uint4(kOnes, kOnes, kOnes, kOnes), xo, sum);
              } else {
                const uint4 &xa = x[u][j][0], &xb = x[u][j][BF16 ? 0 : 1];
                const uint32_t xe[8] = {xa.x, xa.y, xa.z, xa.w, xb.x, xb.y, xb.z, xb.w};
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                  prod = mma_f32((float)((r[j] >> (4 * q)) & 15u), __uint_as_float(xe[q]), prod);
                  sum = mma_f32(1.f, __uint_as_float(xe[q]), sum);
                }
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[j] = fmaf(sc[u][h][j], fmaf(-zc[u][h][j], sum[j], prod[j]), acc[j]);
          }
        }
      }
    }
    // the wanted lanes: column (of either plane) = the pair of their rows
    const int k = g * KK + quad * 4 / NR;
    const bool mine = expert_of(k) >= 0;
    const float wt = a.weights[p0 + min(k, a.topk - 1)];
#pragma unroll
    for (int j = 0; j < 4; ++j) tot[j] = mine ? fmaf(wt, acc[j], tot[j]) : tot[j];
  }
#pragma unroll
  for (int pl = 0; pl < NP; ++pl)
    if (col == pl * KK + quad * 4 / NR)
      *reinterpret_cast<f32x4_t*>(red + (wv * NP + pl) * kTileRows + quad * 4) = tot;
  __syncthreads();
  if (wv != 0) return;
  const bool live = lane < NR && n0 + lane < a.H;
  float y = 0.f;
  if (live) {
#pragma unroll
    for (int j = 0; j < kWaves * NP * KK; ++j) y += red[j * NR + lane];
  }
  // A column that is not finite once more, from its terms in their order: the parts above also give NaN
  // where the definition does not (an infinite h over 4-bit weights, an infinite weight beside a second
  // plane of zeros, an infinite router weight beside a wave's part of zero).
  uint64_t odd = __builtin_amdgcn_ballot_w64(live && !__builtin_isfinite(y));
  const Q4Tables q{a.sc_dn, a.z_dn, ng};
  const PlaneSrc<BF16> src{a.I};
#pragma unroll 1
  for (; odd; odd &= odd - 1) {
    const int j = __builtin_ctzll(odd);
    float sum = 0.f;
#pragma unroll 1
    for (int k = 0; k < a.topk && sum == sum; ++k) {  // (a NaN stays)
      const int e = expert_of(k);
      if (e < 0) continue;
      const __amdgpu_buffer_rsrc_t rsrc =
          expert_rsrc((const char*)a.W_dn + (int64_t)e * a.H * rb, a.H * rb);
      const RowAt at{(uint32_t)((n0 + j) * rb), (int64_t)e * a.H + n0 + j};
      const char* h = (const char*)a.h + (int64_t)(p0 + k) * NP * a.I * ESZ;
      sum = fmaf(a.weights[p0 + k], sum_of_terms<G, BF16, NP>(rsrc, at, q, src, h, a.I, lane), sum);
    }
    y = lane == j ? sum : y;
  }
  if (live) store_elem<BF16>(a.y, (int64_t)m * a.ld_y + n0 + lane, y);
}

template <int G, bool BF16, int NR>
hipError_t launch(const LayerArgs& a, hipStream_t st) {
  const int cgs = (a.H + NR - 1) / NR;
  const int per_xcd = (cgs + kXcds - 1) / kXcds;
  hipLaunchKernelGGL((down_direct_kernel<G, BF16, NR>), dim3(per_xcd * a.M * kXcds),
                     dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

// As many experts in a tile as the token has, up to four (calls of one token when that was chosen: top-1
// 13.2 us, against 13.9 with room for four; top-2 14.6 and 15.9).
template <int G, bool BF16>
hipError_t by_topk(const LayerArgs& a, hipStream_t st) {
  if (a.topk == 1) return launch<G, BF16, 16>(a, st);
  if (a.topk == 2) return launch<G, BF16, 8>(a, st);
  return launch<G, BF16, 4>(a, st);
}

template <bool BF16>
hipError_t by_group(const LayerArgs& a, hipStream_t st) {
  switch (a.group) {
    case 0: return by_topk<0, BF16>(a, st);
    case 32: return by_topk<32, BF16>(a, st);
    case 64: return by_topk<64, BF16>(a, st);
    case 128: return by_topk<128, BF16>(a, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_moe_layer_direct(const LayerArgs& a, bool bf16, hipStream_t st) {
  return bf16 ? by_group<true>(a, st) : by_group<false>(a, st);
}

}  // namespace mol
