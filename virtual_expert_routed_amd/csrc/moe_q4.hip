// The base MoE grouped GEMM of a stage over 4-bit weights with group scales:
//   out[p, n] = round( sum_k (q[t, n, k] - z[t, n, k / G]) s[t, n, k / G] x[p / row_div, k] )
// for every pair p whose base expert t is local; other rows are untouched. Routed like the
// dense grouped GEMM (the aligned blocks of one base expert each).
//
// At decode it reads half a byte of each touched weight once and little else, so a work item is
// (block, 16 output columns): 16 rows of W_t, read once for up to 64 pairs of the block.
#include "skinny.h"

namespace mol {
namespace {

template <int G, bool BF16>
__global__ void __launch_bounds__(kThreads) q4_gemm_kernel(Q4GemmArgs a) {
  __shared__ float red[kWaves * kTiles * 256];
  extern __shared__ __attribute__((aligned(16))) float2 sc[];
  const int blk = fdiv((int)blockIdx.x, a.f_tiles);
  const int n0 = ((int)blockIdx.x - blk * a.tiles) * kTileRows;
  const int npp = *a.npp;
  const int er = a.expert_ids[blk];
  const int nb = npp < 0 ? 0 : fdiv(npp, a.f_bm);
  if (blk >= nb || (unsigned)er >= (unsigned)a.E) return;
  const int e = __builtin_amdgcn_readfirstlane(er);
  const int32_t* sorted = a.sorted + (int64_t)blk * a.BM;
  auto entry = [&](int j) {  // the pair of entry j of the block, or -1
    const int p = j < a.BM ? sorted[j] : a.numel;
    return real_pair(p, a.numel) ? p : -1;
  };
  if (entry(0) < 0) return;
  const int ng = a.K / G;
  stage_scales<BF16>(sc, a.scales, a.zeros, ng, [&](int r) {
    return n0 + r < a.N ? (int64_t)e * a.N + n0 + r : (int64_t)-1;
  });
  __syncthreads();
  const int64_t wbytes = (int64_t)a.N * a.K / 2;
  const int n = n0 + (int)(threadIdx.x & 15);
  const BufRow w{expert_rsrc((const char*)a.W + (int64_t)e * wbytes, wbytes),
                 n < a.N ? (uint32_t)n * (uint32_t)(a.K / 2) : kOutOfRange};
  for (int j0 = 0; j0 < a.BM; j0 += 16 * kTiles) {
    int nt = 0;  // tiles that hold a real pair (the real pairs are a prefix of the block)
#pragma unroll
    for (int t = 0; t < kTiles; ++t) nt += entry(j0 + 16 * t) >= 0 ? 1 : 0;
    if (nt == 0) return;
    auto store = [&](int j, int r, float v) {
      const int p = entry(j);
      if (p >= 0 && n0 + r < a.N) store_elem<BF16>(a.out, (int64_t)p * a.ld_out + n0 + r, v);
    };
    if (nt == 1)
      tile_pass<G, BF16, 1>(w, a.x, a.ld_x, a.f_rd, a.K, sc, entry, j0, 1, red, store);
    else
      tile_pass<G, BF16, kTiles>(w, a.x, a.ld_x, a.f_rd, a.K, sc, entry, j0, nt, red, store);
  }
}

template <int G, bool BF16>
hipError_t launch(const Q4GemmArgs& a, hipStream_t st) {
  const size_t lds = (size_t)(a.K / G) * kTileRows * sizeof(float2);
  hipLaunchKernelGGL((q4_gemm_kernel<G, BF16>), dim3(a.max_blocks * a.tiles), dim3(kThreads), lds,
                     st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_q4_gemm(const Q4GemmArgs& a, bool bf16, hipStream_t st) {
  switch (a.group) {
    case 32: return bf16 ? launch<32, true>(a, st) : launch<32, false>(a, st);
    case 64: return bf16 ? launch<64, true>(a, st) : launch<64, false>(a, st);
    case 128: return bf16 ? launch<128, true>(a, st) : launch<128, false>(a, st);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace mol
