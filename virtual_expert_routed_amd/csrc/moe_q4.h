// The base MoE grouped GEMM of a stage over 4-bit weights with group scales:
//   out[p, n] = round( sum_k (q[t, n, k] - z[t, n, k / G]) s[t, n, k / G] x[p / row_div, k] )
// for every pair p whose base expert t is local; other rows are untouched. Routed like the
// dense grouped GEMM (the aligned blocks of one base expert each).
//
// At decode it reads half a byte of each touched weight once and little else, so a work item is
// (block, 64 to 256 output columns): rows of W_t, read once for up to 64 pairs of the block (32 in
// fp32, whose products of four k's a step take twice the registers). Where 64 make too few items to
// fill the chip (split_k), an item is 16 rows whose k's the four waves split.
//
// What bounds it: an item's own latency (routing reads, then x and the first weights, then LDS), of
// which four workgroups a CU (groups of 128; three otherwise) hide a part, and the unpacking of q.
// 128 experts, top-8, N 1536, K 2048, groups of 128, queued calls: 1 token 9.7 us (13 MB, 1.3 TB/s; the
// kernel 8.8), 23 tokens 38 (161 MB, 4.2), 128 tokens of popular experts 57 (196 MB, 3.4). Groups of 64
// and 32 at 23 tokens: 44 and 70 us. Their dwords move between the quads, with two or four scales a
// load, and the kernels for groups of 32 run out of registers: all but the fp32 one over items of 64
// rows keep 13 to 69 vector registers in scratch.
#pragma once

#include "skinny.h"

namespace mol {
namespace {

template <int G, bool BF16, int KS>
__global__ void __launch_bounds__(kThreads, G == 128 ? 4 : 3) q4_gemm_kernel(Q4GemmArgs a) {
  constexpr int kCols = kPassCols<G, BF16, 1, KS>;
  __shared__ int pair[kCols];
  __shared__ __attribute__((aligned(16))) char lds[StreamLds<G, BF16>::kBytes];
  const int blk = fdiv((int)blockIdx.x, a.f_items);
  const int n0 = ((int)blockIdx.x - blk * a.items) * (KS > 1 ? kTileRows : kItemRows * a.tiles);
  const int npp = *a.npp;
  const int er = a.expert_ids[blk];
  const int32_t* sorted = a.sorted + (int64_t)blk * a.BM;
  // the first entries with the routing reads (their index stays inside the block)
  int p = threadIdx.x < kCols && (int)threadIdx.x < a.BM ? sorted[threadIdx.x] : a.numel;
  const int nb = npp < 0 ? 0 : fdiv(npp, a.f_bm);
  if (blk >= nb || (unsigned)er >= (unsigned)a.E) return;
  const int e = __builtin_amdgcn_readfirstlane(er);
  const int64_t rb = a.K / 2, wbytes = (int64_t)a.N * rb;
  const __amdgpu_buffer_rsrc_t rsrc = expert_rsrc((const char*)a.W + (int64_t)e * wbytes, wbytes);
  const int lane = threadIdx.x & 63, quad = lane >> 4;
  const Q4Tables q{a.scales, a.zeros, a.K / G};
  const RowSrc src{(const char*)a.x, a.ld_x * (BF16 ? 2 : 4), pair, a.f_rd};
  for (int j0 = 0; j0 < a.BM; j0 += kCols) {
    if (j0 > 0) {
      const int j = j0 + (int)threadIdx.x;
      p = threadIdx.x < kCols && j < a.BM ? sorted[j] : a.numel;
      __syncthreads();  // pair is no longer read
    }
    if (threadIdx.x < kCols) pair[threadIdx.x] = p;
    __syncthreads();
    // the real pairs are a prefix of the block
    const int j = threadIdx.x & 63;
    const int ncol = __popcll(
        __builtin_amdgcn_ballot_w64(j < kCols && real_pair(pair[j < kCols ? j : 0], a.numel)));
    if (ncol == 0) return;
#pragma unroll 1
    for (int t = 0; t < (KS > 1 ? 1 : a.tiles); ++t) {
      const int r0 = wave_row0<KS>(n0 + t * kItemRows);
      auto row_at = [&](int i) {
        const int n = r0 + i;
        return n < a.N ? RowAt{(uint32_t)(n * rb), (int64_t)e * a.N + n} : RowAt{kOutOfRange, -1};
      };
      stream_cols<G, BF16, 1, KS>(
          lds, rsrc, row_at(lane & 15), row_at, q, src, ncol, a.K, t > 0,
          [&](int c, const f32x4_t& acc) {
            if (c >= ncol) return;
            const int m = r0 + quad * 4;
            const int64_t at = (int64_t)pair[c] * a.ld_out + m;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (m + i < a.N) store_elem<BF16>(a.out, at + i, acc[i]);
          });
    }
    if (ncol < kCols) return;
  }
}

template <int G, bool BF16>
hipError_t launch_gemm(const Q4GemmArgs& a, hipStream_t st) {
  const dim3 grid(a.max_blocks * a.items);
  if (a.split_k)
    hipLaunchKernelGGL((q4_gemm_kernel<G, BF16, kWaves>), grid, dim3(kThreads), 0, st, a);
  else
    hipLaunchKernelGGL((q4_gemm_kernel<G, BF16, 1>), grid, dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace

// The product over weights of group G: one translation unit each.
template <int G>
hipError_t launch_q4_group(const Q4GemmArgs& a, bool bf16, hipStream_t st) {
  return bf16 ? launch_gemm<G, true>(a, st) : launch_gemm<G, false>(a, st);
}

}  // namespace mol
