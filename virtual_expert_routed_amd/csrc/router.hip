// The router: from the logits of a token to its top-k experts and their weights.
//
// Per row, with candidates C = {e : l_e is neither NaN nor -inf}, m = max over C:
//   selection   the topk largest l_e, equal ones in ascending e (logits are compared as they
//               are, so no rounding of a score can change the choice)
//   softmax     p_e = exp(l_e - m) / sum_C exp(l - m)
//   sigmoid     p_e = 1 / (1 + exp(-l_e))
//   renormalized  p_e / sum of the selected p. Softmax: exp(l_e - m) over the selected sum
//               alone. Sigmoid: each p is first multiplied by exp(-min(m, 0)), which leaves the
//               ratios as they are and keeps the largest from underflowing to zero.
//
// A row is held in the registers of LPR lanes, VPL consecutive experts a lane, and read once.
// Each lane keeps its best remaining (logit, expert); one step of the selection is a maximum
// over the row's lanes, a ballot that finds the lowest lane holding it (lower lanes hold lower
// experts: ties fall to the lowest), and a rescan of that lane's VPL registers. Slot j ends in
// lane j of the row, so topk <= LPR.
//
// A kernel's time (rocprofv3): 3.6 us for one token of 128 experts, top-8: the launch and a chain of topk
// selections of about 0.15 us. 6.5 us for 138 tokens of 160 experts (16 registers a lane, sigmoid). 7.6 us
// for 16384 tokens of 128 (5.2 MB, 0.7 TB/s), bound by issue: all of its 1024 workgroups are resident, and
// on each selection almost every wave runs the rescan of VPL registers for one lane of 16. Calls queued one
// after another take 6.6 to 7.1 us at each of these sizes: the host's time for a call.
#include "router_row.h"

namespace mol {
namespace {

template <bool BF16, int LPR, int VPL>
__global__ void __launch_bounds__(kThreads) router_kernel(RouterArgs a) {
  constexpr int ESZ = BF16 ? 2 : 4;
  static_assert(LPR == 16 || LPR == 64, "a row is a lane group of 16 or a wave");
  const int lane = threadIdx.x & 63;
  const int lr = lane % LPR;
  const int64_t row = (int64_t)blockIdx.x * (kThreads / LPR) + threadIdx.x / LPR;
  const bool live = row < a.M;
  const char* src = (const char*)a.logits + (live ? row : 0) * a.ld * ESZ;
  const int e0 = lr * VPL;
  const int n = live ? min(max(a.E - e0, 0), VPL) : 0;  // experts of this lane

  float v[VPL];
  load_row<BF16, VPL>(src, e0, n, a.vec, v);
  float bv = kMasked;  // this lane's best remaining logit, at register bi
  int bi = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if (v[i] > bv) { bv = v[i]; bi = i; }
  }
  const float m = group_max<LPR>(bv);  // -inf: no candidate in the row
  float sum = 0.f;
  if (!a.sigmoid && !a.renorm) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) sum += v[i] == kMasked ? 0.f : exp_below(v[i], m);
    sum = group_sum<LPR>(sum);
  }

  float mine = kMasked;  // slot lr: its logit and expert
  int expert = -1;
  const int base = lane - lr;
  for (int k = 0; k < a.topk; ++k) {
    const float best = group_max<LPR>(bv);
    const uint64_t holders = __builtin_amdgcn_ballot_w64(bv == best && best != kMasked);
    const uint64_t here = LPR == 64 ? holders : (holders >> base) & 0xffffull;
    const int win = here ? __builtin_ctzll(here) : 0;
    const int e = __shfl(e0 + bi, base + win, 64);
    if (lr == k && here) {
      mine = best;
      expert = e;
    }
    if (here && lr == win) {  // take it out and find this lane's next best
      float nv = kMasked;
      int ni = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (i == bi) v[i] = kMasked;
        if (v[i] > nv) { nv = v[i]; ni = i; }
      }
      bv = nv;
      bi = ni;
    }
  }

  float p = 0.f;
  if (expert >= 0) {
    if (a.sigmoid) {
      const float shift = a.renorm ? fminf(m, 0.f) : 0.f;
      p = mine > 0.f ? 1.f / (1.f + expf(-mine)) : exp_below(mine, shift) / (1.f + expf(mine));
    } else {
      p = exp_below(mine, m);
      if (!a.renorm) p /= sum;
    }
  }
  if (a.renorm) {
    const float sel = group_sum<LPR>(p);
    p = expert >= 0 ? p / sel : 0.f;
  }
  if (live && lr < a.topk) {
    const int id = expert - a.first;
    const bool local = expert >= 0 && id >= 0 && id < a.local;
    a.ids[row * a.topk + lr] = local ? id : -1;
    a.weights[row * a.topk + lr] = local ? p * a.scale : 0.f;
  }
}

template <bool BF16, int LPR, int VPL>
hipError_t launch(const RouterArgs& a, hipStream_t st) {
  const int rows = kThreads / LPR;
  const int grid = (int)(((int64_t)a.M + rows - 1) / rows);
  hipLaunchKernelGGL((router_kernel<BF16, LPR, VPL>), dim3(grid), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

// Rows of up to 256 experts and 16 slots take 16 lanes (four rows a wave, all moves inside a
// lane row); others a wave each, whose lanes hold up to 128 experts. Queued calls of 16384 tokens, 16
// lanes against a wave a row: 128 experts, top-8 7.6 and 19.4 us; 256, top-16 15.5 and 32.2.
template <bool BF16>
hipError_t dispatch(const RouterArgs& a, hipStream_t st) {
  if (router_narrow(a.E, a.topk)) {
    if (a.E <= 64) return launch<BF16, 16, 4>(a, st);
    if (a.E <= 128) return launch<BF16, 16, 8>(a, st);
    return launch<BF16, 16, 16>(a, st);
  }
  if (a.E <= 512) return launch<BF16, 64, 8>(a, st);
  if (a.E <= 1024) return launch<BF16, 64, 16>(a, st);
  return launch<BF16, 64, 128>(a, st);
}

}  // namespace

hipError_t launch_router(const RouterArgs& a, bool bf16, hipStream_t stream) {
  return bf16 ? dispatch<true>(a, stream) : dispatch<false>(a, stream);
}

}  // namespace mol
