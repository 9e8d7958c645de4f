// The balance loss of a routed batch, the experts' counts, and the gradient in the router's logits.
//
// Over the n tokens that count (not masked out, with at least one candidate logit), with c_e the
// number of their top-k slots that hold expert e and p_me the scores of token m over its candidates
// (softmax, or sigmoids over their sum):
//   P_e = sum_m p_me,    loss = alpha E / (k n^2) sum_e c_e P_e
//   d loss / d l_mj = p_mj q_mj (b_j - sum_e p_me b_e),    b_e = alpha / (k n^2) (E c_e - k n)
// with q = 1 for softmax and 1 - sigmoid(l_mj) for sigmoid. b is the derivative in p_me less alpha / n,
// which is the same for every expert and leaves the difference as it is (the p_me of a token add up
// to 1): E c_e - k n is formed in whole numbers, so a nearly balanced batch loses nothing to cancellation.
//
// A row of logits is in the registers of LPR lanes, as in the router. The forward pass gives each
// workgroup a strided set of rows; a thread adds up the scores of its own experts over its rows, the
// workgroup adds its threads in a fixed order and writes one row of partial sums (and of counts, from
// whole-number atomics in LDS). A second launch adds the rows, 8 experts a workgroup; the last
// workgroup to finish forms the loss. Few tokens take one workgroup and one launch. No sum depends
// on the order in which anything arrives: results are the same bit for bit.
//
// Kernel times (rocprofv3): 138 tokens of 160 experts in fp32, sigmoid 5.2 + 5.5 us forward and 4.7 the gradient,
// latency and launches throughout (0.2 MB); 16384 of 128 in bf16, softmax 6.8 + 7.5 and 9.1, of which their 4.2 MB read and
// 8.4 moved take 0.9 and 1.7 at a copy's rate: issue of the exponentials, the reductions over lanes and waves, and the
// second launch's wait for the first.
#include "bf16_pair.h"
#include "router_row.h"

namespace mol {
namespace {

__device__ __forceinline__ int wave_id() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// exp(x) for x <= 0 within 2^-22 of itself down to the smallest normal number (x = -87.3), within 2^-126 below it: the
// hardware's exp2 of x log2(e), corrected by what that product rounds away.
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kL = 1.44269502f, kLlo = 1.92596303e-8f, kLn2 = 0.693147182f;
  x = fmaxf(x, -200.f);
  const float t = x * kL;
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, fmaf(x, kLlo, fmaf(x, kL, -t)) * kLn2, e);
}
// exp(l - m) for l <= m; 1 at l == m, infinite m included
__device__ __forceinline__ float exp_under(float l, float m) { return l == m ? 1.f : exp_neg(l - m); }

// A row's scores before their sum is divided out, in place of its logits, and their sum over the lane; m their
// largest logit; q their 1 - sigmoid where it is asked for. Sigmoids are multiplied by exp(-min(m, 0)), which
// keeps the largest from underflowing. One exponential t = exp(-|l|) gives sigmoid(l) and 1 - sigmoid(l).
template <int VPL, bool SLOPE>
__device__ __forceinline__ float scores(float (&v)[VPL], float (&q)[VPL], float m, bool sigmoid) {
  float sum = 0.f;
  const float shift = fminf(m, 0.f);
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const float l = v[i];
    float w, s = 1.f;
    if (sigmoid) {
      const float t = exp_neg(-fabsf(l)), r = __builtin_amdgcn_rcpf(1.f + t);
      w = l > 0.f ? r : (shift == 0.f ? t : exp_under(l, shift)) * r;
      if (SLOPE) s = l > 0.f ? t * r : r;
    } else {
      w = exp_under(l, m);
    }
    v[i] = l == kMasked ? 0.f : w;
    if (SLOPE) q[i] = s;
    sum += v[i];
  }
  return sum;
}

__device__ __forceinline__ float loss_of(double cp, int n, const BalanceArgs& a) {
  if (n <= 0) return 0.f;
  return (float)((double)a.alpha * a.E * cp / ((double)a.topk * n * n));
}

// sum over the workgroup's waves, in a fixed order, in thread 0
template <int WAVES>
__device__ __forceinline__ double block_sum(double v, double* lds) {
  for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d, 64);
  if ((threadIdx.x & 63) == 0) lds[wave_id()] = v;
  __syncthreads();
  v = 0.0;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < WAVES; ++i) v += lds[i];
  }
  return v;
}

template <bool BF16, int LPR, int VPL>
__global__ void __launch_bounds__(VPL <= 16 ? 1024 : 256) balance_kernel(BalanceArgs a) {
  constexpr int ESZ = BF16 ? 2 : 4;
  constexpr int NT = VPL <= 16 ? 1024 : 256;  // balance_threads()
  constexpr int RPW = NT / LPR;         // rows at a time
  constexpr int W = LPR * VPL;          // experts of the registers, at least E
  __shared__ float part[W];
  __shared__ int hist[W + 1];           // counts, then the tokens that count
  __shared__ double red[NT / 64];
  const int tid = threadIdx.x, lane = tid & 63, lr = lane % LPR;
  for (int e = tid; e <= W; e += NT) hist[e] = 0;
  __syncthreads();
  const int e0 = lr * VPL, n = min(max(a.E - e0, 0), VPL);
  float acc[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) acc[i] = 0.f;
  // a row's logits are loaded while the one before it is at work (a row past the last: all masked)
  auto load = [&](int64_t row, float (&v)[VPL]) __attribute__((always_inline)) {
    const bool in = row < a.M && (!a.mask || a.mask[row]);
    load_row<BF16, VPL>((const char*)a.logits + (in ? row : 0) * a.ld * ESZ, e0, in ? n : 0, a.vec, v);
  };
  const int64_t step = (int64_t)gridDim.x * RPW;
  int64_t row = (int64_t)blockIdx.x * RPW + tid / LPR;
  float ahead[VPL];
  load(row, ahead);
  for (int64_t r0 = (int64_t)blockIdx.x * RPW; r0 < a.M; r0 += step, row += step) {
    float v[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = ahead[i];
    if (r0 + step < a.M) load(row + step, ahead);
    float m = kMasked;
#pragma unroll
    for (int i = 0; i < VPL; ++i) m = fmaxf(m, v[i]);
    m = group_max<LPR>(m);
    float q[VPL];
    const float sum = group_sum<LPR>(scores<VPL, false>(v, q, m, a.sigmoid));
    if (m != kMasked) {  // (the same in all lanes of a row)
      const float inv = 1.f / sum;
#pragma unroll
      for (int i = 0; i < VPL; ++i) acc[i] = fmaf(v[i], inv, acc[i]);
      for (int j = lr; j < a.topk; j += LPR) {
        const int e = a.ids[row * a.topk + j];
        if ((unsigned)e < (unsigned)a.E) atomicAdd(&hist[e], 1);
      }
      if (lr == 0) atomicAdd(&hist[W], 1);
    }
  }
  // the rows of a wave, then wave after wave
  if constexpr (LPR < 64) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      acc[i] += __shfl_xor(acc[i], 16, 64);
      acc[i] += __shfl_xor(acc[i], 32, 64);
    }
  }
  for (int w = 0; w < NT / 64; ++w) {
    if (w == wave_id() && lane < LPR) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) part[e0 + i] = w ? part[e0 + i] + acc[i] : acc[i];
    }
    __syncthreads();
  }
  const bool alone = gridDim.x == 1;
  float* sums = alone ? a.sums : a.part_sums + (int64_t)blockIdx.x * a.E;
  int* counts = alone ? a.counts : a.part_counts + (int64_t)blockIdx.x * (a.E + 1);
  double cp = 0.0;
  for (int e = tid; e < a.E; e += NT) {
    const float p = part[e];
    sums[e] = p;
    counts[e] = hist[e];
    cp += (double)hist[e] * p;
  }
  if (tid == 0) counts[a.E] = hist[W];
  if (alone) {
    cp = block_sum<NT / 64>(cp, red);
    if (tid == 0) *a.loss = loss_of(cp, hist[W], a);
  } else if (blockIdx.x == 0 && tid == 0) {
    *a.done = 0;
  }
}

// Adds the workgroups' rows: 8 experts each (one of them the count of tokens), 32 ranges of rows, whose loads
// are all in flight at once; the last workgroup to finish forms the loss. (One workgroup for all experts: 15.2
// us against 9.3 at 256 rows of 128 experts.)
__global__ void __launch_bounds__(kThreads) balance_finish_kernel(BalanceArgs a) {
  constexpr int X = 8, R = kThreads / X, PER = kBalanceGroups / R;
  __shared__ double part[R][X];
  __shared__ int count[R][X];
  __shared__ double red[kThreads / 64];
  __shared__ bool last;
  const int tid = threadIdx.x, lane = tid & 63, w = wave_id();
  const int e = blockIdx.x * X + tid % X, r = tid / X;
  float p[PER];
  int c[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int g = r + i * R;
    const bool there = g < a.groups;
    c[i] = there && e <= a.E ? a.part_counts[(int64_t)g * (a.E + 1) + e] : 0;
    p[i] = there && e < a.E ? a.part_sums[(int64_t)g * a.E + e] : 0.f;
  }
  double ps = 0.0;
  int cs = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    ps += (double)p[i];
    cs += c[i];
  }
  part[r][tid % X] = ps;
  count[r][tid % X] = cs;
  __syncthreads();
  if (tid < X && e <= a.E) {
    ps = 0.0;
    cs = 0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      ps += part[i][tid];
      cs += count[i][tid];
    }
    __hip_atomic_store(&a.counts[e], cs, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (e < a.E) __hip_atomic_store(&a.sums[e], (float)ps, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  // the workgroup that is the last to have stored its experts sees all of them
  if (w == 0) {
    __threadfence();
    if (lane == 0)
      last = __hip_atomic_fetch_add(a.done, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) ==
             (int)gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double cp = 0.0;
  for (int i = tid; i < a.E; i += kThreads)
    cp += (double)__hip_atomic_load(&a.counts[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) *
          __hip_atomic_load(&a.sums[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  cp = block_sum<kThreads / 64>(cp, red);
  if (tid == 0)
    *a.loss = loss_of(cp, __hip_atomic_load(&a.counts[a.E], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT), a);
}

// No tokens: everything is zero.
__global__ void __launch_bounds__(kThreads) balance_empty_kernel(BalanceArgs a) {
  for (int e = threadIdx.x; e <= a.E; e += kThreads) {
    a.counts[e] = 0;
    if (e < a.E) a.sums[e] = 0.f;
  }
  if (threadIdx.x == 0) *a.loss = 0.f;
}

template <bool BF16, int LPR, int VPL>
__global__ void __launch_bounds__(kThreads) balance_grad_kernel(BalanceArgs a) {
  constexpr int ESZ = BF16 ? 2 : 4;
  constexpr int RPW = kThreads / LPR;
  constexpr int VE = 16 / ESZ;
  const int tid = threadIdx.x, lr = tid % LPR;
  const int e0 = lr * VPL, n = min(max(a.E - e0, 0), VPL);
  const int tokens = a.counts[a.E];
  const float unit = tokens > 0 ? (float)((double)a.alpha / ((double)a.topk * tokens * tokens)) *
                                      (a.up ? *a.up : 1.f)
                                : 0.f;
  float b[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    b[i] = i < n ? (float)((int64_t)a.E * a.counts[e0 + i] - (int64_t)a.topk * tokens) * unit : 0.f;
  for (int64_t r0 = (int64_t)blockIdx.x * RPW; r0 < a.M; r0 += (int64_t)gridDim.x * RPW) {
    const int64_t row = r0 + tid / LPR;
    if (row >= a.M) return;  // (all of a row's lanes; no row of this workgroup comes after)
    const bool in = tokens > 0 && (!a.mask || a.mask[row]);
    float v[VPL], q[VPL];
    load_row<BF16, VPL>((const char*)a.logits + row * a.ld * ESZ, e0, in ? n : 0, a.vec, v);
    float m = kMasked;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      m = fmaxf(m, v[i]);
    }
    m = group_max<LPR>(m);
    const float sum = group_sum<LPR>(scores<VPL, true>(v, q, m, a.sigmoid));
    const float inv = m != kMasked ? 1.f / sum : 0.f;
    float mean = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      v[i] *= inv;
      mean = fmaf(v[i], b[i], mean);
    }
    mean = group_sum<LPR>(mean);
    char* dst = (char*)a.grad + row * a.ld_grad * ESZ;
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = v[i] == 0.f ? 0.f : v[i] * q[i] * (b[i] - mean);
    if (VPL % VE == 0 && a.vec_grad && n == VPL) {
#pragma unroll
      for (int i = 0; i < VPL; i += VE) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (BF16)
            u[j] = bf16_pair(v[i + 2 * j], v[i + 2 * j + 1]);
          else
            u[j] = __float_as_uint(v[i + j]);
        }
        *reinterpret_cast<uint4*>(dst + (int64_t)(e0 + i) * ESZ) = make_uint4(u[0], u[1], u[2], u[3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        if (i >= n) continue;
        if constexpr (BF16) ((uint16_t*)dst)[e0 + i] = f32_to_bf16_rne(v[i]);
        else ((float*)dst)[e0 + i] = v[i];
      }
    }
  }
}

template <bool BF16, int LPR, int VPL>
hipError_t run(const BalanceArgs& a, bool grad, hipStream_t st) {
  if (grad) {
    const int64_t rows = kThreads / LPR, want = ((int64_t)a.M + rows - 1) / rows;
    const int grid = (int)(want < kBalanceGradGroups ? want : kBalanceGradGroups);
    hipLaunchKernelGGL((balance_grad_kernel<BF16, LPR, VPL>), dim3(grid), dim3(kThreads), 0, st, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((balance_kernel<BF16, LPR, VPL>), dim3(a.groups), dim3(VPL <= 16 ? 1024 : 256), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.groups == 1) return e;
  hipLaunchKernelGGL(balance_finish_kernel, dim3(a.E / 8 + 1), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

// 16 lanes a row for many rows of up to 256 experts, else a wave, whose lanes hold up to 128 experts.
template <bool BF16>
hipError_t dispatch(const BalanceArgs& a, bool grad, hipStream_t st) {
  if (balance_narrow(a.M, a.E)) {
    if (a.E <= 64) return run<BF16, 16, 4>(a, grad, st);
    if (a.E <= 128) return run<BF16, 16, 8>(a, grad, st);
    return run<BF16, 16, 16>(a, grad, st);
  }
  if (a.E <= 128) return run<BF16, 64, 2>(a, grad, st);
  if (a.E <= 256) return run<BF16, 64, 4>(a, grad, st);
  if (a.E <= 512) return run<BF16, 64, 8>(a, grad, st);
  if (a.E <= 1024) return run<BF16, 64, 16>(a, grad, st);
  if (a.E <= 2048) return run<BF16, 64, 32>(a, grad, st);
  return run<BF16, 64, 128>(a, grad, st);
}

}  // namespace

hipError_t launch_balance(const BalanceArgs& a, bool bf16, hipStream_t st) {
  if (a.M == 0) {
    hipLaunchKernelGGL(balance_empty_kernel, dim3(1), dim3(kThreads), 0, st, a);
    return hipGetLastError();
  }
  return bf16 ? dispatch<true>(a, false, st) : dispatch<false>(a, false, st);
}

hipError_t launch_balance_grad(const BalanceArgs& a, bool bf16, hipStream_t st) {
  return bf16 ? dispatch<true>(a, true, st) : dispatch<false>(a, true, st);
}

}  // namespace mol
