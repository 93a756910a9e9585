// Token log probabilities, entropy and top alternatives, and the
// distillation loss with its gradient (gfx950).  Definitions are those of
// include/muon.h.
#include "mo_internal.h"
#include "token_internal.h"

namespace mo {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__bf16>(__bf16 v) { return static_cast<float>(v); }

// exp(d) for d <= 0 (or NaN), d given in units of log 2.
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Integer that orders as the value does: NaN above everything, -0 = +0.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

constexpr int kThreads = 256;

// Reductions over the workgroup in a fixed order; every thread gets the
// result.  `red` holds 4 slots and is free again after the call.
template <typename V, typename F>
__device__ __forceinline__ V block_reduce(V v, V* red, F f) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = f(v, __shfl_xor(v, o, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = f(f(red[0], red[1]), f(red[2], red[3]));
  __syncthreads();
  return v;
}

struct Sum { template <typename V> __device__ V operator()(V a, V b) const { return a + b; } };
struct Max { template <typename V> __device__ V operator()(V a, V b) const { return a > b ? a : b; } };

}  // namespace

// One workgroup per row: maximum, then the sums, then one pass per
// alternative.
template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const LogprobArgs a) {
  __shared__ float redf[4];
  __shared__ unsigned long long redu[4];
  const int64_t r = blockIdx.x;
  const T* z = static_cast<const T*>(a.logits) + r * a.ld;
  float m = -INFINITY;
  for (int j = threadIdx.x; j < a.vocab; j += kThreads) m = fmaxf(m, to_f(z[j]));
  m = block_reduce(m, redf, Max());
  float s = 0.0f, t = 0.0f;
  for (int j = threadIdx.x; j < a.vocab; j += kThreads) {
    const float d = (to_f(z[j]) - m) * a.inv_tau;
    const float e = exp2_fast(d * kLog2e);
    s += e;
    t += e > 0.0f ? e * -d : 0.0f;
  }
  s = block_reduce(s, redf, Sum());
  t = block_reduce(t, redf, Sum());
  const float log_s = logf(s);
  if (threadIdx.x == 0) {
    if (a.tokens) {
      const int64_t tok = a.tokens[r];
      a.logprob[r] = tok < 0 ? 0.0f : tok < a.vocab ? (to_f(z[tok]) - m) * a.inv_tau - log_s : NAN;
    }
    if (a.entropy) a.entropy[r] = s != s ? NAN : log_s + t / s;
  }
  unsigned long long last = ~0ull;   // every composite key is below it
  for (int i = 0; i < a.top; ++i) {
    unsigned long long best = 0;
    for (int j = threadIdx.x; j < a.vocab; j += kThreads) {
      const unsigned long long k =
          (static_cast<unsigned long long>(order_key(to_f(z[j]))) << 32) | (0xfffffffeu - static_cast<uint32_t>(j));
      if (k < last && k > best) best = k;
    }
    best = block_reduce(best, redu, Max());
    last = best;
    if (threadIdx.x == 0) {
      const uint32_t j = 0xfffffffeu - static_cast<uint32_t>(best);
      a.top_index[r * a.top + i] = j;
      a.top_logprob[r * a.top + i] = (to_f(z[j]) - m) * a.inv_tau - log_s;
    }
  }
}

size_t logprobs_workspace(int64_t, int64_t, int) { return 0; }

hipError_t launch_logprobs(int dt, const LogprobArgs& a, void*, hipStream_t s) {
  if (dt == F32) logprobs_kernel<float><<<a.rows, kThreads, 0, s>>>(a);
  else logprobs_kernel<__bf16><<<a.rows, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

// One workgroup per row: the teacher's softmax over its slots, the student's
// maximum and sum, the loss, and the gradient (the student's softmax
// everywhere, then the teacher's columns again with their probability taken
// off).
template <typename T>
__global__ void __launch_bounds__(kThreads) distill_kernel(const DistillArgs a) {
  __shared__ float redf[4];
  __shared__ float prob[kMaxTop];
  __shared__ int col[kMaxTop];       // -1: absent or of no weight
  const int64_t r = blockIdx.x;
  const T* z = static_cast<const T*>(a.logits) + r * a.ld;
  const int tid = threadIdx.x;
  int64_t idx = -1;
  float t = -INFINITY;
  if (tid < a.top) {
    idx = a.top_index[r * a.top + tid];
    if (idx >= 0) t = a.top_logit[r * a.top + tid];
  }
  const float bad = (idx >= a.vocab || t != t || t == INFINITY) ? NAN : 0.0f;
  const float tm = block_reduce(t, redf, Max());
  const float nan_row = block_reduce(bad, redf, Sum());
  const bool skip = tm == -INFINITY && nan_row == 0.0f;
  const float g = a.grad_loss ? a.grad_loss[r] : 1.0f;
  T* grad = a.grad ? static_cast<T*>(a.grad) + r * a.ld_grad : nullptr;
  if (grad && (skip || g == 0.0f)) {
    for (int j = tid; j < a.vocab; j += kThreads) grad[j] = static_cast<T>(0.0f);
    grad = nullptr;
  }
  if (skip) {
    if (a.loss && tid == 0) a.loss[r] = 0.0f;
    return;
  }
  const float td = (t - tm) * a.inv_tau;
  float p = exp2_fast(td * kLog2e);
  const float ts = block_reduce(tid < a.top ? p : 0.0f, redf, Sum());
  p = tid < a.top ? p / ts : 0.0f;
  float m = -INFINITY;
  for (int j = tid; j < a.vocab; j += kThreads) m = fmaxf(m, to_f(z[j]));
  m = block_reduce(m, redf, Max());
  float s = 0.0f;
  for (int j = tid; j < a.vocab; j += kThreads) s += exp2_fast((to_f(z[j]) - m) * a.inv_tau * kLog2e);
  s = block_reduce(s, redf, Sum()) + nan_row;
  if (a.loss) {
    const float zk = p > 0.0f && idx < a.vocab ? (to_f(z[idx]) - m) * a.inv_tau : 0.0f;
    const float term = p > 0.0f ? p * ((td - logf(ts)) - (zk - logf(s))) : 0.0f;
    const float l = block_reduce(term, redf, Sum());
    if (tid == 0) a.loss[r] = a.tau * a.tau * l + (s != s ? NAN : 0.0f);
  }
  if (!grad) return;
  if (tid < a.top) {
    prob[tid] = p;
    col[tid] = p > 0.0f && idx < a.vocab ? static_cast<int>(idx) : -1;
  }
  const float c = g * a.tau, qs = 1.0f / s;
  for (int j = tid; j < a.vocab; j += kThreads)
    grad[j] = static_cast<T>(c * (exp2_fast((to_f(z[j]) - m) * a.inv_tau * kLog2e) * qs));
  __builtin_amdgcn_s_waitcnt(0x0f70);   // the stores above before the teacher's columns
  __syncthreads();
  if (tid < a.top && col[tid] >= 0) {
    const int j = col[tid];
    float sum = 0.0f;
    bool first = true;
    for (int k = 0; k < a.top; ++k)
      if (col[k] == j) {
        if (k < tid) first = false;
        sum += prob[k];
      }
    if (first)
      grad[j] = static_cast<T>(c * (exp2_fast((to_f(z[j]) - m) * a.inv_tau * kLog2e) * qs - sum));
  }
}

size_t distill_workspace(int64_t, int64_t, int) { return 0; }

hipError_t launch_distill(int dt, const DistillArgs& a, void*, hipStream_t s) {
  if (dt == F32) distill_kernel<float><<<a.rows, kThreads, 0, s>>>(a);
  else distill_kernel<__bf16><<<a.rows, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace mo
