// The balance loss of a router, its experts' counts, and the gradient for the
// router's logits (gfx950).
//
//   p_t = softmax(logits_t);  c_e = choices of expert e;  f_e = E c_e / sum c
//   loss = w sum_e f_e P_e,  P_e = mean over the n tokens with a choice of p_te
//   dloss/dlogits_tj = (w / n) p_tj (f_j - sum_e f_e p_te)
//
// Counts enter f as numbers: no gradient passes through them.  Three launches:
// partial sums of p and of the choices per workgroup; their join, in a fixed
// order; and the gradient, which forms the softmax again rather than store it:
// 65536 x 64 fp32 with 6 choices 9.6 + 8.0 + 7.5 us, where the logits and the
// choices, 20 MB, come from memory at 2.1 TB/s and then from the caches, and the
// join is the latency of one workgroup over 512 partial sums.
#include <algorithm>

#include "balance_internal.h"
#include "mo_internal.h"
#include "row_vec.h"

namespace mo {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

struct Partials {
  float* p;                     // [groups][experts]
  int* count;                   // [groups][experts]
  int* tokens;                  // [groups][2]: tokens with a choice, choices past the last expert
  float* f;                     // [experts]: f_e, then the factor w / n of the gradient (NaN with a wrong choice)
  int groups;
};

// L lanes share a row, C columns each (column lane + L c).
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = 1; o < L; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = 1; o < L; o <<= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

template <typename T, int L, int C>
__device__ __forceinline__ void load_row(const T* z, int experts, int l, float (&p)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) p[c] = l + L * c < experts ? to_f(z[l + L * c]) : -INFINITY;
}

// The softmax of a row, in place; columns past the last are 0.
template <int L, int C>
__device__ __forceinline__ void softmax_row(int experts, int l, float (&p)[C]) {
  float m = -INFINITY;
#pragma unroll
  for (int c = 0; c < C; ++c) m = fmaxf(m, p[c]);
  m = lanes_max<L>(m);
  float s = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    p[c] = l + L * c < experts ? __builtin_amdgcn_exp2f((p[c] - m) * kLog2e) : 0.0f;
    s += p[c];
  }
  const float inv = 1.0f / lanes_sum<L>(s);
#pragma unroll
  for (int c = 0; c < C; ++c) p[c] *= inv;
}

// Whether a token has a choice.
template <int L>
__device__ __forceinline__ bool has_choice(const int64_t* index, int top, int l) {
  int any = 0;
  for (int k = l; k < top; k += L) any |= index[k] >= 0;
#pragma unroll
  for (int o = 1; o < L; o <<= 1) any |= __shfl_xor(any, o, 64);
  return any != 0;
}

template <typename T, int L, int C>
__global__ void __launch_bounds__(256) balance_sums_kernel(const BalanceArgs a, const Partials w) {
  constexpr int kRows = 256 / L;                // rows at a time
  __shared__ int count[kMaxExperts];
  __shared__ float part[kRows > 1 ? kRows * L * C : 1];
  __shared__ int seen[2];
  for (int e = threadIdx.x; e < a.experts; e += 256) count[e] = 0;
  if (threadIdx.x < 2) seen[threadIdx.x] = 0;
  __syncthreads();
  const int l = threadIdx.x % L, r = threadIdx.x / L;
  float sum[C] = {};
  int live = 0, wrong = 0;
  // kDeep rows at a time, whose loads are all in flight before the first is used
  constexpr int kDeep = C <= 4 ? 4 : C <= 8 ? 2 : 1;
  const int64_t step = static_cast<int64_t>(w.groups) * kRows;
  for (int64_t t0 = static_cast<int64_t>(blockIdx.x) * kRows + r; t0 < a.tokens; t0 += step * kDeep) {
    float p[kDeep][C];
    int64_t first[kDeep];
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const int64_t t = t0 + d * step;
      first[d] = -1;
      if (t < a.tokens) {
        load_row<T, L, C>(static_cast<const T*>(a.logits) + t * a.ld, a.experts, l, p[d]);
        if (l < a.top) first[d] = a.index[t * a.top + l];
      }
    }
#pragma unroll
    for (int d = 0; d < kDeep; ++d) {
      const int64_t t = t0 + d * step;
      if (t >= a.tokens) continue;                          // the same for the row's lanes
      int any = 0;
      int64_t e = first[d];
      for (int k = l; k < a.top; k += L) {
        if (k >= L) e = a.index[t * a.top + k];
        any |= e >= 0;
        if (e >= a.experts) wrong = 1;
        else if (e >= 0) atomicAdd(&count[e], 1);
      }
#pragma unroll
      for (int o = 1; o < L; o <<= 1) any |= __shfl_xor(any, o, 64);
      if (!any) continue;
      if (l == 0) ++live;
      softmax_row<L, C>(a.experts, l, p[d]);
#pragma unroll
      for (int c = 0; c < C; ++c) sum[c] += p[d][c];
    }
  }
  if (live) atomicAdd(&seen[0], live);
  if (wrong) seen[1] = 1;
#pragma unroll
  for (int c = 0; c < C; ++c) part[(r * C + c) * L + l] = sum[c];
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += 256) {
    float v = 0.0f;
    for (int i = 0; i < kRows; ++i) v += part[i * C * L + e];
    w.p[static_cast<int64_t>(blockIdx.x) * a.experts + e] = v;
    w.count[static_cast<int64_t>(blockIdx.x) * a.experts + e] = count[e];
  }
  if (threadIdx.x < 2) w.tokens[blockIdx.x * 2 + threadIdx.x] = seen[threadIdx.x];
}

__device__ __forceinline__ int64_t block_sum(int64_t v, int64_t* red) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  int64_t t = 0;
  for (int i = 0; i < 16; ++i) t += red[i];
  return t;
}

// One workgroup: totals over the groups, f, the loss.  A wave takes 64 experts
// and every 16th group; the waves' sums are added in their order.
__global__ void __launch_bounds__(1024) balance_join_kernel(const BalanceArgs a, const Partials w) {
  __shared__ float psum[16][64];
  __shared__ int csum[16][64];
  __shared__ float mean[kMaxExperts];          // sum of p, then its share of the loss
  __shared__ int64_t red[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t live = 0, wrong = 0, choices = 0;
  for (int g = threadIdx.x; g < w.groups; g += 1024) {
    live += w.tokens[g * 2];
    wrong += w.tokens[g * 2 + 1];
  }
  live = block_sum(live, red);
  wrong = block_sum(wrong, red);
  for (int e0 = 0; e0 < a.experts; e0 += 64) {
    const int e = e0 + lane;
    float p = 0.0f;
    int c = 0;
    if (e < a.experts) {
#pragma unroll 8
      for (int g = wave; g < w.groups; g += 16) {
        p += w.p[static_cast<int64_t>(g) * a.experts + e];
        c += w.count[static_cast<int64_t>(g) * a.experts + e];
      }
    }
    psum[wave][lane] = p;
    csum[wave][lane] = c;
    __syncthreads();
    if (wave == 0 && e < a.experts) {
      float v = 0.0f;
      int64_t n = 0;
      for (int i = 0; i < 16; ++i) {
        v += psum[i][lane];
        n += csum[i][lane];
      }
      mean[e] = v;
      a.counts[e] = n;
      choices += n;
    }
    __syncthreads();
  }
  choices = block_sum(choices, red);
  float loss = 0.0f;
  if (wave == 0)
    for (int e = lane; e < a.experts; e += 64) {              // the lane's own counts and sums
      const float f = choices ? static_cast<float>(a.counts[e]) * static_cast<float>(a.experts) / static_cast<float>(choices) : 0.0f;
      w.f[e] = f;
      loss += f * mean[e];
    }
  for (int o = 32; o > 0; o >>= 1) loss += __shfl_xor(loss, o, 64);
  if (threadIdx.x) return;
  const float n = live ? static_cast<float>(live) : 1.0f;
  *a.loss = wrong ? NAN : a.weight * (loss / n);
  w.f[a.experts] = wrong ? NAN : a.weight * (a.grad_loss ? *a.grad_loss : 1.0f) / n;
}

// The gradient of token t.
template <typename T, int L, int C>
__device__ __forceinline__ void grad_row(const BalanceArgs& a, int64_t t, int l, const float (&f)[C], float factor) {
  T* out = static_cast<T*>(a.grad) + t * a.ld_grad;
  float p[C];
  load_row<T, L, C>(static_cast<const T*>(a.logits) + t * a.ld, a.experts, l, p);
  const bool live = has_choice<L>(a.index + t * a.top, a.top, l);
  softmax_row<L, C>(a.experts, l, p);
  float mean = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) mean += p[c] * f[c];
  mean = lanes_sum<L>(mean);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int e = l + L * c;
    if (e >= a.experts) continue;
    float v = live ? factor * (p[c] * (f[c] - mean)) : 0.0f;
    if (a.accumulate) v += to_f(out[e]);
    out[e] = static_cast<T>(v);
  }
}

// Few tokens: everything in one launch of one workgroup, whose sums and counts
// stay in LDS.
template <typename T, int L, int C>
__global__ void __launch_bounds__(1024) balance_small_kernel(const BalanceArgs a) {
  constexpr int kRows = 1024 / L, kMost = L * C;
  __shared__ int count[kMost];
  __shared__ float part[kRows * kMost], f[kMost], lossf[kMost];
  __shared__ int seen[2], choices;
  const int l = threadIdx.x % L, r = threadIdx.x / L;
  for (int e = threadIdx.x; e < kMost; e += 1024) count[e] = 0;
  if (threadIdx.x < 2) seen[threadIdx.x] = 0;
  if (threadIdx.x == 2) choices = 0;
  __syncthreads();
  float sum[C] = {};
  for (int64_t t = r; t < a.tokens; t += kRows) {
    int any = 0;
    float p[C];
    load_row<T, L, C>(static_cast<const T*>(a.logits) + t * a.ld, a.experts, l, p);
    for (int k = l; k < a.top; k += L) {
      const int64_t e = a.index[t * a.top + k];
      any |= e >= 0;
      if (e >= a.experts) seen[1] = 1;
      else if (e >= 0) atomicAdd(&count[e], 1);
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) any |= __shfl_xor(any, o, 64);
    if (!any) continue;
    if (l == 0) atomicAdd(&seen[0], 1);
    softmax_row<L, C>(a.experts, l, p);
#pragma unroll
    for (int c = 0; c < C; ++c) sum[c] += p[c];
  }
#pragma unroll
  for (int c = 0; c < C; ++c) part[(r * C + c) * L + l] = sum[c];
  __syncthreads();
  for (int e = threadIdx.x; e < kMost; e += 1024) {
    if (e < a.experts) {
      a.counts[e] = count[e];
      if (count[e]) atomicAdd(&choices, count[e]);
    }
    float v = 0.0f;
    for (int i = 0; i < kRows; ++i) v += part[i * kMost + e];
    lossf[e] = v;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < kMost; e += 1024) {
    f[e] = e < a.experts && choices ? static_cast<float>(count[e]) * static_cast<float>(a.experts) / static_cast<float>(choices) : 0.0f;
    lossf[e] *= f[e];
  }
  __syncthreads();
  const float n = seen[0] ? static_cast<float>(seen[0]) : 1.0f;
  if (threadIdx.x < 64) {
    float loss = 0.0f;
    for (int e = threadIdx.x; e < kMost; e += 64) loss += e < a.experts ? lossf[e] : 0.0f;
    loss = lanes_sum<64>(loss);
    if (threadIdx.x == 0) *a.loss = seen[1] ? NAN : a.weight * (loss / n);
  }
  if (!a.grad) return;
  const float factor = seen[1] ? NAN : a.weight * (a.grad_loss ? *a.grad_loss : 1.0f) / n;
  float fr[C];
#pragma unroll
  for (int c = 0; c < C; ++c) fr[c] = f[l + L * c];
  for (int64_t t = r; t < a.tokens; t += kRows) grad_row<T, L, C>(a, t, l, fr, factor);
}

template <typename T, int L, int C>
__global__ void __launch_bounds__(256) balance_grad_kernel(const BalanceArgs a, const Partials w) {
  constexpr int kRows = 256 / L;
  const int l = threadIdx.x % L, r = threadIdx.x / L;
  float f[C];
#pragma unroll
  for (int c = 0; c < C; ++c) f[c] = l + L * c < a.experts ? w.f[l + L * c] : 0.0f;
  const float factor = w.f[a.experts];
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRows + r; t < a.tokens; t += static_cast<int64_t>(gridDim.x) * kRows)
    grad_row<T, L, C>(a, t, l, f, factor);
}

// Workgroups of the first launch: what they leave is read by one workgroup.
int groups_of(int64_t tokens) { return static_cast<int>(std::min<int64_t>(512, (tokens + 63) / 64)); }

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

// Lanes to a row, and whether one workgroup takes all rows, in up to four rounds
// (37 x 64 in bf16: 19 us in three launches, 14 in one, both with the call's 13).
int lanes_of(int experts) { return experts <= 64 ? 16 : 64; }
bool small(int64_t tokens, int experts) { return experts <= 512 && tokens * lanes_of(experts) <= 4 * 1024; }

template <typename T, int L, int C>
hipError_t run(const BalanceArgs& a, const Partials& w, hipStream_t s) {
  if constexpr (C <= 8) {
    if (small(a.tokens, a.experts)) {
      balance_small_kernel<T, L, C><<<1, 1024, 0, s>>>(a);
      return hipGetLastError();
    }
  }
  if (w.groups) balance_sums_kernel<T, L, C><<<w.groups, 256, 0, s>>>(a, w);
  balance_join_kernel<<<1, 1024, 0, s>>>(a, w);
  if (a.grad && a.tokens) {
    const int64_t g = std::min<int64_t>(4096, (a.tokens + 256 / L - 1) / (256 / L));
    balance_grad_kernel<T, L, C><<<static_cast<uint32_t>(g), 256, 0, s>>>(a, w);
  }
  return hipGetLastError();
}

template <typename T>
hipError_t run_t(const BalanceArgs& a, const Partials& w, hipStream_t s) {
  if (a.experts <= 16) return run<T, 16, 1>(a, w, s);
  if (a.experts <= 32) return run<T, 16, 2>(a, w, s);
  if (a.experts <= 64) return run<T, 16, 4>(a, w, s);
  if (a.experts <= 128) return run<T, 64, 2>(a, w, s);
  if (a.experts <= 256) return run<T, 64, 4>(a, w, s);
  if (a.experts <= 512) return run<T, 64, 8>(a, w, s);
  if (a.experts <= 1024) return run<T, 64, 16>(a, w, s);
  return run<T, 64, 64>(a, w, s);
}

}  // namespace

size_t balance_workspace(int64_t tokens, int experts) {
  if (small(tokens, experts)) return 0;
  const size_t g = static_cast<size_t>(groups_of(tokens)), e = static_cast<size_t>(experts);
  return 2 * align256(g * e * 4) + align256(g * 8) + align256((e + 1) * 4);
}

hipError_t launch_balance(int dt, const BalanceArgs& a, void* ws, hipStream_t s) {
  Partials w{};
  w.groups = groups_of(a.tokens);
  uint8_t* base = static_cast<uint8_t*>(ws);
  const size_t part = align256(static_cast<size_t>(w.groups) * a.experts * 4);
  w.p = reinterpret_cast<float*>(base);
  w.count = reinterpret_cast<int*>(base + part);
  w.tokens = reinterpret_cast<int*>(base + 2 * part);
  w.f = reinterpret_cast<float*>(base + 2 * part + align256(static_cast<size_t>(w.groups) * 8));
  return dt == F32 ? run_t<float>(a, w, s) : run_t<__bf16>(a, w, s);
}

}  // namespace mo
