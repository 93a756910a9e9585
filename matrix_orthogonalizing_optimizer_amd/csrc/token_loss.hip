// Token log probabilities, entropy and top alternatives, and the
// distillation loss with its gradient (gfx950).  Definitions are those of
// include/muon.h.
//
// Both read a row of logits once into registers: a workgroup's registers
// hold up to 320 KiB, so the maximum, the sum against it, the alternatives
// and the gradient all come from one reading.  Longer rows (over 64 KiB for
// the log probabilities, over 320 KiB for the loss) are cut into pieces of one
// workgroup each, whose statistics a second launch joins; shorter ones are one
// workgroup each, however few they are.
//
// With m the largest logit of the row (or piece) and x_j = logit_j - m, the
// sums are S = sum exp(x_j / tau) and U = sum exp(x_j / tau) x_j, and
//   log p_j = x_j / tau - ln S,  entropy = ln S - U / (S tau).
// The difference comes before the scaling: it is exact for logits that are
// near each other, and logits of the type's lowest value do not overflow.
// All sums are fp32, in a fixed order.
//
// HBM bound.  Log probabilities, bf16: 4096 x 32000 43 us for the statistics
// (6.1 TB/s), 67 with 32 alternatives and 75 with 64 (the search overlaps other
// rows' loads in part); 501 x 129283 with 8 alternatives 35 + 5 us for the join.
// Distillation, loss and gradient, bf16: 8192 x 32000 (1.05 GB) 233 us, 4.5
// TB/s; rows of 128 to 320 KiB, where one workgroup fills a CU, 2048 x 128256
// 306 us and 1024 x 151936 189 us, 3.3 to 3.4 TB/s.  With few rows the launches
// bound both: 3 x 32000 fp32 with 20 alternatives 7 + 5 us.
#include <type_traits>

#include "mo_internal.h"
#include "token_internal.h"

namespace mo {

namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f, kLowest = -3.0e38f;
typedef unsigned long long u64;

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float log2_(float x) { return __builtin_amdgcn_logf(x); }

// Integer that orders as the value does: NaN above everything, -0 = +0; and
// back.
__device__ __forceinline__ uint32_t order_key(float v) {
  if (v != v) return 0xffffffffu;
  const uint32_t b = __float_as_uint(v + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}
// Largest first, then the lowest column: unique within a row, never 0.
__device__ __forceinline__ u64 top_key(float v, int col) {
  return (static_cast<u64>(order_key(v)) << 32) | (0xfffffffeu - static_cast<uint32_t>(col));
}
__device__ __forceinline__ int key_col(u64 k) { return static_cast<int>(0xfffffffeu - static_cast<uint32_t>(k)); }

// Waves per SIMD that the registers leave room for: the row's own (4 NV), what
// a pass needs beside them, and no more, so that several rows are in flight.
constexpr int waves_for(int, int nv) { return nv >= 16 ? 4 : nv == 8 ? 6 : 8; }

struct Sum { template <typename V> __device__ V operator()(V a, V b) const { return a + b; } };
struct Max { template <typename V> __device__ V operator()(V a, V b) const { return a > b ? a : b; } };

// Reduction over the workgroup in a fixed order; every thread gets the
// result.  `red` (one slot per wave) may be used again after the call.
template <int NT, typename V, typename F>
__device__ __forceinline__ V block_reduce(V v, V* red, F f) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = f(v, __shfl_xor(v, o, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) v = f(v, red[w]);
  __syncthreads();
  return v;
}

// Sixteen bytes of a row, aligned to the element only: rows of odd length
// start anywhere, and the hardware's unaligned access costs less than peeling.
template <typename T> struct Row;
template <> struct Row<float> {
  static constexpr int N = 4;
  typedef float vec __attribute__((ext_vector_type(4), aligned(4)));
  typedef float reg __attribute__((ext_vector_type(4)));
  __device__ static float get(reg v, int j) { return v[j]; }
  __device__ static reg fill() { return reg{-INFINITY, -INFINITY, -INFINITY, -INFINITY}; }
  __device__ static void put(reg& v, int j, float x) { v[j] = x; }
  // element j, not known at compile time
  __device__ static float pick(reg v, int j) { return j < 2 ? (j ? v[1] : v[0]) : (j & 1 ? v[3] : v[2]); }
  __device__ static reg pack(const float (&x)[4]) { return reg{x[0], x[1], x[2], x[3]}; }
};
template <> struct Row<__bf16> {
  static constexpr int N = 8;
  typedef uint32_t vec __attribute__((ext_vector_type(4), aligned(2)));
  typedef uint32_t reg __attribute__((ext_vector_type(4)));
  __device__ static float get(reg v, int j) {
    return __uint_as_float((j & 1) ? (v[j / 2] & 0xffff0000u) : (v[j / 2] << 16));
  }
  __device__ static reg fill() { return reg{0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u}; }
  __device__ static void put(reg& v, int j, float x) {
    const uint32_t h = static_cast<uint32_t>(__builtin_bit_cast(uint16_t, static_cast<__bf16>(x)));
    v[j / 2] = (j & 1) ? (v[j / 2] & 0xffffu) | (h << 16) : (v[j / 2] & 0xffff0000u) | h;
  }
  __device__ static float pick(reg v, int j) {
    const uint32_t w = j < 4 ? (j < 2 ? v[0] : v[1]) : (j < 6 ? v[2] : v[3]);
    return __uint_as_float(j & 1 ? w & 0xffff0000u : w << 16);
  }
  __device__ static reg pack(const float (&x)[8]) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    reg v;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector((f2{x[2 * i], x[2 * i + 1]}), b2));
    return v;
  }
};

// A row, or a piece of one, in the registers of a workgroup of NT threads:
// vector v of thread t holds the N elements from (v NT + t) N on; places past
// the end hold -inf.
template <typename T, int NT, int NV>
struct RowRegs {
  static constexpr int N = Row<T>::N, kCapacity = NT * NV * N;
  typename Row<T>::reg x[NV];
  int len;

  __device__ __forceinline__ int at(int v) const { return (v * NT + static_cast<int>(threadIdx.x)) * N; }

  __device__ __forceinline__ void load(const T* p, int n) {
    len = n;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = at(v);
      if (e + N <= n) {
        x[v] = *reinterpret_cast<const typename Row<T>::vec*>(p + e);
      } else if (e < n && n >= N) {
        // the row's last vector, of which the first elements belong to the one
        // before: shifted out, with -inf behind
        x[v] = tail(*reinterpret_cast<const typename Row<T>::vec*>(p + n - N), n - e);
      } else {
        x[v] = Row<T>::fill();
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (e + j < n) Row<T>::put(x[v], j, static_cast<float>(p[e + j]));
      }
    }
  }
  // the last k elements of w in front, -inf behind them (0 < k < N)
  static __device__ __forceinline__ typename Row<T>::reg tail(typename Row<T>::reg w, int k) {
    typedef u64 u64x2 __attribute__((ext_vector_type(2)));
    const u64x2 a = __builtin_bit_cast(u64x2, w), f = __builtin_bit_cast(u64x2, Row<T>::fill());
    const int keep = k * static_cast<int>(sizeof(T)) * 8, out = 128 - keep;
    u64x2 r;
    r[0] = out >= 64 ? a[1] >> (out - 64) : (a[0] >> out) | (a[1] << (64 - out));
    r[1] = out >= 64 ? 0 : a[1] >> out;
    const u64 m0 = keep >= 64 ? ~u64{0} : (u64{1} << keep) - 1, m1 = keep > 64 ? (u64{1} << (keep - 64)) - 1 : 0;
    r[0] = (r[0] & m0) | (f[0] & ~m0);
    r[1] = (r[1] & m1) | (f[1] & ~m1);
    return __builtin_bit_cast(typename Row<T>::reg, r);
  }
  // Makes the compiler unpack the elements again rather than keep what an
  // earlier pass unpacked (twice the registers, half the rows in flight).
  __device__ __forceinline__ void fresh() {
#pragma unroll
    for (int v = 0; v < NV; ++v) asm volatile("" : "+v"(x[v]));
  }
  // f(value) over the thread's places
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < N; ++j) f(Row<T>::get(x[v], j));
  }
  __device__ __forceinline__ float max_value() const {
    float m = -INFINITY;
    each([&](float z) { m = fmaxf(m, z); });
    return m;
  }
  // emit(value, column) for every element that is not below `thr`
  template <typename F>
  __device__ __forceinline__ void scan(float thr, F emit) const {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      bool any = false;
#pragma unroll
      for (int j = 0; j < N; ++j) any |= !(Row<T>::get(x[v], j) < thr);
      if (any) {
        uint32_t hits = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) hits |= !(Row<T>::get(x[v], j) < thr) ? 1u << j : 0u;
        for (; hits; hits &= hits - 1) {
          const int j = __builtin_ctz(hits);
          if (at(v) + j < len) emit(Row<T>::pick(x[v], j), at(v) + j);
        }
      }
    }
  }
};

// ------------------------------------------------------------ alternatives
// The n largest keys, sorted, into lds.keys.  A lower bound comes from the n-th
// largest of the threads' own maxima (n elements are at least that large; the
// search looks at the upper half of the keys and rounds down); the elements
// that reach it, little more than n unless many are equal, go to a list, and
// each takes its place by counting the larger ones.  A list that overflows
// (plateaus; rows whose mask leaves fewer threads with a token than n) is
// replaced by an exact search for the n-th key over all elements, a bit at a
// time, each of which reads the row again: 4096 x 32000 bf16 with 64
// alternatives takes 10.9 ms instead of 75 us when every row comes to that
// (one column in a thousand left, or all equal), 3 rows 136 us instead of 16.
constexpr int kCand = 512;
template <int NT>
struct TopLds {
  __attribute__((aligned(16))) u64 cand[kCand];
  u64 keys[kMaxTop];
  uint32_t upper[NT];
  int count;
  uint32_t bound;
  int red[NT / 64];
};

// The n-th largest upper half among NT threads' maxima, found by one wave.
template <int NT>
__device__ __forceinline__ float top_bound(uint32_t mine, int n, TopLds<NT>& l) {
  l.upper[threadIdx.x] = mine >> 16;
  if (threadIdx.x == 0) l.count = 0;
  __syncthreads();
  if (threadIdx.x < 64) {
    uint32_t u[NT / 64];
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) u[w] = l.upper[w * 64 + threadIdx.x];
    uint32_t b = 0;
#pragma unroll
    for (int bit = 15; bit >= 0; --bit) {
      const uint32_t t = b | (1u << bit);
      int c = 0;
#pragma unroll
      for (int w = 0; w < NT / 64; ++w) c += __popcll(__ballot(u[w] >= t));
      if (c >= n) b = t;
    }
    if (threadIdx.x == 0) l.bound = b;
  }
  __syncthreads();
  return key_value(l.bound << 16);
}

template <int NT>
__device__ __forceinline__ void rank_sort(int count, int n, TopLds<NT>& l) {
  // four keys at a time, the last ones filled up with the lowest
  if (threadIdx.x < 4 && count + threadIdx.x < kCand) l.cand[count + threadIdx.x] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < count; i += NT) {
    const u64 k = l.cand[i];
    int rank = 0;
    for (int j = 0; j < count; j += 4)
#pragma unroll
      for (int q = 0; q < 4; ++q) rank += l.cand[j + q] > k;
    if (rank < n) l.keys[rank] = k;
  }
  __syncthreads();
}

template <int NT>
__device__ __forceinline__ void append(u64 k, TopLds<NT>& l) {
  const int i = atomicAdd(&l.count, 1);       // any order: ranks decide
  if (i < kCand) l.cand[i] = k;
}

// The exact search over key(0) .. key(len - 1): the n-th largest a bit at a
// time, then the list again.
template <int NT, typename K>
__device__ __forceinline__ void exact_top(K key, int len, int n, TopLds<NT>& l) {
  u64 low = 0;
  for (int bit = 63; bit >= 0; --bit) {
    const u64 t = low | (u64{1} << bit);
    int c = 0;
    for (int i = threadIdx.x; i < len; i += NT) c += key(i) >= t;
    if (block_reduce<NT>(c, l.red, Sum()) >= n) low = t;
  }
  if (threadIdx.x == 0) l.count = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < len; i += NT)
    if (key(i) >= low) append<NT>(key(i), l);
  __syncthreads();
}

template <typename T, int NT, int NV>
__device__ __forceinline__ void select_top(RowRegs<T, NT, NV>& row, const T* z, float mine, int col0, int n, TopLds<NT>& l) {
  const float thr = top_bound<NT>(row.at(0) < row.len ? order_key(mine) : 0u, n, l);
  row.fresh();
  row.scan(thr, [&](float v, int c) { append<NT>(top_key(v, col0 + c), l); });
  __syncthreads();
  int count = l.count;
  __syncthreads();
  if (count > kCand) {
    exact_top<NT>([&](int c) { return top_key(static_cast<float>(z[c]), col0 + c); }, row.len, n, l);
    count = n;
  }
  rank_sort<NT>(count, n, l);
}

struct Stats { float ref, s, u; };

// The largest element (-inf for a row without any), S and U.
template <bool kEntropy, typename T, int NT, int NV>
__device__ __forceinline__ Stats row_stats(RowRegs<T, NT, NV>& row, float m, float c, float* red) {
  m = block_reduce<NT>(m, red, Max());
  Stats st;
  st.ref = m == -INFINITY ? 0.0f : m;
  float s = 0.0f, u = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    // a vector at a time: unpacking the next ones early takes registers from
    // other rows
    asm volatile("" : "+v"(row.x[v]), "+v"(s), "+v"(u));
#pragma unroll
    for (int j = 0; j < Row<T>::N; ++j) {
      const float x = Row<T>::get(row.x[v], j) - st.ref, e = exp2_(x * c);
      s += e;
      if constexpr (kEntropy) u = fmaf(e, fmaxf(x, kLowest), u);   // 0 times -inf counts as 0
    }
  }
  st.s = block_reduce<NT>(s, red, Sum());
  st.u = kEntropy ? block_reduce<NT>(u, red, Sum()) : 0.0f;
  if (m == -INFINITY) st.ref = -INFINITY;
  return st;
}

// The outputs of one row.
struct RowOut {
  const LogprobArgs& a;
  int64_t r;
  Stats st;
  float lg;
  __device__ RowOut(const LogprobArgs& args, int64_t row, Stats s) : a(args), r(row), st(s) {
    lg = s.ref == -INFINITY ? NAN : log2_(s.s) * kLn2;
  }
  __device__ float logp(float z) const { return (z - st.ref) * a.inv_tau - lg; }
  template <typename T>
  __device__ void scalars(const T* z) const {
    if (a.tokens) {
      const int64_t tok = a.tokens[r];
      a.logprob[r] = tok < 0 ? 0.0f : tok < a.vocab ? logp(static_cast<float>(z[tok])) : NAN;
    }
    if (a.entropy) a.entropy[r] = lg - st.u / st.s * a.inv_tau;
  }
  __device__ void top(int i, u64 k) const {
    a.top_index[r * a.top + i] = key_col(k);
    a.top_logprob[r * a.top + i] = logp(key_value(static_cast<uint32_t>(k >> 32)));
  }
};

// One workgroup per row (pieces = 1) or per piece, whose statistics and
// sorted keys then go to the workspace.
template <typename T, int NT, int NV>
__global__ void __launch_bounds__(NT, waves_for(NT, NV)) logprobs_kernel(const LogprobArgs a) {
  __shared__ float red[NT / 64];
  __shared__ TopLds<NT> lds;
  const uint32_t pieces = static_cast<uint32_t>(a.pieces);
  const int64_t r = blockIdx.x / pieces;
  const int piece = static_cast<int>(blockIdx.x % pieces);
  const T* z = static_cast<const T*>(a.logits) + r * a.ld;
  const int col0 = piece * a.piece_len;
  RowRegs<T, NT, NV> row;
  row.load(z + col0, min(a.piece_len, a.vocab - col0));
  const float mine = row.max_value();
  const Stats st = row_stats<true>(row, mine, a.inv_tau * kLog2e, red);
  const int n = min(a.top, row.len);
  if (n > 0) select_top(row, z + col0, mine, col0, n, lds);
  if (pieces == 1) {
    const RowOut out(a, r, st);
    if (threadIdx.x == 0) out.scalars(z);
    if (threadIdx.x < static_cast<uint32_t>(n)) out.top(threadIdx.x, lds.keys[threadIdx.x]);
  } else {
    if (threadIdx.x == 0) a.part[blockIdx.x] = {st.ref, st.s, st.u, 0.0f};
    if (threadIdx.x < static_cast<uint32_t>(a.top))
      a.part_keys[static_cast<int64_t>(blockIdx.x) * a.top + threadIdx.x] = threadIdx.x < static_cast<uint32_t>(n) ? lds.keys[threadIdx.x] : 0;
  }
}

// Joined statistics of a row's pieces.
template <int NT>
__device__ __forceinline__ Stats join(const float4* part, int pieces, float c, float* red) {
  Stats st{-INFINITY, 0.0f, 0.0f};
  for (int i = threadIdx.x; i < pieces; i += NT) st.ref = fmaxf(st.ref, part[i].x);
  st.ref = block_reduce<NT>(st.ref, red, Max());
  for (int i = threadIdx.x; i < pieces; i += NT) {
    const float4 p = part[i];
    // a piece of -inf only adds nothing (but NaN, if that is its sum)
    const float x = p.x - st.ref, w = st.ref == -INFINITY ? 0.0f : exp2_(x * c);
    const float ws = w * p.y;
    st.s += ws;
    st.u += fmaf(ws, fmaxf(x, kLowest), w * p.z);
  }
  st.s = block_reduce<NT>(st.s, red, Sum());
  st.u = block_reduce<NT>(st.u, red, Sum());
  return st;
}

template <typename T>
__global__ void __launch_bounds__(256) logprobs_join_kernel(const LogprobArgs a) {
  constexpr int NT = 256;
  __shared__ float red[NT / 64];
  __shared__ TopLds<NT> lds;
  const int64_t r = blockIdx.x;
  const RowOut out(a, r, join<NT>(a.part + r * a.pieces, a.pieces, a.inv_tau * kLog2e, red));
  if (threadIdx.x == 0) out.scalars(static_cast<const T*>(a.logits) + r * a.ld);
  const int n = a.top;
  if (n == 0) return;
  const u64* keys = a.part_keys + r * a.pieces * static_cast<int64_t>(n);
  const int len = a.pieces * n;
  // the keys of all pieces, as above; a piece's own n are sorted, so the
  // threads' maxima spread over the pieces
  uint32_t mine = 0;
  for (int i = threadIdx.x; i < len; i += NT) mine = max(mine, static_cast<uint32_t>(keys[i] >> 32));
  top_bound<NT>(mine, n, lds);
  const u64 bound = static_cast<u64>(lds.bound) << 48;
  for (int i = threadIdx.x; i < len; i += NT)
    if (keys[i] >= bound && keys[i]) append<NT>(keys[i], lds);
  __syncthreads();
  int count = lds.count;
  __syncthreads();
  if (count > kCand) {
    exact_top<NT>([&](int i) { return keys[i]; }, len, n, lds);
    count = n;
  }
  rank_sort<NT>(count, n, lds);
  if (threadIdx.x < static_cast<uint32_t>(n)) out.top(threadIdx.x, lds.keys[threadIdx.x]);
}

// ------------------------------------------------------------- distillation
// The teacher's side of a row: softmax over its present slots, slot k in
// thread k of the first two waves.
struct Teacher {
  float p, tau_logp;     // (tau log p stays finite where log p does not)
  int col;               // -1: absent, of no weight, or not a column
  bool skip, bad;
};

template <int NT>
__device__ __forceinline__ Teacher teacher(const DistillArgs& a, int64_t r, float* red) {
  const int tid = threadIdx.x;
  int64_t idx = -1;
  float t = -INFINITY;
  if (tid < a.top) {
    idx = a.top_index[r * a.top + tid];
    if (idx >= 0) t = a.top_logit[r * a.top + tid];
  }
  const float wrong = idx >= a.vocab || t != t || t == INFINITY ? 1.0f : 0.0f;
  Teacher q;
  q.bad = block_reduce<NT>(wrong, red, Max()) > 0.0f;
  if (q.bad) t = -INFINITY;
  const float m = block_reduce<NT>(t, red, Max());
  q.skip = m == -INFINITY && !q.bad;
  const float x = t - (m == -INFINITY ? 0.0f : m), e = exp2_(x * a.inv_tau * kLog2e), s = block_reduce<NT>(e, red, Sum());
  q.p = s > 0.0f ? e / s : 0.0f;
  q.tau_logp = x - log2_(s) * (kLn2 * a.tau);
  q.col = q.p > 0.0f ? static_cast<int>(idx) : -1;
  return q;
}

// tau^2 sum p (log p - log q) as tau sum p (tau log p - tau log q), in every
// thread: tau^2 underflows below tau = 2^-75, and a logit's distance from the
// largest, over tau, overflows near 2^-126, where the loss itself does neither.
template <int NT, typename T>
__device__ __forceinline__ float distill_value(const DistillArgs& a, const Teacher& q, const T* z, Stats st, float* red) {
  const float lq = q.col >= 0 ? (static_cast<float>(z[q.col]) - st.ref) - log2_(st.s) * (kLn2 * a.tau) : 0.0f;
  const float l = block_reduce<NT>(q.col >= 0 ? q.p * (q.tau_logp - lq) : 0.0f, red, Sum());
  return q.bad || st.ref == -INFINITY || st.s != st.s ? NAN : a.tau * l;
}

template <int NT>
struct SlotLds {
  float prob[kMaxTop];
  int col[kMaxTop];
};

// Writes the gradient of the registers' elements: g tau q everywhere, then the
// teacher's columns that lie in them again with their probabilities taken
// off (a column's first slot adds up all of its slots).
template <typename T, int NT, int NV>
__device__ __forceinline__ void write_grad(const DistillArgs& a, RowRegs<T, NT, NV>& row, const T* z, T* grad, int col0,
                                           const Teacher& q, Stats st, float g, SlotLds<NT>& l) {
  const int tid = threadIdx.x;
  if (tid < a.top) {
    l.prob[tid] = q.p;
    l.col[tid] = q.col;
  }
  const bool nan_row = q.bad || st.ref == -INFINITY;
  const bool zero = q.skip || g == 0.0f;
  const float c = a.inv_tau * kLog2e, scale = zero ? 0.0f : g * a.tau;
  const float w = nan_row ? NAN : scale / st.s, ref = nan_row ? 0.0f : st.ref;
  T* out = grad + col0;
  row.fresh();
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = row.at(v);
    float x[Row<T>::N];
#pragma unroll
    for (int j = 0; j < Row<T>::N; ++j) x[j] = zero ? 0.0f : exp2_((Row<T>::get(row.x[v], j) - ref) * c) * w;
    const typename Row<T>::reg o = Row<T>::pack(x);
    if (e + Row<T>::N <= row.len) {
      *reinterpret_cast<typename Row<T>::vec*>(out + e) = o;
    } else {
#pragma unroll
      for (int j = 0; j < Row<T>::N; ++j)
        if (e + j < row.len) out[e + j] = static_cast<T>(Row<T>::get(o, j));
    }
  }
  if (zero || nan_row) return;
  __builtin_amdgcn_s_waitcnt(0x0f70);            // these stores before the teacher's columns
  __syncthreads();
  if (tid < a.top) {
    const int j = l.col[tid];
    if (j >= col0 && j < col0 + row.len) {
      float sum = 0.0f;
      bool first = true;
      for (int k = 0; k < a.top; ++k)
        if (l.col[k] == j) {
          if (k < tid) first = false;
          sum += l.prob[k];
        }
      if (first) grad[j] = static_cast<T>(exp2_((static_cast<float>(z[j]) - ref) * c) * w - scale * sum);
    }
  }
}

// kPhase 0: a workgroup per row does everything.  1: a workgroup per piece
// writes the piece's statistics.  2: a workgroup per piece joins its row's
// and writes the piece's gradient (and, for the first piece, the loss).
template <typename T, int NT, int NV, int kPhase>
__global__ void __launch_bounds__(NT, waves_for(NT, NV)) distill_kernel(const DistillArgs a) {
  __shared__ float red[NT / 64];
  __shared__ SlotLds<NT> lds;
  const uint32_t pieces = kPhase == 0 ? 1u : static_cast<uint32_t>(a.pieces);
  const int64_t r = blockIdx.x / pieces;
  const int piece = static_cast<int>(blockIdx.x % pieces);
  const T* z = static_cast<const T*>(a.logits) + r * a.ld;
  const int col0 = piece * a.piece_len;
  if (kPhase == 2 && !a.grad && piece) return;
  RowRegs<T, NT, NV> row;
  if (kPhase != 2 || a.grad) row.load(z + col0, min(a.piece_len, a.vocab - col0));
  if constexpr (kPhase == 1) {
    const Stats st = row_stats<false>(row, row.max_value(), a.inv_tau * kLog2e, red);
    if (threadIdx.x == 0) a.part[blockIdx.x] = {st.ref, st.s, 0.0f, 0.0f};
    return;
  } else {
    const Teacher q = teacher<NT>(a, r, red);
    const float g = a.grad && a.grad_loss ? a.grad_loss[r] : 1.0f;
    Stats st;
    if constexpr (kPhase == 0) st = row_stats<false>(row, row.max_value(), a.inv_tau * kLog2e, red);
    else st = join<NT>(a.part + r * pieces, static_cast<int>(pieces), a.inv_tau * kLog2e, red);
    if (a.loss && piece == 0) {
      const float l = q.skip ? 0.0f : distill_value<NT>(a, q, z, st, red);
      if (threadIdx.x == 0) a.loss[r] = l;
    }
    if (a.grad) write_grad(a, row, z, static_cast<T*>(a.grad) + r * a.ld_grad, col0, q, st, g, lds);
  }
}

}  // namespace

// -------------------------------------------------------------------- launches
// Pieces of a row: a row of at most `whole` bytes, which a workgroup's
// registers hold, is not cut, however few rows there are.  Longer ones are cut
// into 64 KiB, or, where that leaves most of the chip idle, into 16 KiB.
namespace {
constexpr int64_t kSmallPiece = 16 << 10, kLargePiece = 64 << 10;

struct Cut { int pieces, len; };

Cut cut(int64_t rows, int64_t vocab, int esz, int64_t whole) {
  const int64_t bytes = vocab * esz;
  int64_t piece = bytes;
  if (bytes > whole) piece = rows * bytes < 256 * kLargePiece ? kSmallPiece : kLargePiece;
  const int64_t n = (bytes + piece - 1) / piece;
  int64_t len = (vocab + n - 1) / n;                   // pieces of about equal length, in whole vectors
  if (n > 1) len = (len + 7) / 8 * 8;
  return {static_cast<int>((vocab + len - 1) / len), static_cast<int>(len)};
}

constexpr int64_t kLogprobsWhole = 64 << 10, kDistillWhole = 320 << 10;

size_t up(size_t x) { return (x + 255) / 256 * 256; }
}  // namespace

static size_t logprobs_ws(const Cut& c, int64_t rows, int top) {
  if (c.pieces == 1) return 0;
  const size_t n = static_cast<size_t>(rows) * static_cast<size_t>(c.pieces);
  return up(n * sizeof(float4)) + up(n * static_cast<size_t>(top) * 8);
}

// The query does not know the element type: the larger of the two.
size_t logprobs_workspace(int64_t rows, int64_t vocab, int top) {
  const size_t a = logprobs_ws(cut(rows, vocab, 4, kLogprobsWhole), rows, top);
  const size_t b = logprobs_ws(cut(rows, vocab, 2, kLogprobsWhole), rows, top);
  return a > b ? a : b;
}

size_t distill_workspace(int64_t rows, int64_t vocab, int) {
  size_t n = 0;
  for (int esz : {4, 2}) {
    const Cut c = cut(rows, vocab, esz, kDistillWhole);
    const size_t b = c.pieces == 1 ? 0 : up(static_cast<size_t>(rows) * static_cast<size_t>(c.pieces) * sizeof(float4));
    n = b > n ? b : n;
  }
  return n;
}

// Workgroups of a launch that covers `rows` rows.
bool token_grid_fits(int64_t rows, int64_t vocab) {
  for (int esz : {4, 2})
    for (int64_t whole : {kLogprobsWhole, kDistillWhole}) {
      const Cut c = cut(rows, vocab, esz, whole);
      if (rows * c.pieces > int64_t{0xffffffff} / 1024) return false;
    }
  return true;
}

// Calls f with the smallest (threads, vectors) whose registers hold `bytes`:
// enough waves per row to have many loads in flight, few enough that several
// rows share a CU.
template <int64_t kWhole, typename F>
static hipError_t with_size(int64_t bytes, F f) {
#define MO_SIZE(NT, NV) f(std::integral_constant<int, NT>{}, std::integral_constant<int, NV>{})
  if (bytes <= 4 << 10) return MO_SIZE(256, 1);
  if (bytes <= 8 << 10) return MO_SIZE(256, 2);
  if (bytes <= 16 << 10) return MO_SIZE(256, 4);
  if (bytes <= 32 << 10) return MO_SIZE(256, 8);
  if constexpr (kWhole > 64 << 10) {
    if (bytes > 256 << 10) return MO_SIZE(1024, 20);
    if (bytes > 128 << 10) return MO_SIZE(1024, 16);
    if (bytes > 64 << 10) return MO_SIZE(512, 16);
  }
  return MO_SIZE(256, 16);
#undef MO_SIZE
}

template <typename T>
static hipError_t run_logprobs(LogprobArgs a, void* ws, hipStream_t s) {
  const Cut c = cut(a.rows, a.vocab, sizeof(T), kLogprobsWhole);
  a.pieces = c.pieces;
  a.piece_len = c.len;
  const size_t n = static_cast<size_t>(a.rows) * static_cast<size_t>(c.pieces);
  a.part = static_cast<float4*>(ws);
  a.part_keys = reinterpret_cast<u64*>(static_cast<char*>(ws) + up(n * sizeof(float4)));
  const hipError_t e = with_size<kLogprobsWhole>(static_cast<int64_t>(c.len) * sizeof(T), [&](auto NT, auto NV) {
    logprobs_kernel<T, NT, NV><<<static_cast<uint32_t>(n), NT.value, 0, s>>>(a);
    return hipGetLastError();
  });
  if (e != hipSuccess || c.pieces == 1) return e;
  logprobs_join_kernel<T><<<a.rows, 256, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_logprobs(int dt, const LogprobArgs& a, void* ws, hipStream_t s) {
  return dt == F32 ? run_logprobs<float>(a, ws, s) : run_logprobs<__bf16>(a, ws, s);
}

template <typename T>
static hipError_t run_distill(DistillArgs a, void* ws, hipStream_t s) {
  const Cut c = cut(a.rows, a.vocab, sizeof(T), kDistillWhole);
  a.pieces = c.pieces;
  a.piece_len = c.len;
  a.part = static_cast<float4*>(ws);
  const uint32_t n = static_cast<uint32_t>(a.rows) * static_cast<uint32_t>(c.pieces);
  const int64_t bytes = static_cast<int64_t>(c.len) * sizeof(T);
  if (c.pieces == 1)
    return with_size<kDistillWhole>(bytes, [&](auto NT, auto NV) {
      distill_kernel<T, NT, NV, 0><<<n, NT.value, 0, s>>>(a);
      return hipGetLastError();
    });
  // pieces have one of two sizes
  auto both = [&](auto NT, auto NV) {
    distill_kernel<T, NT, NV, 1><<<n, NT.value, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    distill_kernel<T, NT, NV, 2><<<n, NT.value, 0, s>>>(a);
    return hipGetLastError();
  };
  return bytes <= kSmallPiece ? both(std::integral_constant<int, 256>{}, std::integral_constant<int, 4>{})
                              : both(std::integral_constant<int, 256>{}, std::integral_constant<int, 16>{});
}

hipError_t launch_distill(int dt, const DistillArgs& a, void* ws, hipStream_t s) {
  return dt == F32 ? run_distill<float>(a, ws, s) : run_distill<__bf16>(a, ws, s);
}

}  // namespace mo
