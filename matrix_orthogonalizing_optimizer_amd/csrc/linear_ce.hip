// Cross entropy of logits z = x W^T that no caller keeps, with the gradients for
// x and W (gfx950).
//
//   loss_t = log sum_v exp z_tv - z_{t, target}
//   dz_tv = g_t (exp(z_tv - log sum exp z_t) - [v = target]),  dx = dz W,  dW = dz^T x
//
// The products run on the matrix cores in bf16 with fp32 sums, in pieces of the
// vocabulary.  A first product's tiles leave each row's largest logit and sum of
// exponentials per tile, and the logits where the workspace holds them.  With the
// row's statistics known a pass over the logits, or a second product, makes a
// piece's dz, which two further products contract with the piece's weights and
// with x.
#include <algorithm>
#include <cmath>

#include "linear_ce_internal.h"
#include "mo_internal.h"
#include "tile_product.h"

namespace mo {

namespace {

typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.44269504088896340736f;

// dz enters its products as a sum of bf16 terms: one where the gradient is
// bf16 itself (its rounding, up to 2^-8 of a value, is of the size of the result's
// own: the 2-norm of a gradient's error grows from 0.0017 to 0.0020 of its own,
// 8192 x 32000 x 2048), three where it is fp32 (2^-26: x and W are exact in bf16, so
// that the statistics and the fp32 sums are the only other errors).
constexpr int terms_of(int dt) { return dt == F32 ? 3 : 1; }

// LDS that only one wave uses: the hardware keeps the wave's accesses in order,
// and the compiler keeps them so here.
__device__ __forceinline__ void wave_order() { asm volatile("" ::: "memory"); }

int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// Rows of the workspace's matrices lie an odd number of 256 bytes apart, so that
// the rows of a tile spread over the memory's channels: 1024 x 2048 x 31744 in 8
// splits takes 118 us with rows 63744 bytes apart, 134 with 65024.  (Products whose
// contraction is not split take the same with either.)
int64_t apart(int64_t elements) { return ((elements + 127) / 128 | 1) * 128; }

// ------------------------------------------------------------ rows and packing
// Rows' weights in dz are relative to the largest |g| of those that take part (so
// that equal g do not add a rounding of their own to dz's): scale[0], or 1.  One
// workgroup finds it beside those that pack x.
struct CeRows {
  const int64_t* targets;       // null: nothing to do
  const float* g;               // or null: 1
  float* scale;
  int rows;
};
__device__ __forceinline__ void ce_scale(const CeRows& a) {
  constexpr int kAtOnce = 8;                                  // rows of a thread whose loads are in flight
  __shared__ float most[4];
  float m = 0.0f;
  if (a.g)
    for (int t0 = threadIdx.x; t0 < a.rows; t0 += 256 * kAtOnce) {
      int64_t y[kAtOnce];
      float r[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int t = min(t0 + 256 * i, a.rows - 1);          // some twice
        y[i] = a.targets[t];
        r[i] = a.g[t];
      }
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) m = y[i] >= 0 ? fmaxf(m, fabsf(r[i])) : m;      // NaN is left out
    }
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
  if ((threadIdx.x & 63) == 0) most[threadIdx.x >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3]));
  if (threadIdx.x == 0) *a.scale = m > 0.0f && m < INFINITY ? m : 1.0f;
}

// bf16 copies of a [rows, cols] matrix: dst [rows][pitch] (columns past `cols`,
// up to a multiple of 64, zero) and its transpose dst_t [cols][pitch_t] (rows
// past `rows` likewise, and of x those that take no part, whatever they hold).  64 rows x 128 columns per workgroup, through LDS; HBM bound:
// 129283 x 2045 fp32 to both 425 us, 5.0 TB/s.
constexpr int kPackRows = 64, kPackCols = 128;
// Eight rows of a column.
__device__ __forceinline__ u32x4v column8(const uint32_t (&tile)[kPackRows][kPackCols / 2 + 1], int r, int c) {
  const int shift = (c & 1) * 16;
  u32x4v v;
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = ((tile[r + 2 * k][c / 2] >> shift) & 0xffffu) | ((tile[r + 2 * k + 1][c / 2] >> shift) << 16);
  return v;
}

template <typename T>
__global__ void __launch_bounds__(256) ce_pack_kernel(const T* src, int64_t ld, int rows, int cols, uint16_t* dst, int64_t pitch,
                                                      uint16_t* dst_t, int64_t pitch_t, const CeRows job) {
  const int64_t tile_r = static_cast<int64_t>(blockIdx.x) - (job.targets ? 1 : 0);
  if (tile_r < 0) {                                          // the first one, as it takes longest
    if (blockIdx.y == 0) ce_scale(job);
    return;
  }
  const int64_t cols_p = (static_cast<int64_t>(cols) + 63) / 64 * 64, rows_p = (static_cast<int64_t>(rows) + 63) / 64 * 64;
  __shared__ uint32_t tile[kPackRows][kPackCols / 2 + 1];       // pairs of columns; odd rows of dwords: columns spread over the banks
  const int64_t r0 = tile_r * kPackRows, c0 = static_cast<int64_t>(blockIdx.y) * kPackCols;
  const int cl = (threadIdx.x & 15) * 8, rl = threadIdx.x >> 4;
  const int left = static_cast<int>(min(int64_t{8}, cols - c0 - cl));
  Oct<T> o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[i].clear();
    if (r0 + rl + 16 * i < rows && left > 0) o[i].load(src + (r0 + rl + 16 * i) * ld + c0 + cl, left);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + rl + 16 * i;
    const u32x4v v = {pack_bf16x2(o[i].get(0), o[i].get(1)), pack_bf16x2(o[i].get(2), o[i].get(3)),
                      pack_bf16x2(o[i].get(4), o[i].get(5)), pack_bf16x2(o[i].get(6), o[i].get(7))};
    if (dst && r < rows && c0 + cl < cols_p) *reinterpret_cast<u32x4v*>(dst + r * pitch + c0 + cl) = v;
    const bool out = job.targets && r < rows && (job.targets[r] < 0 || (job.g && job.g[r] == 0.0f));
#pragma unroll
    for (int k = 0; k < 4; ++k) tile[rl + 16 * i][cl / 2 + k] = out ? 0u : v[k];
  }
  if (!dst_t) return;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int u = i * 256 + threadIdx.x, c = u >> 3, r = (u & 7) * 8;       // 8 rows of a column
    if (c0 + c >= cols || r0 + r >= rows_p) continue;
    *reinterpret_cast<u32x4v*>(dst_t + (c0 + c) * pitch_t + r0 + r) = column8(tile, r, c);
  }
}

hipError_t pack(int dt, const void* src, int64_t ld, int rows, int cols, uint16_t* dst, int64_t pitch, uint16_t* dst_t, int64_t pitch_t,
                const CeRows& job, hipStream_t s) {
  // rows along the grid's long axis: up to 2^22 columns are 2^15 workgroups
  const int64_t tiles = (static_cast<int64_t>(rows) + kPackRows - 1) / kPackRows + (job.targets ? 1 : 0);
  const dim3 g(static_cast<uint32_t>(tiles), static_cast<uint32_t>((cols + kPackCols - 1) / kPackCols));
  if (dt == F32) ce_pack_kernel<float><<<g, 256, 0, s>>>(static_cast<const float*>(src), ld, rows, cols, dst, pitch, dst_t, pitch_t, job);
  else ce_pack_kernel<__bf16><<<g, 256, 0, s>>>(static_cast<const __bf16*>(src), ld, rows, cols, dst, pitch, dst_t, pitch_t, job);
  return hipGetLastError();
}

// ------------------------------------------------------------ statistics
// A row's reference m is its largest logit, sums are of exp(z - m): the difference
// first, as the rounding of a product z log2(e) passes every exponent from logits
// of 2^31 on.  (z log2(e) - m' in one multiply-add saves nothing: 8192 x 32000 x 2048
// 3075 us either way, logits multiplied again, x 128, 838 instead of 834.)  The
// target's column stays out of both and joins them last: a likely token's loss and
// dz are made of the other columns' sum, as 1 - p of a rounded p has none of their
// digits left.
//
// The product bounds it: 8192 x 28160 x 2048 takes 773 us without the logits (1.22
// PFLOP/s), 8192 x 32000 x 2048 970 to 1090 with them (1.05 GB), 838 stored in bf16
// without statistics.  3 x
// 32000 x 2048 takes 21 us, the weights from the last-level cache.
struct CeStatsArgs {
  const int64_t* targets;
  int64_t col0;                 // the piece's first column
  float2* part;                 // [rows][tiles_n]: reference, sum
  float* target;                // the target's logit, written by the tile that holds it
  float* z;                     // or null: the logits, rows `pitch_z` apart
  int64_t pitch_z;
  int stream_z;
};

// exp(z - ref), where z is not above ref.
__device__ __forceinline__ float exp_below(float z, float ref) { return __builtin_amdgcn_exp2f((z - ref) * kLog2e); }

// Adds (m2, s2) to (m, s).  References of -inf stand for columns of -inf only.
__device__ __forceinline__ void join_stats(float& m, float& s, float m2, float s2) {
  const float n = fmaxf(m, m2), ref = n == -INFINITY ? 0.0f : n;
  s = s * exp_below(m, ref) + s2 * exp_below(m2, ref);
  m = n;
}

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kMinWaves) ce_stats_kernel(const ProductArgs p, const CeStatsArgs e) {
  constexpr int W = C::TN / C::WN;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::kLds];
  const TilePlace q = tile_place<C>(p);
  f32x16v acc[C::FM][C::FN];
  tile_sums<C>(p, q, smem, acc);
  if (e.z) {
    tile_store<C, float>({e.z + e.col0, e.pitch_z, 0, 0, nullptr, e.stream_z}, q, smem, acc);
    __syncthreads();
  }
  float2* waves = reinterpret_cast<float2*>(smem);                      // [TM][WN]
  const int inside = q.nlast + 1 - q.wn * W;                            // of the wave's columns
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
    if (inside < W) {
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (32 * j + 8 * (r / 4) + 4 * q.half + r % 4 >= inside) acc[i][j][r] = -INFINITY;
    }
    const int row = q.wm * (C::TM / C::WM) + 32 * i + q.r32;
    const bool in = row <= q.mlast;
    const int64_t t = q.m0 + row;
    // the target's logit, where these columns hold it, goes by itself
    const int64_t y = in ? e.targets[t] - e.col0 - q.n0 - q.wn * W : -1;
    const bool mine = y >= 0 && y < min(W, inside) && ((y >> 2) & 1) == q.half;
    if (__any(mine)) {
      float z = 0.0f;
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r)
          if (mine && y == 32 * j + 8 * (r / 4) + 4 * q.half + r % 4) {
            z = acc[i][j][r];
            acc[i][j][r] = -INFINITY;
          }
      if (mine) e.target[t] = z;
    }
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) m = fmaxf(m, acc[i][j][r]);
    m = fmaxf(m, __uint_as_float(lane_xor32(__float_as_uint(m))));
    const float ref = m == -INFINITY ? 0.0f : m;            // columns of -inf alone: a sum of zero
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) s += exp_below(acc[i][j][r], ref);
    s += __uint_as_float(lane_xor32(__float_as_uint(s)));
    if (q.half == 0) waves[row * C::WN + q.wn] = make_float2(m, s);
  }
  __syncthreads();
  for (int row = threadIdx.x; row <= q.mlast; row += C::kThreads) {
    float2 v = waves[row * C::WN];
    for (int w = 1; w < C::WN; ++w) join_stats(v.x, v.y, waves[row * C::WN + w].x, waves[row * C::WN + w].y);
    e.part[(q.m0 + row) * p.tiles_n + q.tn] = v;
  }
}

// Joins a piece's statistics with those of the pieces before it, kLanes
// threads per row; after the last piece, with the target's logit, the row's {m, 1 /
// sum}, p - 1 of its target (in the logit's place), its loss and its weight in dz: 0
// where it takes no part, NaN for a target that is no column.
// Latency bound: 3 rows of 500 tiles take 3.9 us with 256 threads to a row and 5.8
// with 16, 1021 of 506 6.2 and 9.7, 8192 of 125 12.5 and 6.0.
template <int kLanes>
__global__ void __launch_bounds__(256) ce_join_kernel(const float2* part, int cols, int rows, int vocab, int first, int last,
                                                      const int64_t* targets, float* target, float2* stat, float* loss,
                                                      const float* g, const float* scale, float* factor) {
  __shared__ float2 waves[4];
  const int lane = threadIdx.x % kLanes;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (256 / kLanes) + threadIdx.x / kLanes;
  const bool in = t < rows;
  float m = -INFINITY, s = 0.0f;
  if (in)
#pragma unroll 4
    for (int c = lane; c < cols; c += kLanes) {
      const float2 v = part[t * cols + c];
      join_stats(m, s, v.x, v.y);
    }
  // a tree whose two sides always add in the same order
#pragma unroll
  for (int o = 1; o < (kLanes < 64 ? kLanes : 64); o <<= 1) {
    const float m2 = __shfl_xor(m, o, 64), s2 = __shfl_xor(s, o, 64);
    const bool low = (lane & o) == 0;
    float a = low ? m : m2, b = low ? s : s2;
    join_stats(a, b, low ? m2 : m, low ? s2 : s);
    m = a;
    s = b;
  }
  if constexpr (kLanes == 256) {
    if ((threadIdx.x & 63) == 0) waves[threadIdx.x >> 6] = make_float2(m, s);
    __syncthreads();
    m = waves[0].x;
    s = waves[0].y;
    for (int w = 1; w < 4; ++w) join_stats(m, s, waves[w].x, waves[w].y);
  }
  if (!in || lane) return;
  if (!first) {
    float2 v = stat[t];
    join_stats(v.x, v.y, m, s);
    m = v.x;
    s = v.y;
  }
  if (!last) {
    stat[t] = make_float2(m, s);
    return;
  }
  // -inf alone, or a NaN or +inf anywhere, gives NaN
  const int64_t y = targets[t];
  const bool column = y >= 0 && y < vocab;
  const float z = column ? target[t] : -INFINITY, top = fmaxf(m, z);
  const bool none = top == -INFINITY;
  const float rest = s * exp_below(m, none ? 0.0f : top), own = column ? exp_below(z, none ? 0.0f : top) : 0.0f;
  const float inv = none ? NAN : 1.0f / (rest + own);
  stat[t] = make_float2(top, inv);
  target[t] = -rest * inv;
  if (factor) {
    const float r = g ? g[t] : 1.0f;
    factor[t] = y < 0 || r == 0.0f ? 0.0f : y >= vocab ? NAN : r / *scale;
  }
  loss[t] = y < 0 ? 0.0f : !column || none ? NAN : (z == top ? log1pf(rest) : logf(rest + own)) + (top - z);
}

// ------------------------------------------------------------ dz
// Written as rows for dx and as columns for dw, both as whole lines.  From a
// second product: 8192 x 28160 x 2048 996 us, of which the product is 740.
struct CeGradArgs {
  const int64_t* targets;
  int64_t col0;
  const float2* stat;
  const float* target;          // p - 1 of the target's column
  const float* factor;
  uint16_t* dz;                 // [rows]: terms_x times vp, rows pitch_x apart
  uint16_t* dz_t;               // [columns]: terms_w times tp, pitch_w apart
  int terms_x, terms_w;         // 0: not wanted
  int vp, tp;                   // the piece's columns and the rows, padded (zeros)
  int64_t pitch_x, pitch_w;
};

template <class C>
__global__ void __launch_bounds__(C::kThreads, C::kMinWaves) ce_grad_kernel(const ProductArgs p, const CeGradArgs e) {
  constexpr int W = C::TN / C::WN;
  // places of a wave's 32 rows in LDS: rows of W bf16, and columns of 32, with
  // padding against bank conflicts
  constexpr int kPitch = W * 2 + 16, kPitchT = 80, kPlace = 32 * kPitch > W * kPitchT ? 32 * kPitch : W * kPitchT;
  static_assert(C::NW * kPlace <= C::kLds, "they fit the ring's place");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::kLds];
  const TilePlace q = tile_place<C>(p);
  f32x16v acc[C::FM][C::FN];
  tile_sums<C>(p, q, smem, acc);
  uint8_t* turn = smem + (q.wm * C::WN + q.wn) * kPlace;
  const int inside = q.nlast + 1 - q.wn * W;                            // of the wave's columns
  const int terms = max(e.terms_x, e.terms_w);
  const bool odd = q.lane & 1;
  // rows r and r + 1 of a column: an even lane takes its own and its neighbour's
  // first column of a pair, an odd lane their second
  const uint32_t pick = odd ? 0x07060302u : 0x01000504u;
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
    const int row = q.wm * (C::TM / C::WM) + 32 * i + q.r32;
    const bool in = row <= q.mlast;
    const int64_t t = q.m0 + (in ? row : 0);
    const float f = in ? e.factor[t] : 0.0f;
    const float2 st = e.stat[t];
    const float there = e.target[t];
    const int64_t y = e.targets[t] - e.col0 - q.n0 - q.wn * W;
    const int hot = y >= 0 && y < W ? static_cast<int>(y) : -1;
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int c = 32 * j + 8 * (r / 4) + 4 * q.half + r % 4;
        float v = exp_below(acc[i][j][r], st.x) * st.y;
        v = f * (c == hot ? there : v);
        acc[i][j][r] = f == 0.0f || c >= inside ? 0.0f : v;
      }
    for (int term = 0; term < terms; ++term) {
      // bf16 terms, largest first: what is left goes to the next
      uint32_t u[C::FN][8];                                             // columns 2 k, 2 k + 1 of the lane's
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          u[j][k] = pack_bf16x2(acc[i][j][2 * k], acc[i][j][2 * k + 1]);
          acc[i][j][2 * k] -= __uint_as_float(u[j][k] << 16);
          acc[i][j][2 * k + 1] -= __uint_as_float(u[j][k] & 0xffff0000u);
        }
      if (term < e.terms_x) {
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int g = 0; g < 4; ++g)
            *reinterpret_cast<u32x2v*>(turn + q.r32 * kPitch + (32 * j + 8 * g + 4 * q.half) * 2) = u32x2v{u[j][2 * g], u[j][2 * g + 1]};
        wave_order();
        constexpr int kLanes = W / 8;                                   // to a row
#pragma unroll
        for (int k = 0; k < 32 * kLanes / 64; ++k) {
          const int lr = k * (64 / kLanes) + q.lane / kLanes, lc = q.lane % kLanes * 8;
          const u32x4v v = *reinterpret_cast<const u32x4v*>(turn + lr * kPitch + lc * 2);
          const int64_t rr = q.wm * (C::TM / C::WM) + 32 * i + lr, cc = q.n0 + q.wn * W + lc;
          if (rr <= q.mlast && cc < e.vp) *reinterpret_cast<u32x4v*>(e.dz + (q.m0 + rr) * e.pitch_x + static_cast<int64_t>(term) * e.vp + cc) = v;
        }
        wave_order();
      }
      if (term < e.terms_w) {
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t other = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(u[j][k]), 0xB1, 0xf, 0xf, true));   // lanes 1 0 3 2
            const int c = 32 * j + 8 * (k / 2) + 4 * q.half + 2 * (k % 2) + (odd ? 1 : 0);
            *reinterpret_cast<uint32_t*>(turn + c * kPitchT + (q.r32 >> 1) * 4) = __builtin_amdgcn_perm(u[j][k], other, pick);
          }
        wave_order();
#pragma unroll
        for (int k = 0; k < W * 4 / 64; ++k) {
          const int c = k * 16 + q.lane / 4, ch = q.lane % 4;
          const u32x4v v = *reinterpret_cast<const u32x4v*>(turn + c * kPitchT + ch * 16);
          const int64_t cc = q.wn * W + c, rr = q.m0 + q.wm * (C::TM / C::WM) + 32 * i + ch * 8;
          if (cc <= q.nlast && rr < e.tp) *reinterpret_cast<u32x4v*>(e.dz_t + (q.n0 + cc) * e.pitch_w + static_cast<int64_t>(term) * e.tp + rr) = v;
        }
        wave_order();
      }
    }
  }
}

// The same from a piece of kept logits: 64 rows x 128 columns per workgroup; HBM
// bound: 8192 x 32000 to a bf16 term of each 380 us (5.5 TB/s), 1021 x 129283 to
// one and three 290 (5.5).
__global__ void __launch_bounds__(256) ce_kept_grad_kernel(const CeGradArgs e, const float* z, int64_t pitch_z, int rows, int cols) {
  __shared__ uint32_t tile[kPackRows][kPackCols / 2 + 1];
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * kPackRows, c0 = static_cast<int64_t>(blockIdx.x) * kPackCols;
  const int cl = (threadIdx.x & 15) * 8, rl = threadIdx.x >> 4;
  const int64_t c = c0 + cl;
  float v[4][8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = r0 + rl + 16 * i;
    const bool in = t < rows && c < cols;
    f32x4v lo = {}, hi = {};
    if (in) {
      lo = *reinterpret_cast<const f32x4v*>(z + t * pitch_z + c);
      hi = *reinterpret_cast<const f32x4v*>(z + t * pitch_z + c + 4);
    }
    const float f = in ? e.factor[t] : 0.0f;
    const float2 st = in ? e.stat[t] : make_float2(0.0f, 0.0f);
    const float there = in ? e.target[t] : 0.0f;
    const int64_t y = in ? e.targets[t] - e.col0 - c : -1;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float x = exp_below(k < 4 ? lo[k] : hi[k - 4], st.x) * st.y;
      x = f * (k == y ? there : x);
      v[i][k] = f == 0.0f || c + k >= cols ? 0.0f : x;
    }
  }
  for (int term = 0; term < max(e.terms_x, e.terms_w); ++term) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = r0 + rl + 16 * i;
      const u32x4v h = {pack_bf16x2(v[i][0], v[i][1]), pack_bf16x2(v[i][2], v[i][3]), pack_bf16x2(v[i][4], v[i][5]), pack_bf16x2(v[i][6], v[i][7])};
      if (term < e.terms_x && t < rows && c < e.vp) *reinterpret_cast<u32x4v*>(e.dz + t * e.pitch_x + static_cast<int64_t>(term) * e.vp + c) = h;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        tile[rl + 16 * i][cl / 2 + k] = h[k];
        v[i][2 * k] -= __uint_as_float(h[k] << 16);
        v[i][2 * k + 1] -= __uint_as_float(h[k] & 0xffff0000u);
      }
    }
    if (term >= e.terms_w) continue;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int u = i * 256 + threadIdx.x, cc = u >> 3, r = (u & 7) * 8;
      if (c0 + cc < cols && r0 + r < e.tp)
        *reinterpret_cast<u32x4v*>(e.dz_t + (c0 + cc) * e.pitch_w + static_cast<int64_t>(term) * e.tp + r0 + r) = column8(tile, r, cc);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------ dx of few rows
// Parts of dz W where there are few rows: the weights' bytes are all there is to
// it, so they are read as they lie, along their rows, instead of as a transposed
// copy.  A lane loads 4 columns of 8 rows of W, and the matrix instruction takes
// those 8 as its contraction: the lanes' first columns are one operand, their
// second ones another.  A workgroup takes 128 columns and a share of the
// vocabulary, whose rows its waves take in turn, 64 at a time; the waves' sums
// meet in LDS in a fixed order.
//
// HBM bound: 4 x 128000 x 4096 178 us, 5.9 TB/s, 64 rows 286, where dz is half as
// much to load as W (the transposed copy alone takes 410, its product 230; all of
// the call 1104 to 696 and 1174 to 825 us).  128 rows in four blocks of 32 and two
// columns a lane took 598, no less than the copy and its product.
struct CeDxRowsArgs {
  const uint16_t* dz;           // [rows]: TERMS times vp, rows pitch_x apart
  const uint8_t* w;             // bf16, rows pitch_w bytes apart
  float* part;                  // [splits][rows][hp]
  int64_t pitch_x, pitch_w;
  int rows, cols, vp, hp;       // cols: the piece's rows of W
  int per;                      // rows of W to a split, a multiple of 256
  int accumulate;
};

template <int TB, int TERMS>
__global__ void __launch_bounds__(256, 2) ce_dx_rows_kernel(const CeDxRowsArgs e) {
  constexpr int NC = 4, kSums = TB * NC;
  constexpr int kSets = TERMS == 1 ? 4 : 2;                 // 16 rows of W each, on their way
  typedef uint32_t wvec __attribute__((ext_vector_type(2)));
  __shared__ f32x4v meet[2][kSums * 4][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r32 = lane & 31, half = lane >> 5;
  const int c0 = blockIdx.x * (32 * NC), c = min(c0 + r32 * NC, e.hp - NC);
  const int s0 = blockIdx.y * e.per, s1 = min(s0 + e.per, e.vp);
  f32x16v acc[TB][NC];
#pragma unroll
  for (int t = 0; t < TB; ++t)
#pragma unroll
    for (int j = 0; j < NC; ++j) acc[t][j] = f32x16v{};
  const uint8_t* wcol = e.w + static_cast<int64_t>(c) * 2;
  const uint16_t* zrow[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t) zrow[t] = e.dz + static_cast<int64_t>(min(32 * t + r32, e.rows - 1)) * e.pitch_x + 8 * half;
  wvec w[kSets][8];
  u32x4v z[kSets][TB][TERMS];
  // rows past the piece's last repeat it: dz is 0 there
  auto load = [&](int set, int v) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      w[set][i] = *reinterpret_cast<const wvec*>(wcol + static_cast<int64_t>(min(v + 8 * half + i, e.cols - 1)) * e.pitch_w);
#pragma unroll
    for (int t = 0; t < TB; ++t)
#pragma unroll
      for (int k = 0; k < TERMS; ++k) z[set][t][k] = *reinterpret_cast<const u32x4v*>(zrow[t] + static_cast<int64_t>(k) * e.vp + v);
  };
  auto add = [&](int set) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      u32x4v b;                                             // column j of the lane's, 8 rows
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = __builtin_amdgcn_perm(w[set][2 * i + 1][j / 2], w[set][2 * i][j / 2], j % 2 ? 0x07060302u : 0x05040100u);
#pragma unroll
      for (int k = 0; k < TERMS; ++k)
#pragma unroll
        for (int t = 0; t < TB; ++t) acc[t][j] = mma_bf16(b, z[set][t][k], acc[t][j]);
    }
  };
  // the wave's blocks of 64 rows, kSets times 16 of them in flight
  int v = s0 + wave * 64;
  if (v < s1) {
#pragma unroll
    for (int k = 0; k < kSets; ++k) load(k, v + 16 * k);
    for (;;) {
      const int next = v + 256;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        add(k % kSets);
        const int ahead = k + kSets < 4 ? v + 16 * (k + kSets) : next + 16 * (k + kSets - 4);
        if (k + kSets < 4 || next < s1) load(k % kSets, ahead);
      }
      if (next >= s1) break;
      v = next;
    }
  }
  // waves 2 and 3 to 0 and 1, then 1 to 0
#pragma unroll
  for (int step = 2; step >= 1; step >>= 1) {
    if (wave >= step && wave < 2 * step) {
#pragma unroll
      for (int q = 0; q < kSums; ++q)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x16v& a = acc[q / NC][q % NC];
          meet[wave - step][q * 4 + g][lane] = f32x4v{a[4 * g], a[4 * g + 1], a[4 * g + 2], a[4 * g + 3]};
        }
    }
    __syncthreads();
    if (wave < step) {
#pragma unroll
      for (int q = 0; q < kSums; ++q)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const f32x4v a = meet[wave][q * 4 + g][lane];
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[q / NC][q % NC][4 * g + k] += a[k];
        }
    }
    __syncthreads();
  }
  if (wave) return;
  // lane r32 has row 32 t + r32; element r of operand j is column NC (8 (r / 4) + 4 half + r % 4) + j
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    const int row = 32 * t + r32;
    if (row >= e.rows) continue;
    float* to = e.part + (static_cast<int64_t>(blockIdx.y) * e.rows + row) * e.hp;
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int h = c0 + NC * (8 * (r / 4) + 4 * half + r % 4);
      if (h >= e.hp) continue;
#pragma unroll
      for (int j = 0; j < NC; ++j) to[h + j] = e.accumulate ? to[h + j] + acc[t][j][r] : acc[t][j][r];
    }
  }
}

template <int TB>
hipError_t run_dx_rows(const CeDxRowsArgs& e, int terms, int splits, hipStream_t s) {
  const dim3 g(static_cast<uint32_t>((e.hp + 127) / 128), static_cast<uint32_t>(splits));
  if (terms == 1) ce_dx_rows_kernel<TB, 1><<<g, 256, 0, s>>>(e);
  else ce_dx_rows_kernel<TB, 3><<<g, 256, 0, s>>>(e);
  return hipGetLastError();
}

// dx = scale times the sum of the splits' parts (rows of `pitch`, a multiple of
// 4), 0 in rows that take no part: a workgroup per row and 1024 columns, as a
// single long row with 64 parts would keep one CU busy (84 x 4352 with 32 parts
// 66 us with a workgroup per row, 10 so).
template <typename T>
__global__ void __launch_bounds__(256) ce_finish_kernel(const float* part, int splits, int64_t stride, int64_t pitch, int hidden,
                                                        const float* scale, const float* factor, T* dx, int64_t ld) {
  const int64_t t = blockIdx.x;
  const int c = blockIdx.y * 1024 + threadIdx.x * 4;
  if (c >= hidden) return;
  const float f = factor[t] == 0.0f ? 0.0f : *scale;
  f32x4v v = {};
#pragma unroll 4
  for (int s = 0; s < splits; ++s) v += *reinterpret_cast<const f32x4v*>(part + s * stride + t * pitch + c);
#pragma unroll
  for (int k = 0; k < 4; ++k) v[k] = f == 0.0f ? 0.0f : v[k] * f;
  store4_out(dx + t * ld + c, v, hidden - c, 0);
}

// ------------------------------------------------------------ tiles
typedef TileCfgT<OpBf16, 64, 64, 2, 2, 7> Cfg64;
typedef TileCfgT<OpBf16, 64, 64, 2, 2, 5, true> Cfg64Sliced;
typedef TileCfgT<OpBf16, 128, 128, 2, 2, 5> Cfg128;
typedef TileCfgT<OpBf16, 256, 256, 2, 4, 5> Cfg256;

// Measured (see tile_us): 4096 x 4096 x 8192 takes 211 us in tiles of 256, 2048
// x 2048 x 8192 70 in tiles of 128, 1024 x 1024 x 8192 39 in tiles of 64 and 30 in
// sliced ones; 64 x 1024 x 8192 37 and 19, 64 x 1024 x 512 5.4 and 5.8, 64 x 32000 x
// 2048 22 and 28.
enum Tile { kTile64, kTile64Sliced, kTile128, kTile256, kTiles };
constexpr TileCost kCosts[kTiles] = {{64, 3, 4.5, 0.137, 0.108}, {64, 1, 5.6, 0.055, 0.10}, {128, 2, 7.0, 0.24, 0.222}, {256, 1, 10.0, 0.45, 0.765}};

// The quickest tile for a product, and how many workgroups should share each
// tile's contraction (their parts are written, and read by the pass that adds
// them, at 4 TB/s).
struct Choice {
  Tile tile;
  int splits;
};
Choice choose(int64_t m, int64_t n, int64_t stages, bool may_split) {
  Choice best{kTile64, 1};
  double least = 1e30;
  for (int t = 0; t < kTiles; ++t)
    for (int s = 1; s == 1 || (may_split && s <= 64 && stages >= 16 * s); s *= 2) {
      const double us = tile_us(kCosts[t], m, n, (stages + s - 1) / s, s) + (s - 1) * static_cast<double>(m) * n * 8 / 4e6;
      if (us < least) {
        least = us;
        best = {static_cast<Tile>(t), s};
      }
    }
  return best;
}

// f with the configuration of a tile.
template <class F>
hipError_t with(Tile t, F f) {
  switch (t) {
    case kTile256: return f(Cfg256{});
    case kTile128: return f(Cfg128{});
    case kTile64Sliced: return f(Cfg64Sliced{});
    default: return f(Cfg64{});
  }
}

template <typename T>
hipError_t store(Tile tile, const ProductArgs& p, const StoreArgs<T>& e, hipStream_t s) {
  return with(tile, [&](auto c) { return run_product_store<decltype(c), T>(p, e, s); });
}

// ------------------------------------------------------------ the plan
constexpr int64_t kDxRows = 64;                             // at most, for ce_dx_rows_kernel

// Pieces of the vocabulary, and the places of everything in the workspace.
struct Plan {
  int64_t hp, tp;              // hidden size and rows, padded to whole pairs of stages
  int64_t ph, pt;              // and how far apart rows of that length lie
  int64_t vf, vb;              // columns of a forward and of a backward piece
  int splits;                  // of the product for dx
  Tile tile_dx;
  bool dx_rows;                // which reads the weights along their rows
  int terms_x, terms_w;
  bool keep;                   // the logits stay
  bool keep_w;                 // so does the bf16 copy of the weights, where they are copied
  int64_t pz;                  // their rows' distance
  size_t part, stat, zt, factor, scale, x, w, x_t, w_t, z, dz, dz_t, dxp, total;
};

// Pieces of at most `most` columns, of about equal length, in whole tiles.
int64_t piece_of(int64_t vocab, int64_t most) {
  const int64_t n = (vocab + most - 1) / most;
  return std::min(up((vocab + n - 1) / n, 256), up(vocab, 256));
}

Plan make_plan(int64_t rows, int64_t hidden, int64_t vocab, int x_dt, int dw_dt, bool dx, bool dw) {
  Plan p{};
  p.hp = up(hidden, 64);
  p.tp = up(rows, 64);
  p.ph = apart(p.hp);
  p.pt = apart(p.tp);
  p.terms_x = dx ? terms_of(x_dt) : 0;
  p.terms_w = dw ? terms_of(dw_dt) : 0;
  // Of the workspace: dz and its transpose take up to 1 GiB for a piece, the
  // weights and their transpose up to 1 GiB each (8192 x 32000 x 512 in bf16 takes
  // 1.71 ms with a quarter of that for dz, 1.51 with half and 1.29 so; 1021 x
  // 129283 x 2045 with dw in fp32 3.69 with a quarter of that for weights, 3.40 so).
  // Logits that 4 GiB hold stay in fp32 between the statistics and dz, instead of
  // being multiplied again: 8192 x 32000 x 2048 4.04 to 3.36 ms, 8192 x 128256 x
  // 2048 15.8 to 13.1.  Where the product is quicker than that writing and
  // reading (x 256 1.12 and 1.08 ms, x 128 0.90 and 0.93), they stay only where
  // the last-level cache holds them.  Their rows are not spread over the channels as
  // the operands' are, which gains nothing here (8192 x 131072 x 256 4.47 ms either
  // way, 8192 x 32768 x 2048 2.95) and would pass the 4 GiB.
  const int64_t r = std::max<int64_t>(rows, 1), vocab_p = up(vocab, 64);
  const int64_t held = int64_t{1} << (hidden >= 256 ? 30 : 26);
  p.keep = (dx || dw) && vocab_p <= held && r <= held / vocab_p;
  const int64_t terms = std::max(p.terms_x + p.terms_w, 2);
  const int64_t by_w = (int64_t{1} << 29) / p.hp, by_z = (int64_t{1} << 29) / (terms * r);
  p.vb = piece_of(vocab, std::min(std::max(std::min(by_w, by_z) / 256 * 256, int64_t{1024}), int64_t{1} << 20));
  p.pz = vocab_p;
  // with gradients a copy of up to 1 GiB is made once, not once for each product
  p.keep_w = (dx || dw) && vocab <= (int64_t{1} << 29) / p.ph;
  p.vf = piece_of(vocab, std::max((int64_t{1} << 28) / std::max<int64_t>(rows, 1) / 256 * 256, int64_t{4096}));
  p.dx_rows = dx && rows <= kDxRows;
  if (p.dx_rows) {
    // some workgroups for every CU, but 1024 rows of weights at least to each
    const int64_t chunks = (p.hp + 127) / 128;
    p.splits = static_cast<int>(std::max<int64_t>(1, std::min({int64_t{64}, (1024 + chunks - 1) / chunks, p.vb / 1024})));
  } else {
    const Choice of_dx = choose(rows, hidden, p.vb / 32 * p.terms_x, true);
    p.splits = of_dx.splits;
    p.tile_dx = of_dx.tile;
  }
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at += (bytes + 255) / 256 * 256;
    return o;
  };
  const size_t t = static_cast<size_t>(rows);
  p.part = take(t * static_cast<size_t>(up(std::max(p.vf, p.vb), 256) / 64) * 8);
  p.stat = take(t * 8);
  p.zt = take(t * 4);
  p.factor = take(t * 4);
  p.scale = take(4);
  p.x = take(t * p.ph * 2);
  p.w = take(static_cast<size_t>(p.keep_w ? vocab : p.vb) * p.ph * 2);
  if (dw) p.x_t = take(static_cast<size_t>(hidden) * p.pt * 2);
  if (dx && !p.dx_rows) p.w_t = take(static_cast<size_t>(hidden) * apart(p.vb) * 2);
  if (p.keep) p.z = take(t * p.pz * 4);
  if (dx) p.dz = take(t * apart(p.vb * p.terms_x) * 2);
  if (dw) p.dz_t = take(static_cast<size_t>(p.vb) * apart(p.tp * p.terms_w) * 2);
  if (dx) p.dxp = take(static_cast<size_t>(p.splits) * t * p.hp * 4);
  p.total = rows ? at : 0;
  return p;
}

template <class C>
dim3 tiles_of(ProductArgs& p) {
  p.tiles_m = (p.m + C::TM - 1) / C::TM;
  p.tiles_n = (p.n + C::TN - 1) / C::TN;
  return dim3(static_cast<uint32_t>(static_cast<int64_t>(p.tiles_m) * p.tiles_n));
}

template <class C>
hipError_t run_stats(ProductArgs p, const CeStatsArgs& e, int& cols, hipStream_t s) {
  const dim3 g = tiles_of<C>(p);
  cols = p.tiles_n;
  ce_stats_kernel<C><<<g, C::kThreads, 0, s>>>(p, e);
  return hipGetLastError();
}

template <class C>
hipError_t run_grad(ProductArgs p, const CeGradArgs& e, hipStream_t s) {
  const dim3 g = tiles_of<C>(p);
  ce_grad_kernel<C><<<g, C::kThreads, 0, s>>>(p, e);
  return hipGetLastError();
}

}  // namespace

size_t linear_ce_workspace(int64_t rows, int64_t hidden, int64_t vocab, int x_dt, int dw_dt, bool dx, bool dw) {
  return make_plan(rows, hidden, vocab, x_dt, dw_dt, dx, dw).total;
}

#define MO_TRY(e)                          \
  do {                                     \
    const hipError_t err_ = (e);           \
    if (err_ != hipSuccess) return err_;   \
  } while (0)

hipError_t launch_linear_ce(const LinearCeArgs& a, void* ws, hipStream_t s) {
  if (a.rows == 0)                   // accumulating calls and those without dw do not come here
    return a.dw_dt == F32 ? run_product_zero(static_cast<float*>(a.dw), a.ld_dw, a.vocab, a.hidden, s)
                          : run_product_zero(static_cast<__bf16*>(a.dw), a.ld_dw, a.vocab, a.hidden, s);
  const bool want_dx = a.dx != nullptr, want_dw = a.dw != nullptr, grad = want_dx || want_dw;
  const Plan pl = make_plan(a.rows, a.hidden, a.vocab, a.x_dt, a.dw_dt, want_dx, want_dw);
  uint8_t* base = static_cast<uint8_t*>(ws);
  float2* part = reinterpret_cast<float2*>(base + pl.part);
  float2* stat = reinterpret_cast<float2*>(base + pl.stat);
  float* zt = reinterpret_cast<float*>(base + pl.zt);
  float* factor = reinterpret_cast<float*>(base + pl.factor);
  float* scale = reinterpret_cast<float*>(base + pl.scale);
  uint16_t* xb = reinterpret_cast<uint16_t*>(base + pl.x);
  uint16_t* wb = reinterpret_cast<uint16_t*>(base + pl.w);
  uint16_t* x_t = want_dw ? reinterpret_cast<uint16_t*>(base + pl.x_t) : nullptr;
  uint16_t* w_t = want_dx && !pl.dx_rows ? reinterpret_cast<uint16_t*>(base + pl.w_t) : nullptr;
  uint16_t* dz = want_dx ? reinterpret_cast<uint16_t*>(base + pl.dz) : nullptr;
  uint16_t* dz_t = want_dw ? reinterpret_cast<uint16_t*>(base + pl.dz_t) : nullptr;
  float* dxp = want_dx ? reinterpret_cast<float*>(base + pl.dxp) : nullptr;
  float* z = pl.keep ? reinterpret_cast<float*>(base + pl.z) : nullptr;

  // operands that the products can read in place
  auto plain = [&](const void* q, int dt, int64_t ld) {
    return dt == BF16 && a.hidden % 64 == 0 && ld % 8 == 0 && ld <= kCeMaxHidden && reinterpret_cast<uintptr_t>(q) % 16 == 0;
  };
  const bool plain_x = plain(a.x, a.x_dt, a.ldx), plain_w = plain(a.w, a.w_dt, a.ldw);
  const int esz_w = a.w_dt == F32 ? 4 : 2, esz_dw = a.dw_dt == F32 ? 4 : 2;

  const CeRows job{grad ? a.targets : nullptr, a.grad_loss, scale, a.rows};
  if (!plain_x || want_dw) MO_TRY(pack(a.x_dt, a.x, a.ldx, a.rows, a.hidden, plain_x ? nullptr : xb, pl.ph, x_t, pl.pt, job, s));
  else if (grad) MO_TRY(pack(a.x_dt, a.x, a.ldx, 0, 1, nullptr, 0, nullptr, 0, job, s));

  ProductArgs logits{};
  logits.a = static_cast<const uint8_t*>(plain_x ? a.x : xb);
  logits.pitch_a = static_cast<uint32_t>((plain_x ? a.ldx : pl.ph) * 2);
  logits.pitch_b = static_cast<uint32_t>((plain_w ? a.ldw : pl.ph) * 2);
  logits.m = a.rows;
  logits.stages = logits.stages_b = static_cast<int>(pl.hp / 32);
  logits.splits = 1;

  // weights as given, and as the products read them
  auto weights = [&](int64_t v0) { return static_cast<const uint8_t*>(a.w) + v0 * a.ldw * esz_w; };
  auto operand = [&](int64_t v0) {
    return plain_w ? weights(v0) : reinterpret_cast<const uint8_t*>(wb + (pl.keep_w ? v0 * pl.ph : 0));
  };
  const int64_t vf = plain_w || pl.keep_w ? pl.vf : pl.vb;
  const bool once = pl.keep && vf >= a.vocab && pl.vb >= a.vocab;      // one piece of weights, too: its transpose comes with it
  for (int64_t v0 = 0; v0 < a.vocab; v0 += vf) {
    const int v = static_cast<int>(std::min<int64_t>(vf, a.vocab - v0));
    if (!plain_w || (once && w_t))
      MO_TRY(pack(a.w_dt, weights(v0), a.ldw, v, a.hidden, plain_w ? nullptr : wb + (pl.keep_w ? v0 * pl.ph : 0), pl.ph, once ? w_t : nullptr,
                  apart(up(v, 64)), {}, s));
    logits.b = operand(v0);
    logits.n = v;
    const CeStatsArgs e{a.targets, v0, part, zt, z, pl.pz, pl.keep && worth_streaming(z, pl.pz, a.rows, a.vocab)};
    int cols;
    MO_TRY(with(choose(a.rows, v, logits.stages, false).tile, [&](auto c) { return run_stats<decltype(c)>(logits, e, cols, s); }));
    const bool wide = a.rows <= 2048 || cols > 256;
    const auto join = wide ? ce_join_kernel<256> : ce_join_kernel<16>;
    const int per = wide ? 1 : 16;
    join<<<(a.rows + per - 1) / per, 256, 0, s>>>(part, cols, a.rows, a.vocab, v0 == 0,
                                                    v0 + v >= a.vocab, a.targets, zt, stat, a.loss, a.grad_loss, scale, grad ? factor : nullptr);
    MO_TRY(hipGetLastError());
  }
  if (!grad) return hipSuccess;

  for (int64_t v0 = 0; v0 < a.vocab; v0 += pl.vb) {
    const int v = static_cast<int>(std::min<int64_t>(pl.vb, a.vocab - v0));
    const int64_t vp = up(v, 64), pv = apart(vp);
    const bool copied = !plain_w && pl.keep_w;                          // already there
    const bool need_w = (!pl.keep || pl.dx_rows) && !plain_w && !copied, need_w_t = w_t && !once;
    if (need_w || need_w_t)
      MO_TRY(copied ? pack(BF16, operand(v0), pl.ph, v, a.hidden, nullptr, 0, w_t, pv, {}, s)
                    : pack(a.w_dt, weights(v0), a.ldw, v, a.hidden, need_w ? wb : nullptr, pl.ph, need_w_t ? w_t : nullptr, pv, {}, s));
    const CeGradArgs e{a.targets, v0, stat, zt, factor, dz, dz_t, pl.terms_x, pl.terms_w, static_cast<int>(vp), static_cast<int>(pl.tp),
                       apart(vp * pl.terms_x), apart(pl.tp * pl.terms_w)};
    if (pl.keep) {
      const dim3 g(static_cast<uint32_t>((v + kPackCols - 1) / kPackCols), static_cast<uint32_t>((a.rows + kPackRows - 1) / kPackRows));
      ce_kept_grad_kernel<<<g, 256, 0, s>>>(e, z + v0, pl.pz, a.rows, v);
      MO_TRY(hipGetLastError());
    } else {
      logits.b = operand(v0);
      logits.n = v;
      MO_TRY(with(choose(a.rows, v, logits.stages, false).tile, [&](auto c) { return run_grad<decltype(c)>(logits, e, s); }));
    }
    if (want_dx && pl.dx_rows) {
      const CeDxRowsArgs r{dz, operand(v0), dxp, apart(vp * pl.terms_x), static_cast<int64_t>(logits.pitch_b), a.rows, v, static_cast<int>(vp),
                           static_cast<int>(pl.hp), static_cast<int>(up((vp + pl.splits - 1) / pl.splits, 256)), v0 > 0};
      MO_TRY(a.rows <= 32 ? run_dx_rows<1>(r, pl.terms_x, pl.splits, s) : run_dx_rows<2>(r, pl.terms_x, pl.splits, s));
    } else if (want_dx) {
      // a piece's terms lie side by side along the contraction
      ProductArgs p{};
      p.a = reinterpret_cast<const uint8_t*>(dz);
      p.b = reinterpret_cast<const uint8_t*>(w_t);
      p.pitch_a = static_cast<uint32_t>(apart(vp * pl.terms_x) * 2);
      p.pitch_b = static_cast<uint32_t>(pv * 2);
      p.m = a.rows;
      p.n = a.hidden;
      p.stages_b = static_cast<int>(vp / 32);
      p.stages = p.stages_b * pl.terms_x;
      p.splits = pl.splits;
      MO_TRY((store<float>(pl.tile_dx, p, {dxp, pl.hp, static_cast<int64_t>(a.rows) * pl.hp, v0 > 0, nullptr, 0}, s)));
    }
    if (want_dw) {
      ProductArgs p{};
      p.a = reinterpret_cast<const uint8_t*>(dz_t);
      p.b = reinterpret_cast<const uint8_t*>(x_t);
      p.pitch_a = static_cast<uint32_t>(apart(pl.tp * pl.terms_w) * 2);
      p.pitch_b = static_cast<uint32_t>(pl.pt * 2);
      p.m = v;
      p.n = a.hidden;
      p.stages_b = static_cast<int>(pl.tp / 32);
      p.stages = p.stages_b * pl.terms_w;
      p.splits = 1;
      const int stream_dw = a.dw_dt == F32 ? worth_streaming(static_cast<float*>(a.dw), a.ld_dw, a.vocab, a.hidden)
                                           : worth_streaming(static_cast<__bf16*>(a.dw), a.ld_dw, a.vocab, a.hidden);
      const Tile tile_dw = choose(v, a.hidden, p.stages, false).tile;
      uint8_t* out = static_cast<uint8_t*>(a.dw) + v0 * a.ld_dw * esz_dw;
      if (a.dw_dt == F32) MO_TRY((store<float>(tile_dw, p, {reinterpret_cast<float*>(out), a.ld_dw, 0, a.accumulate, scale, stream_dw}, s)));
      else MO_TRY((store<__bf16>(tile_dw, p, {reinterpret_cast<__bf16*>(out), a.ld_dw, 0, a.accumulate, scale, stream_dw}, s)));
    }
  }
  if (want_dx) {
    const int64_t n = static_cast<int64_t>(a.rows) * pl.hp;
    const dim3 g(static_cast<uint32_t>(a.rows), static_cast<uint32_t>((a.hidden + 1023) / 1024));
    if (a.x_dt == F32) ce_finish_kernel<float><<<g, 256, 0, s>>>(dxp, pl.splits, n, pl.hp, a.hidden, scale, factor, static_cast<float*>(a.dx), a.ld_dx);
    else ce_finish_kernel<__bf16><<<g, 256, 0, s>>>(dxp, pl.splits, n, pl.hp, a.hidden, scale, factor, static_cast<__bf16*>(a.dx), a.ld_dx);
    MO_TRY(hipGetLastError());
  }
  return hipSuccess;
}

}  // namespace mo
