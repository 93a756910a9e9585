// The product of two matrices whose rows both run along the contraction, a
// tile of outputs per workgroup (gfx950): 8-bit codes with a scale byte per
// 128 on the scaled matrix instruction, or bf16.  What becomes of a tile's sums
// is the caller's: stored, or turned into a softmax's statistics or gradient.
#pragma once

#include "product.h"

namespace mo {

typedef float f32x16v __attribute__((ext_vector_type(16)));
typedef int i32x8v __attribute__((ext_vector_type(8)));

// Both operands have rows of whole stages of 64 bytes (32 bf16 or 64 codes).
struct ProductArgs {
  const uint8_t *a, *b;          // 16-byte aligned
  uint32_t pitch_a, pitch_b;     // bytes from a row to the next
  const uint8_t *sa, *sb;        // 8-bit: scale bytes of each row
  uint32_t sp;                   // bytes of a row of them
  int m, n;
  int stages;                    // of 64 bytes of a row, even
  int stages_b;                  // of b's rows, which then repeat (even): b = [b b ..] for a = [hi lo ..]
  int tiles_m, tiles_n;
  int splits;                    // workgroups that share a tile's contraction
};

// 32 x 32 outputs, 64 bytes of each row: lane l gives row l & 31 and two
// chunks of 16 bytes, at 32 (l / 32) bytes of the stage.  (Any order of the
// contraction is right as long as both operands agree.)
struct OpBf16 {
  static constexpr bool kScaled = false;
  static __device__ __forceinline__ f32x16v mma(const u32x4v (&a)[2], const u32x4v (&b)[2], f32x16v c, uint32_t, uint32_t) {
    c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a[0]), __builtin_bit_cast(bf16x8_t, b[0]), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a[1]), __builtin_bit_cast(bf16x8_t, b[1]), c, 0, 0, 0);
  }
};
struct OpFp8 {
  static constexpr bool kScaled = true;
  static __device__ __forceinline__ i32x8v codes(const u32x4v (&x)[2]) {
    return i32x8v{static_cast<int>(x[0][0]), static_cast<int>(x[0][1]), static_cast<int>(x[0][2]), static_cast<int>(x[0][3]),
                  static_cast<int>(x[1][0]), static_cast<int>(x[1][1]), static_cast<int>(x[1][2]), static_cast<int>(x[1][3])};
  }
  static __device__ __forceinline__ f32x16v mma(const u32x4v (&a)[2], const u32x4v (&b)[2], f32x16v c, uint32_t sa, uint32_t sb) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(codes(a), codes(b), c, 0, 0, 0, static_cast<int>(sa), 0, static_cast<int>(sb));
  }
};

template <class OpT, int TMv, int TNv, int WMv, int WNv>
struct TileCfgT {
  typedef OpT Op;
  static constexpr int TM = TMv, TN = TNv, WM = WMv, WN = WNv, NW = WM * WN;
  static constexpr int FM = TM / (32 * WM), FN = TN / (32 * WN);
  static constexpr int kThreads = 64 * NW;
  // LDS: what the epilogues need to turn 32 rows per wave
  static constexpr int kTurnPitch = TN / WN * 4 + 16;
  static constexpr int kLds = NW * 32 * kTurnPitch;
};

// Where a workgroup's tile is: its first row and column, the last ones inside
// it that exist, the wave's and the lane's place.
struct TilePlace {
  int tm, tn, wm, wn, lane, r32, half, mlast, nlast;
  int64_t m0, n0;
};

template <class C>
__device__ __forceinline__ TilePlace tile_place(const ProductArgs& p) {
  TilePlace q;
  q.lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  q.wm = wave / C::WN;
  q.wn = wave % C::WN;
  q.r32 = q.lane & 31;
  q.half = q.lane >> 5;
  q.tm = blockIdx.x % p.tiles_m;
  q.tn = blockIdx.x / p.tiles_m;
  q.m0 = static_cast<int64_t>(q.tm) * C::TM;
  q.n0 = static_cast<int64_t>(q.tn) * C::TN;
  q.mlast = static_cast<int>(min(static_cast<int64_t>(C::TM), p.m - q.m0)) - 1;
  q.nlast = static_cast<int>(min(static_cast<int64_t>(C::TN), p.n - q.n0)) - 1;
  return q;
}

// The stages of split `s`, in pairs.
__device__ __forceinline__ void split_range(const ProductArgs& p, int s, int& k0, int& k1) {
  const int pairs = p.stages / 2, per = (pairs + p.splits - 1) / p.splits;
  k0 = 2 * min(s * per, pairs);
  k1 = 2 * min((s + 1) * per, pairs);
}

// acc[i][j]: lane (r32, half), element 4 e + k of the tile's row
// wm TM / WM + 32 i + r32, column wn TN / WN + 32 j + 8 e + 4 half + k.
// Straight from memory: every wave reads its own rows of both operands.
template <class C>
__device__ __forceinline__ void tile_sums(const ProductArgs& p, const TilePlace& q, uint8_t*, f32x16v (&acc)[C::FM][C::FN]) {
  typedef typename C::Op Op;
  const uint8_t *a[C::FM], *b[C::FN], *sa[C::FM], *sb[C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
    const int64_t r = q.m0 + min(q.wm * (C::TM / C::WM) + 32 * i + q.r32, q.mlast);   // rows past the end: the last again
    a[i] = p.a + r * p.pitch_a + q.half * 32;
    if constexpr (Op::kScaled) sa[i] = p.sa + r * p.sp;
  }
#pragma unroll
  for (int j = 0; j < C::FN; ++j) {
    const int64_t r = q.n0 + min(q.wn * (C::TN / C::WN) + 32 * j + q.r32, q.nlast);
    b[j] = p.b + r * p.pitch_b + q.half * 32;
    if constexpr (Op::kScaled) sb[j] = p.sb + r * p.sp;
  }
  int k0, k1;
  split_range(p, blockIdx.y, k0, k1);
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) acc[i][j] = f32x16v{};
  for (int t = k0; t < k1; ++t) {
    u32x4v av[C::FM][2], bv[C::FN][2];
    uint32_t as[C::FM] = {}, bs[C::FN] = {};
    const int64_t ka = static_cast<int64_t>(t) * 64, kb = static_cast<int64_t>(t % p.stages_b) * 64;
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      av[i][0] = *reinterpret_cast<const u32x4v*>(a[i] + ka);
      av[i][1] = *reinterpret_cast<const u32x4v*>(a[i] + ka + 16);
      if constexpr (Op::kScaled) as[i] = sa[i][t >> 1];
    }
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      bv[j][0] = *reinterpret_cast<const u32x4v*>(b[j] + kb);
      bv[j][1] = *reinterpret_cast<const u32x4v*>(b[j] + kb + 16);
      if constexpr (Op::kScaled) bs[j] = sb[j][t >> 1];
    }
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j) acc[i][j] = Op::mma(bv[j], av[i], acc[i][j], bs[j], as[i]);
  }
}

// Stores the sums, times a factor in device memory where one is given.  Each
// wave turns 32 rows at a time through LDS of its own, so that rows leave as
// whole lines; the 16 bytes of padding per row spread 16 rows over all banks.
template <typename T>
struct StoreArgs {
  T* out;
  int64_t ldo, split_stride;     // elements from a split's outputs to the next split's
  int accumulate;
  const float* scale;            // or null
};
template <class C, typename T>
__device__ __forceinline__ void tile_store(const StoreArgs<T>& e, const TilePlace& q, uint8_t* smem, const f32x16v (&acc)[C::FM][C::FN]) {
  constexpr int W = C::TN / C::WN, kPitch = C::kTurnPitch, kLanes = W / 4;       // columns, and lanes to a row
  uint8_t* turn = smem + (q.wm * C::WN + q.wn) * 32 * kPitch;
  T* out = e.out + blockIdx.y * e.split_stride + q.m0 * e.ldo + q.n0;
  const float f = e.scale ? *e.scale : 1.0f;
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g)
        *reinterpret_cast<f32x4v*>(turn + q.r32 * kPitch + (32 * j + 8 * g + 4 * q.half) * 4) =
            f32x4v{acc[i][j][4 * g] * f, acc[i][j][4 * g + 1] * f, acc[i][j][4 * g + 2] * f, acc[i][j][4 * g + 3] * f};
#pragma unroll
    for (int k = 0; k < 32 * kLanes / 64; ++k) {
      const int row = k * (64 / kLanes) + q.lane / kLanes, col = q.lane % kLanes * 4;
      const f32x4v v = *reinterpret_cast<const f32x4v*>(turn + row * kPitch + col * 4);
      const int r = q.wm * (C::TM / C::WM) + 32 * i + row, c = q.wn * W + col;
      if (r <= q.mlast) store4_out(out + r * e.ldo + c, v, q.nlast + 1 - c, e.accumulate);
    }
  }
}

// The product of nothing: rows of zeros.
template <typename T>
__global__ void __launch_bounds__(256) product_zero_kernel(T* out, int64_t ldo, int64_t rows, int64_t cols) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int64_t c = threadIdx.x; c < cols; c += 256) out[r * ldo + c] = static_cast<T>(0.0f);
}
template <typename T>
hipError_t run_product_zero(T* out, int64_t ldo, int64_t rows, int64_t cols, hipStream_t s) {
  product_zero_kernel<T><<<static_cast<uint32_t>(rows < 4096 ? rows : 4096), 256, 0, s>>>(out, ldo, rows, cols);
  return hipGetLastError();
}

template <class C, typename T>
__global__ void __launch_bounds__(C::kThreads) product_store_kernel(const ProductArgs p, const StoreArgs<T> e) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[C::kLds];
  const TilePlace q = tile_place<C>(p);
  f32x16v acc[C::FM][C::FN];
  tile_sums<C>(p, q, smem, acc);
  tile_store<C, T>(e, q, smem, acc);
}

template <class C, typename T>
hipError_t run_product_store(ProductArgs p, const StoreArgs<T>& e, hipStream_t s) {
  p.tiles_m = (p.m + C::TM - 1) / C::TM;
  p.tiles_n = (p.n + C::TN - 1) / C::TN;
  const dim3 g(static_cast<uint32_t>(static_cast<int64_t>(p.tiles_m) * p.tiles_n), static_cast<uint32_t>(p.splits));
  product_store_kernel<C, T><<<g, C::kThreads, 0, s>>>(p, e);
  return hipGetLastError();
}

}  // namespace mo
