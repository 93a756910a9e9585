// Eight consecutive elements of a row in registers, and the block scales of the
// low-bit images that are made from them (gfx950).
#pragma once

#include "ns_common.h"

namespace mo {

typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
typedef float f32x4v __attribute__((ext_vector_type(4)));

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__bf16>(__bf16 v) { return static_cast<float>(v); }

// Sixteen bytes, aligned to the element only: rows may start anywhere, and the
// hardware's unaligned access costs less than peeling.
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x4u2 __attribute__((ext_vector_type(4), aligned(2)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
typedef float f32x2v __attribute__((ext_vector_type(2)));

// Eight consecutive elements of a row.
template <typename T> struct Oct;
template <> struct Oct<float> {
  f32x4v lo, hi;
  __device__ __forceinline__ void load(const float* p, int n) {        // n > 0 present, the others 0
    if (n >= 8) {
      lo = *reinterpret_cast<const f32x4u*>(p);
      hi = *reinterpret_cast<const f32x4u*>(p + 4);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        lo[j] = j < n ? p[j] : 0.0f;
        hi[j] = j + 4 < n ? p[j + 4] : 0.0f;
      }
    }
  }
  __device__ __forceinline__ void clear() { lo = hi = f32x4v{0.0f, 0.0f, 0.0f, 0.0f}; }
  __device__ __forceinline__ float get(int j) const { return j < 4 ? lo[j] : hi[j - 4]; }
  __device__ __forceinline__ uint32_t bits(int j) const { return __float_as_uint(get(j)) & 0x7fffffffu; }
  // bits of the largest magnitude
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, bits(j));
    return m;
  }
};
template <> struct Oct<__bf16> {
  u32x4v v;
  __device__ __forceinline__ void load(const __bf16* p, int n) {
    if (n >= 8) {
      v = *reinterpret_cast<const u32x4u2*>(p);
    } else {
      const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = (2 * j < n ? q[2 * j] : 0u) | (2 * j + 1 < n ? static_cast<uint32_t>(q[2 * j + 1]) << 16 : 0u);
    }
  }
  __device__ __forceinline__ void clear() { v = u32x4v{0u, 0u, 0u, 0u}; }
  __device__ __forceinline__ bf16x2v pair(int i) const {
    const uint32_t w = v[i];             // a bit cast of the vector's element itself reads element 0
    return __builtin_bit_cast(bf16x2v, w);
  }
  __device__ __forceinline__ float get(int j) const {
    return __uint_as_float((j & 1) ? (v[j / 2] & 0xffff0000u) : (v[j / 2] << 16));
  }
  __device__ __forceinline__ uint32_t bits(int j) const { return __float_as_uint(get(j)) & 0x7fffffffu; }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, bits(j));
    return m;
  }
};

// The scale of a block as the conversions take it: only its exponent counts,
// and an exponent of 0 means 2^-127.
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// Largest of a quad of lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0xB1, 0xf, 0xf, true)));   // lanes 1 0 3 2
  return max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x4E, 0xf, 0xf, true)));   // lanes 2 3 0 1
}

// The matrix that workgroup `b` belongs to: the last whose first one is not
// past it.
template <typename A>
__device__ __forceinline__ int find_item(const A& a, int64_t b) {
  int lo = 0, hi = a.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.item[mid].tile0 <= b) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace mo
