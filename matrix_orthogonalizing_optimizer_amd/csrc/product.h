// What the matrix products that are staged through LDS share (gfx950): waits,
// direct-to-LDS requests from uniform addresses, stores of outputs.
#pragma once

#include "row_vec.h"

namespace mo {

// Waits until at most `kLeft` of this wave's loads are outstanding, and for
// its LDS reads.
template <int kLeft>
__device__ __forceinline__ void wait_loads() {
  static_assert(kLeft < 64, "the counter has 6 bits");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(waitcnt_vm(kLeft) & (kWaitLgkm0 | (63 & 15) | (3 << 14)));
  asm volatile("" ::: "memory");
}

// A wave-uniform address, said to be one.
__device__ __forceinline__ const uint8_t* uniform_ptr(const uint8_t* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u >> 32));
  return reinterpret_cast<const uint8_t*>(static_cast<uint64_t>(lo) | (static_cast<uint64_t>(hi) << 32));
}

// lds_dma16 to lds_base + kPlus.
template <int kPlus>
__device__ __forceinline__ void lds_dma16_at(const void* sbase, uint32_t voff, uint32_t lds_base) {
  asm volatile("s_add_u32 m0, %2, %3\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(voff), "s"(sbase), "s"(lds_base), "n"(kPlus)
               : "memory", "m0", "scc");
}

// The same from the lanes of `lanes` (a scalar), in a wave whose lanes are all
// active: from none it counts as a load that is done and touches no memory.
template <int kPlus>
__device__ __forceinline__ void lds_dma16_masked(const void* sbase, uint32_t voff, uint32_t lds_base, uint64_t lanes) {
  asm volatile("s_add_u32 m0, %2, %3\n\ts_mov_b64 exec, %4\n\tglobal_load_lds_dwordx4 %0, %1\n\ts_mov_b64 exec, -1"
               :
               : "v"(voff), "s"(sbase), "s"(lds_base), "n"(kPlus), "s"(lanes)
               : "memory", "m0", "scc");
}

template <typename T>
__device__ __forceinline__ void store_out(T* o, float v, int accumulate) {
  if (accumulate) v += to_f(*o);
  *o = static_cast<T>(v);
}

// Four consecutive outputs past the caches: for outputs that are larger than
// those, where keeping them would only evict what other tiles still read.
template <typename T>
__device__ __forceinline__ void stream4_out(T* o, f32x4v v) {
  if constexpr (sizeof(T) == 4) {
    __builtin_nontemporal_store(v, reinterpret_cast<f32x4u*>(o));
  } else {
    typedef uint32_t u32x2u2 __attribute__((ext_vector_type(2), aligned(2)));
    __builtin_nontemporal_store(u32x2u2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])}, reinterpret_cast<u32x2u2*>(o));
  }
}

// Four consecutive outputs as they are, n of them inside.
template <typename T>
__device__ __forceinline__ f32x4v load4_out(const T* o, int n) {
  f32x4v v = {};
  if (n >= 4) {
    if constexpr (sizeof(T) == 4) {
      v = *reinterpret_cast<const f32x4u*>(o);
    } else {
      typedef uint32_t u32x2u2 __attribute__((ext_vector_type(2), aligned(2)));
      const u32x2u2 w = *reinterpret_cast<const u32x2u2*>(o);
      v = f32x4v{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u), __uint_as_float(w[1] << 16),
                 __uint_as_float(w[1] & 0xffff0000u)};
    }
  } else {
#pragma unroll
    for (int k = 0; k < 3; ++k)
      if (k < n) v[k] = to_f(o[k]);
  }
  return v;
}

// Four consecutive outputs, n of them inside.
template <typename T>
__device__ __forceinline__ void store4_out(T* o, f32x4v v, int n, int accumulate) {
  if (n >= 4) {
    if constexpr (sizeof(T) == 4) {
      if (accumulate) v += *reinterpret_cast<const f32x4u*>(o);
      *reinterpret_cast<f32x4u*>(o) = v;
    } else {
      typedef uint32_t u32x2u2 __attribute__((ext_vector_type(2), aligned(2)));
      if (accumulate) {
        const u32x2u2 w = *reinterpret_cast<const u32x2u2*>(o);
        v += f32x4v{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u), __uint_as_float(w[1] << 16),
                    __uint_as_float(w[1] & 0xffff0000u)};
      }
      *reinterpret_cast<u32x2u2*>(o) = u32x2u2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < n) store_out(o + k, v[k], accumulate);
  }
}

}  // namespace mo
