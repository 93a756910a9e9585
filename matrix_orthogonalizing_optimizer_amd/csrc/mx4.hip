// MX4: quantisation to microscaled 4-bit images, reading back, and the
// product of two images on the matrix cores (gfx950).  Layout and rounding
// are those of include/muon.h.
#include "mo_internal.h"
#include "mx4_internal.h"

namespace mo {

namespace {

typedef uint32_t u32x4v __attribute__((ext_vector_type(4)));
typedef int i32x8v __attribute__((ext_vector_type(8)));
typedef float f32x4v __attribute__((ext_vector_type(4)));

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f<__bf16>(__bf16 v) { return static_cast<float>(v); }

// Scale byte of a block from the bits of its largest magnitude: the biased
// exponent less 2 (the list's largest binade starts at 4 = 2^2), 255 for a
// NaN or an infinity.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const uint32_t e = amax_bits >> 23;
  return e > 2u ? e - 2u : 0u;
}

// One block of 32 values, `n` of them present, `step` elements apart.
template <typename T>
__device__ void quant_block(const T* p, int64_t step, int n, uint8_t* codes, uint8_t* scale) {
  float v[32];
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    v[j] = j < n ? to_f(p[j * step]) : 0.0f;
    amax = max(amax, __float_as_uint(v[j]) & 0x7fffffffu);
  }
  const uint32_t sb = scale_byte(amax);
  u32x4v q = {0u, 0u, 0u, 0u};
  if (sb != 255u) {
    const float s = __uint_as_float(sb << 23);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t r = 0;
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[8 * w + 0], v[8 * w + 1], s, 0);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[8 * w + 2], v[8 * w + 3], s, 1);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[8 * w + 4], v[8 * w + 5], s, 2);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[8 * w + 6], v[8 * w + 7], s, 3);
      q[w] = r;
    }
  }
  *reinterpret_cast<u32x4v*>(codes) = q;
  *scale = static_cast<uint8_t>(sb);
}

}  // namespace

// One thread per block: the row image's blocks first, then the transpose's.
// The thread of a row's last block also clears the row's scale padding.
template <typename T>
__global__ void __launch_bounds__(256) mx4_quant_kernel(const Mx4QuantArgs a) {
  int i = 0;
  while (i + 1 < a.count && static_cast<int64_t>(blockIdx.x) >= a.item[i + 1].tile0) ++i;
  const Mx4QuantItem& it = a.item[i];
  const T* src = static_cast<const T*>(it.src);
  int64_t t = (static_cast<int64_t>(blockIdx.x) - it.tile0) * 256 + threadIdx.x;
  const int64_t nb = mx4_blocks(it.cols), nbt = mx4_blocks(it.rows);
  if (it.codes) {
    if (t < it.rows * nb) {
      const int64_t r = t / nb, b = t % nb;
      const int64_t sp = mx4_scale_pitch(it.cols);
      quant_block(src + r * it.ld + b * 32, 1, static_cast<int>(min(int64_t{32}, it.cols - b * 32)),
                  it.codes + (r * nb + b) * 16, it.scales + r * sp + b);
      if (b == nb - 1)
        for (int64_t p = nb; p < sp; ++p) it.scales[r * sp + p] = 0;
      return;
    }
    t -= it.rows * nb;
  }
  if (it.codes_t && t < it.cols * nbt) {
    const int64_t c = t % it.cols, b = t / it.cols;
    const int64_t sp = mx4_scale_pitch(it.rows);
    quant_block(src + b * 32 * it.ld + c, it.ld, static_cast<int>(min(int64_t{32}, it.rows - b * 32)),
                it.codes_t + (c * nbt + b) * 16, it.scales_t + c * sp + b);
    if (b == nbt - 1)
      for (int64_t p = nbt; p < sp; ++p) it.scales_t[c * sp + p] = 0;
  }
}

int64_t mx4_quant_tiles(int64_t rows, int64_t cols, bool row_image, bool col_image) {
  const int64_t t = (row_image ? rows * mx4_blocks(cols) : 0) + (col_image ? cols * mx4_blocks(rows) : 0);
  return (t + 255) / 256;
}

hipError_t launch_mx4_quant(int dt, const Mx4QuantArgs& a, int64_t tiles, hipStream_t s) {
  const dim3 g(static_cast<uint32_t>(tiles));
  if (dt == F32) mx4_quant_kernel<float><<<g, 256, 0, s>>>(a);
  else mx4_quant_kernel<__bf16><<<g, 256, 0, s>>>(a);
  return hipGetLastError();
}

// Value of a code: sign, two exponent bits, one mantissa bit.
__device__ __forceinline__ float code_value(uint32_t c) {
  const uint32_t e = (c >> 1) & 3u, m = c & 1u;
  const float v = e ? __uint_as_float(((e + 126u) << 23) | (m << 22)) : 0.5f * static_cast<float>(m);
  return (c & 8u) ? -v : v;
}

// 2^(byte - 127); NaN for 255.  Byte 0 is the subnormal 2^-127.
__device__ __forceinline__ float scale_value(uint32_t sb) {
  return sb == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float(sb ? sb << 23 : 0x00400000u);
}

template <typename T>
__global__ void __launch_bounds__(256) mx4_dequant_kernel(const Mx4DequantArgs a) {
  int i = 0;
  while (i + 1 < a.count && static_cast<int64_t>(blockIdx.x) >= a.item[i + 1].tile0) ++i;
  const Mx4DequantItem& it = a.item[i];
  const int64_t nb = mx4_blocks(it.cols), sp = mx4_scale_pitch(it.cols);
  const int64_t t = (static_cast<int64_t>(blockIdx.x) - it.tile0) * 256 + threadIdx.x;
  if (t >= it.rows * nb) return;
  const int64_t r = t / nb, b = t % nb;
  const float s = scale_value(it.scales[r * sp + b]);
  T* dst = static_cast<T*>(it.dst) + r * it.cols + b * 32;
  const int n = static_cast<int>(min(int64_t{32}, it.cols - b * 32));
  for (int j = 0; j < n; ++j) {
    const uint32_t c = it.codes[(r * nb + b) * 16 + j / 2] >> (4 * (j & 1));
    dst[j] = static_cast<T>(code_value(c & 15u) * s);
  }
}

int64_t mx4_dequant_tiles(int64_t rows, int64_t cols) { return (rows * mx4_blocks(cols) + 255) / 256; }

hipError_t launch_mx4_dequant(int dt, const Mx4DequantArgs& a, int64_t tiles, hipStream_t s) {
  const dim3 g(static_cast<uint32_t>(tiles));
  if (dt == F32) mx4_dequant_kernel<float><<<g, 256, 0, s>>>(a);
  else mx4_dequant_kernel<__bf16><<<g, 256, 0, s>>>(a);
  return hipGetLastError();
}

// C = A B^T, one wave per 32 x 32 outputs (2 x 2 tiles of 16 x 16), four
// waves per workgroup.  The scaled 16 x 16 x 128 instruction takes from lane
// l the 32 codes and the scale byte of row l % 16, block l / 16 of a step.
template <typename T>
__global__ void __launch_bounds__(256) mx4_matmul_kernel(const Mx4MatmulArgs p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * 64 + (wave >> 1) * 32;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 64 + (wave & 1) * 32;
  const int r16 = lane & 15, kb = lane >> 4;
  const uint8_t *ac[2], *as[2], *bc[2], *bs[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    // rows past the end read the last row; their products are not stored
    const int64_t ar = min(m0 + 16 * i + r16, static_cast<int64_t>(p.m) - 1);
    const int64_t br = min(n0 + 16 * i + r16, static_cast<int64_t>(p.n) - 1);
    ac[i] = p.a + ar * p.nb * 16;
    as[i] = p.sa + ar * p.sp;
    bc[i] = p.b + br * p.nb * 16;
    bs[i] = p.sb + br * p.sp;
  }
  f32x4v acc[2][2] = {};
  for (int k = 0; k < p.nb; k += 4) {
    const int b = k + kb;
    i32x8v av[2] = {}, bv[2] = {};
    int asv[2] = {}, bsv[2] = {};
    if (b < p.nb) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const u32x4v x = *reinterpret_cast<const u32x4v*>(ac[i] + static_cast<int64_t>(b) * 16);
        const u32x4v y = *reinterpret_cast<const u32x4v*>(bc[i] + static_cast<int64_t>(b) * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          av[i][j] = static_cast<int>(x[j]);
          bv[i][j] = static_cast<int>(y[j]);
        }
        asv[i] = as[i][b];
        bsv[i] = bs[i][b];
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av[i], bv[j], acc[i][j], 4, 4, 0, asv[i], 0, bsv[j]);
  }
  T* out = static_cast<T*>(p.out);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t r = m0 + 16 * i + 4 * kb + q, c = n0 + 16 * j + r16;
        if (r < p.m && c < p.n) {
          T* o = out + r * p.ldo + c;
          float v = acc[i][j][q];
          if (p.accumulate) v += to_f(*o);
          *o = static_cast<T>(v);
        }
      }
}

hipError_t launch_mx4_matmul(int out_dt, const Mx4MatmulArgs& a, hipStream_t s) {
  const dim3 g((a.n + 63) / 64, (a.m + 63) / 64);
  if (out_dt == F32) mx4_matmul_kernel<float><<<g, 256, 0, s>>>(a);
  else mx4_matmul_kernel<__bf16><<<g, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace mo
