// 8-bit matrices (e4m3 with a power-of-two scale for each block of 128):
// quantisation, reading back, and the product of two images on the matrix
// cores (gfx950).  Layout and rounding are those of include/muon.h.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "fp8_internal.h"
#include "mo_internal.h"
#include "tile_product.h"

namespace mo {

namespace {

typedef short i16x2v __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2v __attribute__((ext_vector_type(2)));

// Scale byte of a block from the bits of its largest magnitude a = 1.m 2^E:
// the least e with a <= 448 2^e is E - 8, or E - 7 where 1.m passes 1.75 (448 =
// 1.75 2^8); 255 for a NaN or an infinity.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const uint32_t e = (amax_bits + 0x1fffffu) >> 23;      // carries into the exponent exactly above 1.75
  return e > 8u ? e - 8u : 0u;
}

// Under the largest scale, 2^120, the next number after 240 2^120 is 2^128, past
// fp32: what would round there stays below it.
__device__ __forceinline__ float clip(float x) { return __builtin_amdgcn_fmed3f(x, -0x1.ep127f, 0x1.ep127f); }

// Four codes from four elements under the scale, element 0 lowest.
__device__ __forceinline__ uint32_t fp8_codes4(float a, float b, float c, float d, float s) {
  i16x2v r = {0, 0};
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, clip(a), clip(b), s, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, clip(c), clip(d), s, true);
  return __builtin_bit_cast(uint32_t, r);
}
template <typename T>
__device__ __forceinline__ u32x2v fp8_codes(const Oct<T>& o, float s) {
  return u32x2v{fp8_codes4(o.get(0), o.get(1), o.get(2), o.get(3), s), fp8_codes4(o.get(4), o.get(5), o.get(6), o.get(7), s)};
}

// Largest of 16 neighbouring lanes.
__device__ __forceinline__ uint32_t row16_max(uint32_t x) {
  x = quad_max(x);
  x = max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x124, 0xf, 0xf, true)));   // rotated by 4
  return max(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x128, 0xf, 0xf, true)));   // by 8
}

}  // namespace

// Row images: a thread takes 8 columns, 16 neighbours a block, so that a wave
// reads and writes whole lines.  Four eighths per thread are in flight before
// the first is used.  HBM bound: 3 (bf16) or 5 (fp32) bytes an element; 8192 x
// 8192 bf16 in 35 us, 5.8 TB/s.
constexpr int kOctsPerThread = 4;
template <typename T, int G>
__global__ void __launch_bounds__(256) fp8_quant_rows_kernel(const Fp8QuantArgs<G> a) {
  const Fp8QuantItem& it = a.item[G == 1 ? 0 : find_item(a, blockIdx.x)];
  const T* src = static_cast<const T*>(it.src);
  const uint32_t nb = static_cast<uint32_t>(fp8_blocks(it.cols)), sp = static_cast<uint32_t>(fp8_scale_pitch(it.cols));
  const int64_t octs = static_cast<int64_t>(it.rows) * nb * 16;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) - it.tile0) * (256 * kOctsPerThread) + threadIdx.x;
  Oct<T> o[kOctsPerThread];
  int64_t row[kOctsPerThread];
  uint32_t col8[kOctsPerThread];
#pragma unroll
  for (int i = 0; i < kOctsPerThread; ++i) {
    const int64_t u = first + i * 256;
    o[i].clear();
    row[i] = -1;
    if (u < octs) {
      row[i] = octs <= 0xffffffffll ? static_cast<uint32_t>(u) / (nb * 16) : u / (nb * 16);
      col8[i] = static_cast<uint32_t>(u - row[i] * (nb * 16));
      const int64_t left = it.cols - static_cast<int64_t>(col8[i]) * 8;
      if (left > 0) o[i].load(src + row[i] * it.ld + static_cast<int64_t>(col8[i]) * 8, static_cast<int>(min(left, int64_t{8})));
    }
  }
#pragma unroll
  for (int i = 0; i < kOctsPerThread; ++i) {
    const uint32_t byte = scale_byte(row16_max(o[i].amax()));       // whole groups of 16 are inside or outside
    u32x2v c = fp8_codes(o[i], scale_of(byte));
    if (byte == 255u) c = u32x2v{0u, 0u};
    if (row[i] < 0) continue;
    *reinterpret_cast<u32x2v*>(it.codes + (row[i] * nb * 16 + col8[i]) * 8) = c;
    if ((col8[i] & 15) == 0) {
      uint8_t* s = it.scales + row[i] * sp;
      const uint32_t b = col8[i] / 16;
      s[b] = static_cast<uint8_t>(byte);
      if (b == nb - 1)
        for (uint32_t p = nb; p < sp; ++p) s[p] = 0;
    }
  }
}

// 128 x 128 elements per workgroup of 4 waves: the image of the matrix, of its
// transpose, or both from one reading.  A wave takes 32 rows, lane l the
// columns 8 (l & 15) .. + 7 of rows 8 (l / 16) .. + 7.  A row's block is then 16
// neighbours; a column's lies in lanes l, l ^ 16, l ^ 32, l ^ 48 of the four
// waves, whose maxima meet in LDS, as does the whole tile's for a square image.
// The transpose's codes go through LDS so that they leave as whole 128-byte
// lines.  HBM bound: 24 fp32 matrices of 2048 x 1408, both images, 104 us (4.0
// TB/s: the images' lines lie a row apart); 8192 x 5632 bf16 36 us (5.1 TB/s).
constexpr int kTile = 128, kRun = 16;
template <typename T, int G>
__global__ void __launch_bounds__(256) fp8_quant_tiles_kernel(const Fp8QuantArgs<G> a) {
  __shared__ uint32_t codes[kTile][33];            // 128 bytes a column, and a dword against bank conflicts
  __shared__ uint32_t most[4][kTile];
  const Fp8QuantItem& it = a.item[G == 1 ? 0 : find_item(a, blockIdx.x)];
  const T* src = static_cast<const T*>(it.src);
  // each XCD (workgroup index mod 8) takes runs of kRun neighbours, so that
  // lines that two tiles share meet in its L2 (the last ones as they come)
  const int64_t tiles_c = (it.cols + kTile - 1) / kTile;
  const int64_t tiles = (it.rows + kTile - 1) / kTile * tiles_c;
  const uint32_t b = blockIdx.x - static_cast<uint32_t>(it.tile0), g = b / (8 * kRun) * (8 * kRun);
  const int64_t tile = g + 8 * kRun <= tiles ? g + (b % 8) * kRun + (b - g) / 8 : b;
  const int64_t row0 = tile / tiles_c * kTile, col0 = tile % tiles_c * kTile;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int rl = wave * 32 + (lane >> 4) * 8, cl = (lane & 15) * 8;           // the lane's place in the tile
  const int64_t r0 = row0 + rl, c0 = col0 + cl;
  const int left_c = static_cast<int>(min(int64_t{8}, it.cols - c0)), left_r = static_cast<int>(min(int64_t{8}, it.rows - r0));

  Oct<T> o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    o[i].clear();
    if (i < left_r && left_c > 0) o[i].load(src + (r0 + i) * it.ld + c0, left_c);
  }
  const int64_t nb = fp8_blocks(it.cols), sp = fp8_scale_pitch(it.cols), nbt = fp8_blocks(it.rows), spt = fp8_scale_pitch(it.rows);
  const int64_t br = col0 / kTile, bt = row0 / kTile;                          // block of the rows, of the columns
  uint32_t whole = 0;
  if (a.square) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, o[i].amax());
    m = row16_max(m);
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16, 64)));
    m = max(m, lane_xor32(m));
    if (lane == 0) most[wave][0] = m;
    __syncthreads();
    whole = scale_byte(max(max(most[0][0], most[1][0]), max(most[2][0], most[3][0])));
  } else if (it.codes_t) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, o[i].bits(j));
      m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16, 64)));
      m = max(m, lane_xor32(m));
      if (lane < 16) most[wave][cl + j] = m;
    }
    __syncthreads();
  }
  if (it.codes) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t byte = a.square ? whole : scale_byte(row16_max(o[i].amax()));
      u32x2v c = fp8_codes(o[i], scale_of(byte));
      if (byte == 255u) c = u32x2v{0u, 0u};
      const int64_t r = r0 + i;
      if (i < left_r) {
        *reinterpret_cast<u32x2v*>(it.codes + r * nb * kTile + c0) = c;
        if ((lane & 15) == 0) {
          it.scales[r * sp + br] = static_cast<uint8_t>(byte);
          if (br == nb - 1)
            for (int64_t p = nb; p < sp; ++p) it.scales[r * sp + p] = 0;
        }
      }
    }
  }
  if (!it.codes_t) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int c = cl + j;
    const uint32_t byte = a.square ? whole : scale_byte(max(max(most[0][c], most[1][c]), max(most[2][c], most[3][c])));
    const float s = scale_of(byte);
    const uint32_t lo = fp8_codes4(o[0].get(j), o[1].get(j), o[2].get(j), o[3].get(j), s);
    const uint32_t hi = fp8_codes4(o[4].get(j), o[5].get(j), o[6].get(j), o[7].get(j), s);
    codes[c][rl / 4] = byte == 255u ? 0u : lo;
    codes[c][rl / 4 + 1] = byte == 255u ? 0u : hi;
    if (wave == 0 && lane < 16 && col0 + c < it.cols) {
      it.scales_t[(col0 + c) * spt + bt] = static_cast<uint8_t>(byte);
      if (bt == nbt - 1)
        for (int64_t p = nbt; p < spt; ++p) it.scales_t[(col0 + c) * spt + p] = 0;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int u = i * 256 + threadIdx.x, c = u >> 3, k = u & 7;       // 16 bytes k of column c
    if (col0 + c < it.cols) {
      const u32x4v v = {codes[c][k * 4], codes[c][k * 4 + 1], codes[c][k * 4 + 2], codes[c][k * 4 + 3]};
      *reinterpret_cast<u32x4v*>(it.codes_t + ((col0 + c) * nbt + bt) * kTile + k * 16) = v;
    }
  }
}

int64_t fp8_quant_tiles(int64_t rows, int64_t cols, bool tiles) {
  if (tiles) return ((rows + kTile - 1) / kTile) * ((cols + kTile - 1) / kTile);
  const int64_t octs = rows * fp8_blocks(cols) * 16;
  return (octs + 256 * kOctsPerThread - 1) / (256 * kOctsPerThread);
}

template <int G>
hipError_t launch_fp8_quant(int dt, bool tiles, const Fp8QuantArgs<G>& a, int64_t count, hipStream_t s) {
  const dim3 g(static_cast<uint32_t>(count));
  if (tiles) {
    if (dt == F32) fp8_quant_tiles_kernel<float, G><<<g, 256, 0, s>>>(a);
    else fp8_quant_tiles_kernel<__bf16, G><<<g, 256, 0, s>>>(a);
  } else {
    if (dt == F32) fp8_quant_rows_kernel<float, G><<<g, 256, 0, s>>>(a);
    else fp8_quant_rows_kernel<__bf16, G><<<g, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}
template hipError_t launch_fp8_quant<1>(int, bool, const Fp8QuantArgs<1>&, int64_t, hipStream_t);
template hipError_t launch_fp8_quant<kFp8Group>(int, bool, const Fp8QuantArgs<kFp8Group>&, int64_t, hipStream_t);

// Reading back: a thread takes 16 bytes of output at a time (4 or 8 columns),
// consecutive threads consecutive ones.  HBM bound: 48 images of 2048 x 1408 to
// bf16 69 us, 6.0 TB/s.
template <typename T>
__device__ __forceinline__ void store_unit(T* p, u32x2v codes, uint32_t byte, int n);
template <>
__device__ __forceinline__ void store_unit<float>(float* p, u32x2v codes, uint32_t byte, int n) {
  const float s = scale_of(byte), nan = __uint_as_float(0x7fc00000u);
  const f32x2v a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes[0], s, false), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes[0], s, true);
  f32x4v v = {a[0], a[1], b[0], b[1]};
  if (byte == 255u) v = f32x4v{nan, nan, nan, nan};
  if (n >= 4) {
    *reinterpret_cast<f32x4u*>(p) = v;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < n) p[j] = v[j];
  }
}
template <>
__device__ __forceinline__ void store_unit<__bf16>(__bf16* p, u32x2v codes, uint32_t byte, int n) {
  const float s = scale_of(byte);
  u32x4v v;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const f32x2v a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes[j], s, false), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(codes[j], s, true);
    v[2 * j] = pack_bf16x2(a[0], a[1]);
    v[2 * j + 1] = pack_bf16x2(b[0], b[1]);
  }
  if (byte == 255u) v = u32x4v{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
  if (n >= 8) {
    *reinterpret_cast<u32x4u2*>(p) = v;
  } else {
    uint16_t* q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) q[j] = static_cast<uint16_t>(v[j / 2] >> (16 * (j & 1)));
  }
}

constexpr int kUnitsPerThread = 4;
template <typename T, int G>
__global__ void __launch_bounds__(256) fp8_dequant_kernel(const Fp8DequantArgs<G> a) {
  constexpr int kCols = 16 / sizeof(T), kPerBlock = 128 / kCols;
  const Fp8DequantItem& it = a.item[G == 1 ? 0 : find_item(a, blockIdx.x)];
  const uint32_t nb = static_cast<uint32_t>(fp8_blocks(it.cols)), sp = static_cast<uint32_t>(fp8_scale_pitch(it.cols));
  const uint32_t per_row = nb * kPerBlock;
  const int64_t units = static_cast<int64_t>(it.rows) * per_row;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) - it.tile0) * (256 * kUnitsPerThread) + threadIdx.x;
  u32x2v codes[kUnitsPerThread];
  uint32_t byte[kUnitsPerThread];
  int64_t at[kUnitsPerThread];
  int left[kUnitsPerThread];
#pragma unroll
  for (int i = 0; i < kUnitsPerThread; ++i) {
    const int64_t u = first + i * 256;
    left[i] = 0;
    if (u < units) {
      const int64_t row = units <= 0xffffffffll ? static_cast<uint32_t>(u) / per_row : u / per_row;
      const uint32_t unit = static_cast<uint32_t>(u - row * per_row);
      if constexpr (kCols == 4) codes[i] = u32x2v{reinterpret_cast<const uint32_t*>(it.codes)[u], 0u};
      else codes[i] = reinterpret_cast<const u32x2v*>(it.codes)[u];
      byte[i] = it.scales[row * sp + unit / kPerBlock];
      left[i] = static_cast<int>(max(it.cols - static_cast<int64_t>(unit) * kCols, int64_t{0}));
      at[i] = row * it.cols + static_cast<int64_t>(unit) * kCols;
    }
  }
#pragma unroll
  for (int i = 0; i < kUnitsPerThread; ++i)
    if (left[i] > 0) store_unit(static_cast<T*>(it.dst) + at[i], codes[i], byte[i], left[i]);
}

int64_t fp8_dequant_tiles(int dt, int64_t rows, int64_t cols) {
  const int64_t units = rows * fp8_blocks(cols) * (dt == F32 ? 32 : 16);
  return (units + 256 * kUnitsPerThread - 1) / (256 * kUnitsPerThread);
}

template <int G>
hipError_t launch_fp8_dequant(int dt, const Fp8DequantArgs<G>& a, int64_t tiles, hipStream_t s) {
  const dim3 g(static_cast<uint32_t>(tiles));
  if (dt == F32) fp8_dequant_kernel<float, G><<<g, 256, 0, s>>>(a);
  else fp8_dequant_kernel<__bf16, G><<<g, 256, 0, s>>>(a);
  return hipGetLastError();
}
template hipError_t launch_fp8_dequant<1>(int, const Fp8DequantArgs<1>&, int64_t, hipStream_t);
template hipError_t launch_fp8_dequant<kFp8Group>(int, const Fp8DequantArgs<kFp8Group>&, int64_t, hipStream_t);

// ------------------------------------------------------------------ product
// A grid holds fewer than 2^32 threads, whichever kernel is taken.
bool fp8_matmul_fits(int64_t m, int64_t n) { return ((m + 63) / 64) * ((n + 63) / 64) <= int64_t{0xffffffff} / 256; }

template <class C, typename T>
static hipError_t run(const ProductArgs& p, const Fp8MatmulArgs& a, hipStream_t s) {
  return run_product_store<C, T>(p, {static_cast<T*>(a.out), a.ldo, 0, a.accumulate, nullptr, worth_streaming(static_cast<T*>(a.out), a.ldo, a.m, a.n)}, s);
}

// Measured (see tile_us), in tiles of 64, 128 and 256: 1024 x 1024 x 8192 24, 2048
// x 2048 x 8192 40, 4096 x 4096 x 8192 104 us from codes; in sliced tiles of 64 and
// in tiles of 128 and 256 22, 72 and 200 decoded.
constexpr TileCost kCostCodes[3] = {{64, 2, 4.5, 0.16, 0.13}, {128, 2, 8.0, 0.25, 0.22}, {256, 1, 12.0, 0.60, 0.705}};
constexpr TileCost kCostExact[3] = {{64, 1, 5.5, 0.12, 0.124}, {128, 2, 8.0, 0.50, 0.40}, {256, 1, 14.0, 1.10, 1.40}};
// Few tiles of a long contraction are bound by the waits of a wave that adds all
// of it up: sliced, 64 x 1024 x 8192 takes 12.3 instead of 22.3 us and 1024 x 1024 x
// 8192 17.2 instead of 24.2; 64 x 1024 x 1024 8.2 instead of 6.0, 64 x 28672 x 8192
// 42 instead of 39.  Decoded, each wave then decodes its own codes, half as many in
// all, and 64 x 64 tiles are always sliced (1024 x 1024 x 8192 22 instead of 43).
constexpr TileCost kCostSliced = {64, 1, 6.4, 0.04, 0.10};

template <class Op, typename T>
static hipError_t run_op(const TileCost (&cost)[3], const ProductArgs& p, const Fp8MatmulArgs& a, hipStream_t s) {
  double us[3];
  for (int i = 0; i < 3; ++i) us[i] = tile_us(cost[i], a.m, a.n, p.stages, 1);
  bool sliced = Op::kDecoded;
  if (const double v = tile_us(kCostSliced, a.m, a.n, p.stages, 1); !Op::kDecoded && v < us[0]) {
    sliced = true;
    us[0] = v;
  }
  if (us[2] <= us[1] && us[2] <= us[0]) return run<TileCfgT<Op, 256, 256, 2, 4, 5>, T>(p, a, s);
  if (us[1] <= us[0]) return run<TileCfgT<Op, 128, 128, 2, 2, 5>, T>(p, a, s);
  if constexpr (!Op::kDecoded)
    if (!sliced) return run<TileCfgT<Op, 64, 64, 2, 2, 7>, T>(p, a, s);
  return run<TileCfgT<Op, 64, 64, 2, 2, 5, true>, T>(p, a, s);
}

hipError_t launch_fp8_matmul(int out_dt, const Fp8MatmulArgs& a, hipStream_t s) {
  if (a.nb == 0)                     // accumulating calls do not come here
    return out_dt == F32 ? run_product_zero(static_cast<float*>(a.out), a.ldo, a.m, a.n, s)
                         : run_product_zero(static_cast<__bf16*>(a.out), a.ldo, a.m, a.n, s);
  ProductArgs p{};
  p.a = a.a;
  p.b = a.b;
  p.sa = a.sa;
  p.sb = a.sb;
  p.sp = static_cast<uint32_t>(a.sp);
  p.pitch_a = p.pitch_b = static_cast<uint32_t>(a.nb) * 128u;
  p.m = a.m;
  p.n = a.n;
  p.stages = p.stages_b = 2 * a.nb;
  p.splits = 1;
  return out_dt == F32 ? run_op<OpFp8Exact, float>(kCostExact, p, a, s) : run_op<OpFp8, __bf16>(kCostCodes, p, a, s);
}

}  // namespace mo
