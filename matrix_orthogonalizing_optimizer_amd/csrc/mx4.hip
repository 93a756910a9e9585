// MX4: quantisation to microscaled 4-bit images, reading back, and the
// product of two images on the matrix cores (gfx950).  Layout and rounding
// are those of include/muon.h.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "mo_internal.h"
#include "mx4_internal.h"
#include "product.h"

namespace mo {

namespace {

typedef int i32x8v __attribute__((ext_vector_type(8)));

// Scale byte of a block from the bits of its largest magnitude: the biased
// exponent less 2 (the list's largest binade starts at 4 = 2^2), 255 for a
// NaN or an infinity.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return 255u;
  const uint32_t e = amax_bits >> 23;
  return e > 2u ? e - 2u : 0u;
}

// The eight codes, element 0 lowest.
__device__ __forceinline__ uint32_t fp4_codes(const Oct<float>& o, float s) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, o.lo[0], o.lo[1], s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, o.lo[2], o.lo[3], s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, o.hi[0], o.hi[1], s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, o.hi[2], o.hi[3], s, 3);
}
__device__ __forceinline__ uint32_t fp4_codes(const Oct<__bf16>& o, float s) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, o.pair(0), s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, o.pair(1), s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, o.pair(2), s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, o.pair(3), s, 3);
}

// Codes of the lane's eighth of a row's block, whose scale byte it also gives:
// the four lanes of a quad share a block.
template <typename T>
__device__ __forceinline__ uint32_t row_codes(const Oct<T>& o, uint32_t& byte) {
  byte = scale_byte(quad_max(o.amax()));
  const uint32_t c = fp4_codes(o, scale_of(byte));
  return byte == 255u ? 0u : c;
}

}  // namespace

// Row images: a thread takes eighths of blocks (8 columns), consecutive
// threads consecutive ones, so that a wave reads and writes whole lines.  HBM
// bound: 2.53 (bf16) or 4.53 (fp32) bytes an element.  8192 x 8192: bf16 28 us,
// fp32 51 us, 6.0 TB/s (a large copy reaches 5.4); a block per thread, which
// strides over lines, took three times as long.  Four eighths per thread are
// in flight before the first is used.
constexpr int kOctsPerThread = 4;
template <typename T, int G>
__global__ void __launch_bounds__(256) mx4_quant_rows_kernel(const Mx4QuantArgs<G> a) {
  const Mx4QuantItem& it = a.item[G == 1 ? 0 : find_item(a, blockIdx.x)];
  const T* src = static_cast<const T*>(it.src);
  const uint32_t nb = static_cast<uint32_t>(mx4_blocks(it.cols)), sp = static_cast<uint32_t>(mx4_scale_pitch(it.cols));
  const int64_t octs = static_cast<int64_t>(it.rows) * nb * 4;
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
      row[i] = octs <= 0xffffffffll ? static_cast<uint32_t>(u) / (nb * 4) : u / (nb * 4);
      col8[i] = static_cast<uint32_t>(u - row[i] * (nb * 4));
      const int left = it.cols - static_cast<int>(col8[i]) * 8;
      if (left > 0) o[i].load(src + row[i] * it.ld + col8[i] * 8, left);
    }
  }
#pragma unroll
  for (int i = 0; i < kOctsPerThread; ++i) {
    uint32_t byte;
    const uint32_t c = row_codes(o[i], byte);       // whole quads are inside or outside
    if (row[i] < 0) continue;
    *reinterpret_cast<uint32_t*>(it.codes + (row[i] * nb * 4 + col8[i]) * 4) = c;
    if ((col8[i] & 3) == 0) {
      uint8_t* s = it.scales + row[i] * sp;
      const uint32_t b = col8[i] / 4;
      s[b] = static_cast<uint8_t>(byte);
      if (b == nb - 1)
        for (uint32_t p = nb; p < sp; ++p) s[p] = 0;
    }
  }
}

// Images of the transpose (and, with codes given, of the matrix itself) from
// one reading: a workgroup of 8 waves takes 256 rows x 128 columns, a wave 32
// rows, lane l the columns 8 (l & 15) .. + 7 of rows 8 (l / 16) .. + 7.  A
// column's block then lies in 4 lanes of a wave (l, l ^ 16, l ^ 32, l ^ 48),
// each with 8 consecutive codes of it, and a row's block in 4 neighbours.  The
// columns' codes go through LDS so that they leave as whole 128-byte lines.
// HBM bound: 8192 x 8192 bf16 29 us for the transpose alone, 39 us with both
// (3.06 bytes an element, 5.2 TB/s); fp32 53 and 70 us.  Two workgroups of 8
// waves fill a CU.
constexpr int kColTileRows = 256, kColTileCols = 128, kRun = 16;
template <typename T, int G>
__global__ void __launch_bounds__(512, 4) mx4_quant_cols_kernel(const Mx4QuantArgs<G> a) {
  __shared__ uint32_t codes[kColTileCols][33];     // 128 bytes a column, and a dword against bank conflicts
  __shared__ __attribute__((aligned(8))) uint8_t bytes[kColTileCols][8];
  const Mx4QuantItem& it = a.item[G == 1 ? 0 : find_item(a, blockIdx.x)];
  const T* src = static_cast<const T*>(it.src);
  // each XCD (workgroup index mod 8) takes runs of kRun neighbours, so that
  // lines that two tiles share meet in its L2 (the last ones as they come):
  // 8192 x 28672 bf16, both images, 185 to 171 us; whole matrices in eight
  // ranges 168, but fp32 8192 x 8192 77 instead of 70
  const int64_t tiles_c = (it.cols + kColTileCols - 1) / kColTileCols;
  const int64_t tiles = (it.rows + kColTileRows - 1) / kColTileRows * tiles_c;
  const uint32_t b = blockIdx.x - static_cast<uint32_t>(it.tile0), g = b / (8 * kRun) * (8 * kRun);
  const int64_t tile = g + 8 * kRun <= tiles ? g + (b % 8) * kRun + (b - g) / 8 : b;
  const int64_t row0 = tile / tiles_c * kColTileRows, col0 = tile % tiles_c * kColTileCols;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t r0 = row0 + wave * 32 + (lane >> 4) * 8, c0 = col0 + (lane & 15) * 8;
  const int left_c = static_cast<int>(min(int64_t{8}, it.cols - c0)), left_r = static_cast<int>(min(int64_t{8}, it.rows - r0));

  Oct<T> o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    o[i].clear();
    if (i < left_r && left_c > 0) o[i].load(src + (r0 + i) * it.ld + c0, left_c);
  }
  if (it.codes) {
    const int64_t nb = mx4_blocks(it.cols), sp = mx4_scale_pitch(it.cols);
    const int64_t b = c0 / 32;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t byte;
      const uint32_t c = row_codes(o[i], byte);
      const int64_t r = r0 + i;
      if (i < left_r && b < nb) {
        *reinterpret_cast<uint32_t*>(it.codes + r * nb * 16 + c0 / 2) = c;
        if ((lane & 3) == 0) {
          it.scales[r * sp + b] = static_cast<uint8_t>(byte);
          if (b == nb - 1)
            for (int64_t p = nb; p < sp; ++p) it.scales[r * sp + p] = 0;
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, o[i].bits(j));
    m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16, 64)));
    m = max(m, lane_xor32(m));
    const uint32_t byte = scale_byte(m);
    const float s = scale_of(byte);
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, o[0].get(j), o[1].get(j), s, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, o[2].get(j), o[3].get(j), s, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, o[4].get(j), o[5].get(j), s, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, o[6].get(j), o[7].get(j), s, 3);
    const int c = (lane & 15) * 8 + j;
    codes[c][wave * 4 + (lane >> 4)] = byte == 255u ? 0u : r;
    if (lane < 16) bytes[c][wave] = static_cast<uint8_t>(byte);
  }
  __syncthreads();
  const int64_t nbt = mx4_blocks(it.rows), spt = mx4_scale_pitch(it.rows), b0 = row0 / 32;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int u = i * 512 + threadIdx.x, c = u >> 3, b = u & 7;       // block b of column c
    if (col0 + c < it.cols && b0 + b < nbt) {
      u32x4v v;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = codes[c][b * 4 + k];
      *reinterpret_cast<u32x4v*>(it.codes_t + ((col0 + c) * nbt + b0 + b) * 16) = v;
    }
  }
  if (threadIdx.x < kColTileCols * 2) {
    // scale bytes past the last block come from rows that are not there: zero
    const int c = threadIdx.x >> 1, d = (threadIdx.x & 1) * 4;
    if (col0 + c < it.cols && b0 + d < spt)
      *reinterpret_cast<uint32_t*>(it.scales_t + (col0 + c) * spt + b0 + d) = *reinterpret_cast<const uint32_t*>(&bytes[c][d]);
  }
}

int64_t mx4_quant_tiles(int64_t rows, int64_t cols, bool cols_image) {
  if (cols_image) return ((rows + kColTileRows - 1) / kColTileRows) * ((cols + kColTileCols - 1) / kColTileCols);
  const int64_t octs = rows * mx4_blocks(cols) * 4;
  return (octs + 256 * kOctsPerThread - 1) / (256 * kOctsPerThread);
}

template <int G>
hipError_t launch_mx4_quant(int dt, bool cols_image, const Mx4QuantArgs<G>& a, int64_t tiles, hipStream_t s) {
  const dim3 g(static_cast<uint32_t>(tiles));
  if (cols_image) {
    if (dt == F32) mx4_quant_cols_kernel<float, G><<<g, 512, 0, s>>>(a);
    else mx4_quant_cols_kernel<__bf16, G><<<g, 512, 0, s>>>(a);
  } else {
    if (dt == F32) mx4_quant_rows_kernel<float, G><<<g, 256, 0, s>>>(a);
    else mx4_quant_rows_kernel<__bf16, G><<<g, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}
template hipError_t launch_mx4_quant<1>(int, bool, const Mx4QuantArgs<1>&, int64_t, hipStream_t);
template hipError_t launch_mx4_quant<kMx4Group>(int, bool, const Mx4QuantArgs<kMx4Group>&, int64_t, hipStream_t);

// Reading back: a thread takes 16 bytes of output at a time (4 or 8 columns),
// consecutive threads consecutive ones.  HBM bound: 8192 x 8192 to bf16 27 us,
// 6.3 TB/s, to fp32 65 us, 4.7 TB/s (80 us with 32 bytes a thread, whose two
// stores touch every line twice).
template <typename T>
__device__ __forceinline__ void store_unit(T* p, uint32_t codes, uint32_t byte, int n);
template <>
__device__ __forceinline__ void store_unit<float>(float* p, uint32_t codes, uint32_t byte, int n) {
  const float s = scale_of(byte), nan = __uint_as_float(0x7fc00000u);
  const f32x2v a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, s, 1);
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
__device__ __forceinline__ void store_unit<__bf16>(__bf16* p, uint32_t codes, uint32_t byte, int n) {
  const float s = scale_of(byte);
  u32x4v v = {__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 0)),
              __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 1)),
              __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 2)),
              __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 3))};
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
__global__ void __launch_bounds__(256) mx4_dequant_kernel(const Mx4DequantArgs<G> a) {
  constexpr int kCols = 16 / sizeof(T), kPerBlock = 32 / kCols;
  typedef std::conditional_t<sizeof(T) == 4, uint16_t, uint32_t> code_t;
  const Mx4DequantItem& it = a.item[G == 1 ? 0 : find_item(a, blockIdx.x)];
  const uint32_t nb = static_cast<uint32_t>(mx4_blocks(it.cols)), sp = static_cast<uint32_t>(mx4_scale_pitch(it.cols));
  const uint32_t per_row = nb * kPerBlock;
  const int64_t units = static_cast<int64_t>(it.rows) * per_row;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) - it.tile0) * (256 * kUnitsPerThread) + threadIdx.x;
  uint32_t codes[kUnitsPerThread], byte[kUnitsPerThread];
  int64_t at[kUnitsPerThread];
  int left[kUnitsPerThread];
#pragma unroll
  for (int i = 0; i < kUnitsPerThread; ++i) {
    const int64_t u = first + i * 256;
    left[i] = 0;
    if (u < units) {
      const int64_t row = units <= 0xffffffffll ? static_cast<uint32_t>(u) / per_row : u / per_row;
      const uint32_t unit = static_cast<uint32_t>(u - row * per_row);
      codes[i] = reinterpret_cast<const code_t*>(it.codes)[u];
      byte[i] = it.scales[row * sp + unit / kPerBlock];
      left[i] = it.cols - static_cast<int>(unit * kCols);
      at[i] = row * it.cols + unit * kCols;
    }
  }
#pragma unroll
  for (int i = 0; i < kUnitsPerThread; ++i)
    if (left[i] > 0) store_unit(static_cast<T*>(it.dst) + at[i], codes[i], byte[i], left[i]);
}

int64_t mx4_dequant_tiles(int dt, int64_t rows, int64_t cols) {
  const int64_t units = rows * mx4_blocks(cols) * (dt == F32 ? 8 : 4);
  return (units + 256 * kUnitsPerThread - 1) / (256 * kUnitsPerThread);
}

template <int G>
hipError_t launch_mx4_dequant(int dt, const Mx4DequantArgs<G>& a, int64_t tiles, hipStream_t s) {
  const dim3 g(static_cast<uint32_t>(tiles));
  if (dt == F32) mx4_dequant_kernel<float, G><<<g, 256, 0, s>>>(a);
  else mx4_dequant_kernel<__bf16, G><<<g, 256, 0, s>>>(a);
  return hipGetLastError();
}
template hipError_t launch_mx4_dequant<1>(int, const Mx4DequantArgs<1>&, int64_t, hipStream_t);
template hipError_t launch_mx4_dequant<kMx4Group>(int, const Mx4DequantArgs<kMx4Group>&, int64_t, hipStream_t);

// ------------------------------------------------------------------ product
// C = A B^T on the scaled matrix instruction, whose operands are 32 codes and
// one scale byte per lane.  Three kernels, chosen at the end of this file:
//  * tile: TM x TN outputs per workgroup, both operands staged through LDS;
//  * skinny (few rows of A): B streamed once from memory into registers;
//  * direct (short contractions): both operands straight from memory.
typedef float f32x16v __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4a4 __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ i32x8v codes8(u32x4v x) {
  return i32x8v{static_cast<int>(x[0]), static_cast<int>(x[1]), static_cast<int>(x[2]), static_cast<int>(x[3]), 0, 0, 0, 0};
}

// Byte `kSel` of each scale operand belongs to the lane's block.
template <int kSel>
__device__ __forceinline__ f32x16v mfma32(u32x4v a, u32x4v b, f32x16v c, uint32_t sa, uint32_t sb) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(codes8(a), codes8(b), c, 4, 4, kSel, static_cast<int>(sa), kSel,
                                                         static_cast<int>(sb));
}

// Tile kernel.  The contraction runs in stages of 4 blocks (128 columns):
// two instructions per output fragment, lanes 0..31 of a wave taking the
// stage's first two blocks and lanes 32..63 the others (any order of blocks
// is right as long as A and B agree).  LDS holds NST stages of both operands
// and their scale dwords, filled by loads that bypass the registers:
//   * scale bytes come for 16 stages at a time (64 bytes of a row): a request
//     costs a cache line's lookup and transfer per row however little of the
//     line it takes (4 bytes a row and stage cost 40% of the kernel's time, 16
//     bytes for four stages 13%);
//   * a row of a stage is 4 chunks of 16 bytes, stored at chunk ^ ((row / 4)
//     & 3): the 16 rows that a 16-byte read serves at a time then touch each
//     of the 64 banks once;
//   * at the second step of stage t the wave waits for its requests of stage
//     t + 1, the workgroup meets, and stage t's place is requested again for
//     stage t + NST while the first fragments of t + 1 are read.  Products,
//     reads and requests are interleaved one by one.
// Blocks past the end load the last block's codes under zero scale bytes in
// both operands: 2^-254 of a value of at most 36 is zero in fp32.
//
// 8192 x 28672 x 8192, operands quantised from normal values: 0.95 to 1.08 ms
// by box, 3.6 to 4.0 PFLOP/s.  A loop of nothing but this instruction runs at
// 6.1 to 6.6 on random codes, at the clock that the power limit leaves, and at
// 9.9 on zero codes.  8192^3 takes 220 us with zero codes (5.0 PFLOP/s), 282
// with normal values and 335 with random codes: the power limit costs a
// quarter, and even without it the matrix cores wait half of the time, though
// neither LDS nor the cache path is full: with one wave per SIMD and no second
// workgroup, nothing covers the wait at each stage's barrier, nor the first
// requests and the stores of a tile.  The larger the tile, the fewer bytes each
// product takes from the caches (64 bytes a clock and CU): 256 x 256 with four
// waves of 128 x 128 outputs, one workgroup to a CU, takes half of that path's
// time; two workgroups of 128 x 256 took three quarters of it and 14% longer.
// Eight waves in the 256 tile read twice the LDS bytes per product (6% longer).
// Rings of six and ten stages for the 64 tile, and bands of 2, 8 and 16 tile
// rows, gain nothing.
constexpr int kStageRow = 64;          // bytes of a row in one stage

template <int TM, int TN, int WM, int WN, int NST, typename T>
__global__ void __launch_bounds__(64 * WM * WN, TM * TN / (WM * WN) >= 16384 ? 1 : 2) mx4_tile_kernel(const Mx4MatmulArgs p) {
  constexpr int NW = WM * WN, FM = TM / (32 * WM), FN = TN / (32 * WN);
  constexpr int DA = TM / (16 * NW), DB = TN / (16 * NW);      // code requests of a wave and stage
  constexpr int DPW = DA + DB;
  constexpr int kStage = (TM + TN) * kStageRow, kScales = NST * kStage, kGroup = (TM + TN) * kStageRow;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[NST * kStage + 2 * kGroup];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int r32 = lane & 31, half = lane >> 5;

  int tm, tn;
  {
    // each XCD (workgroup index mod 8) takes a contiguous range of tiles,
    // walked in bands of 4 tile rows so that its L2 shares panels of both
    const uint32_t tiles = static_cast<uint32_t>(p.tiles_m) * static_cast<uint32_t>(p.tiles_n);
    const uint32_t x = blockIdx.x % 8, y = blockIdx.x / 8;
    const uint32_t t = x * (tiles / 8) + min(x, tiles % 8) + y;
    constexpr uint32_t kBand = 4;
    const uint32_t band = t / (kBand * p.tiles_n);
    const uint32_t rows = min(kBand, p.tiles_m - band * kBand);
    const uint32_t in = t - band * kBand * p.tiles_n;
    tm = __builtin_amdgcn_readfirstlane(static_cast<int>(band * kBand + in % rows));
    tn = __builtin_amdgcn_readfirstlane(static_cast<int>(in / rows));
  }
  const int64_t m0 = static_cast<int64_t>(tm) * TM, n0 = static_cast<int64_t>(tn) * TN;
  const uint32_t pitch = static_cast<uint32_t>(p.nb) * 16u, sp = static_cast<uint32_t>(p.sp);
  const uint8_t* a0 = uniform_ptr(p.a + m0 * pitch);
  const uint8_t* b0 = uniform_ptr(p.b + n0 * pitch);
  const uint8_t* sa0 = uniform_ptr(p.sa + m0 * sp);
  const uint8_t* sb0 = uniform_ptr(p.sb + n0 * sp);
  const int mlast = static_cast<int>(min(static_cast<int64_t>(TM), p.m - m0)) - 1;
  const int nlast = static_cast<int>(min(static_cast<int64_t>(TN), p.n - n0)) - 1;
  const int stages = (p.nb + 3) / 4;

  // Requests.  Lane l of a code request copies chunk l & 3 of row l / 4 of 16
  // rows, so it fetches the chunk that is stored there; rows past the end
  // repeat the last row (their products are not stored).
  const int chunk = (lane & 3) ^ (lane >> 4);
  uint32_t arow[DA], brow[DB];
#pragma unroll
  for (int i = 0; i < DA; ++i) arow[i] = min(16 * (wave * DA + i) + lane / 4, mlast) * pitch + chunk * 16;
#pragma unroll
  for (int i = 0; i < DB; ++i) brow[i] = min(16 * (wave * DB + i) + lane / 4, nlast) * pitch + chunk * 16;
  uint32_t asrow[DA], bsrow[DB];
#pragma unroll
  for (int i = 0; i < DA; ++i) asrow[i] = min(16 * (wave * DA + i) + lane / 4, mlast) * sp;
#pragma unroll
  for (int i = 0; i < DB; ++i) bsrow[i] = min(16 * (wave * DB + i) + lane / 4, nlast) * sp;
  const uint32_t lds0 = lds_addr(smem);
  const uint32_t dst = lds0 + wave * DA * 1024, dstb = lds0 + TM * kStageRow + wave * DB * 1024;
  // Bytes by which the lane's chunk of the last stage lies past the last
  // block, which it then loads in its place.
  const uint32_t back_last = static_cast<uint32_t>(max((stages - 1) * 4 + chunk - (p.nb - 1), 0)) * 16u;
  // request i of a stage whose codes start at pa and pb, into the place at byte
  // `to`, `back` as above
  auto request = [&](auto I, const uint8_t* pa, const uint8_t* pb, uint32_t back, uint32_t to) __attribute__((always_inline)) {
    constexpr int i = I;
    if constexpr (i < DA) lds_dma16_at<i * 1024>(pa, arow[i] - back, dst + to);
    else lds_dma16_at<(i - DA) * 1024>(pb, brow[i - DA] - back, dstb + to);
  };
  // Scale bytes come for a group of 16 stages, 64 bytes of a row, chunks of 16
  // placed as those of the codes; two groups in turn in LDS.  A chunk that
  // would pass the row's end is the row's last 16 bytes: its dwords then lie
  // `shift` further on.
  const int last_chunk = (stages - 1) / 4, last_group = last_chunk / 4;
  const uint32_t shift = static_cast<uint32_t>(last_chunk * 16) - min(static_cast<uint32_t>(last_chunk * 16), sp - 16u);
  auto request_scales = [&](int g) __attribute__((always_inline)) {
    const uint32_t off = min(static_cast<uint32_t>(g * 64 + chunk * 16), sp - 16u), to = (g & 1) * kGroup + kScales;
    unroll<DPW>([&](auto I) __attribute__((always_inline)) {
      constexpr int i = I;
      if constexpr (i < DA) lds_dma16_at<i * 1024>(sa0, asrow[i] + off, dst + to);
      else lds_dma16_at<(i - DA) * 1024>(sb0, bsrow[i - DA] + off, dstb + to);
    });
  };

  // Fragments: 32 rows, lane l holds row l & 31.
  const uint8_t* abase = smem + (wm * (TM / WM) + r32) * kStageRow;
  const uint8_t* bbase = smem + TM * kStageRow + (wn * (TN / WN) + r32) * kStageRow;
  const uint8_t* asbase = smem + kScales + (wm * (TM / WM) + r32) * kStageRow;
  const uint8_t* bsbase = smem + kScales + (TM + wn * (TN / WN) + r32) * kStageRow;
  uint32_t xs[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) xs[s] = static_cast<uint32_t>(((half * 2 + s) ^ ((r32 >> 2) & 3)) * 16);
  auto frag = [&](const uint8_t* base, uint32_t at, int f, int s) __attribute__((always_inline)) -> u32x4v {
    return *reinterpret_cast<const u32x4v*>(base + (at + xs[s]) + f * 32 * kStageRow);
  };
  // the lane's offset to the scale dwords of stage t, and that of fragment f
  auto scale_at = [&](int t) __attribute__((always_inline)) -> uint32_t {
    const int c = t >> 2;
    return static_cast<uint32_t>(((c >> 2) & 1) * kGroup + (t & 3) * 4) + (c == last_chunk ? shift : 0u) +
           static_cast<uint32_t>(((c & 3) ^ ((r32 >> 2) & 3)) * 16);
  };
  auto scale = [&](const uint8_t* base, uint32_t sat, int f) __attribute__((always_inline)) -> uint32_t {
    return *reinterpret_cast<const uint32_t*>(base + sat + f * 32 * kStageRow);
  };

  f32x16v acc[FM][FN] = {};
  u32x4v af[2][FM], bf[2][FN];
  uint32_t sa[FM], sb[FN], san[FM], sbn[FN];
  // The lane's two scale bytes of a stage in the low half of a dword; the
  // last stage's bytes of blocks past the end are cleared.
  const uint32_t keep_last = (p.nb & 3) ? (1u << (8 * (p.nb & 3))) - 1u : ~0u;
  auto keep_of = [&](int t) __attribute__((always_inline)) -> uint32_t { return t == stages - 1 ? keep_last : ~0u; };

  // Request c of a stage follows product number when(c) of the 2 NP products
  // between a barrier and the next: spread evenly, as the path from the
  // caches takes about half of that time for them.
  constexpr int NP = FM * FN, NR = FM + FN;
  constexpr auto when = [](int c) constexpr { return c * 2 * NP / DPW + (NP > 2 ? 1 : 0); };
  constexpr int kFirst = [when]() constexpr { int n = 0; while (n < DPW && when(n) < NP) ++n; return n; }();
  static_assert(when(DPW - 1) < 2 * NP, "");

  request_scales(0);
  unroll<NST>([&](auto Q) __attribute__((always_inline)) {
    const int t = min(static_cast<int>(Q), stages - 1);
    const uint8_t *pa = uniform_ptr(a0 + t * 64), *pb = uniform_ptr(b0 + t * 64);
    const uint32_t back = t == stages - 1 ? back_last : 0u;
    unroll<Q == NST - 1 ? kFirst : DPW>([&](auto I) __attribute__((always_inline)) { request(I, pa, pb, back, Q * kStage); });
  });
  wait_loads<(NST - 2) * DPW + kFirst>();
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  {
    const uint32_t keep = keep_of(0);
#pragma unroll
    for (int f = 0; f < FM; ++f) {
      af[0][f] = frag(abase, 0, f, 0);
      sa[f] = (scale(asbase, scale_at(0), f) & keep) >> (16 * half);
    }
#pragma unroll
    for (int f = 0; f < FN; ++f) {
      bf[0][f] = frag(bbase, 0, f, 0);
      sb[f] = (scale(bsbase, scale_at(0), f) & keep) >> (16 * half);
    }
  }

  // Places in LDS of this stage and of the one before, whose requests (of
  // stage tp, at pa and pb) are under way.
  uint32_t at = 0, prev = (NST - 1) * kStage;
  int tp = min(NST - 1, stages - 1);
  const uint8_t *pa = uniform_ptr(a0 + tp * 64), *pb = uniform_ptr(b0 + tp * 64);
  uint32_t backp = tp == stages - 1 ? back_last : 0u;
  for (int g = 0; g <= last_group; ++g) {
    // the next group's scales, into the place of the group before this one,
    // whose last dwords every wave had read by the last barrier
    if (g < last_group) request_scales(g + 1);
    const int end = min(16 * g + 16, stages);
    for (int t = 16 * g; t < end; ++t) {
      uint32_t next = 0, keep = 0, sat = 0;
      unroll<2>([&](auto S) __attribute__((always_inline)) {
        constexpr int s = S, cur = s, nxt = cur ^ 1;
        if constexpr (s == 1) {
          // this wave's reads of stage t are done, its part of t + 1 has come
          wait_loads<(NST - 2) * DPW>();
          __builtin_amdgcn_sched_barrier(0);
          __builtin_amdgcn_s_barrier();
          __builtin_amdgcn_sched_barrier(0);
        }
        constexpr int RP = (2 * NR + NP - 1) / NP;
        // A product at a time, and behind each a little of everything else: a
        // wave issues a handful of instructions while its product runs.
        unroll<NP>([&](auto P) __attribute__((always_inline)) {
          constexpr int i = P / FN, j = P % FN;
          acc[i][j] = mfma32<s>(bf[cur][j], af[cur][i], acc[i][j], sb[j], sa[i]);
          unroll<RP>([&](auto R) __attribute__((always_inline)) {
            constexpr int r = P * RP + R;                 // order of need: A's first, all of B, the rest of A
            constexpr int fa = r == 0 ? 0 : r > FN && r < NR ? r - FN : -1, fb = r >= 1 && r <= FN ? r - 1 : -1;
            if constexpr (fa >= 0) {
              af[nxt][fa] = frag(abase, s == 1 ? next : at, fa, nxt);
              if constexpr (s == 1) san[fa] = scale(asbase, sat, fa);
            }
            if constexpr (fb >= 0) {
              bf[nxt][fb] = frag(bbase, s == 1 ? next : at, fb, nxt);
              if constexpr (s == 1) sbn[fb] = scale(bsbase, sat, fb);
            }
          });
          if constexpr (s == 1 && P == 0) {
            // past the end: the last stage again, unused
            const bool more = tp + 1 < stages;
            tp += more;
            pa = uniform_ptr(pa + (more ? 64 : 0));
            pb = uniform_ptr(pb + (more ? 64 : 0));
            backp = tp == stages - 1 ? back_last : 0u;
            prev = at;
          }
          unroll<DPW>([&](auto C) __attribute__((always_inline)) {
            if constexpr (when(C) == P + (s == 1 ? 0 : NP)) request(C, pa, pb, backp, prev);
          });
          if constexpr (s == 0 && P == NP - 1 - (NP > 4)) {
            next = at + kStage == NST * kStage ? 0u : at + kStage;
            keep = keep_of(t + 1);
            sat = scale_at(min(t + 1, stages - 1));      // past the end: the last stage's again, unused
          }
          __builtin_amdgcn_sched_barrier(0);
        });
      });
#pragma unroll
      for (int f = 0; f < FM; ++f) sa[f] = (san[f] & keep) >> (16 * half);
#pragma unroll
      for (int f = 0; f < FN; ++f) sb[f] = (sbn[f] & keep) >> (16 * half);
      at = next;
    }
  }
  wait_loads<0>();                                     // no request outlives the workgroup

  __syncthreads();
  // Lane l holds row l & 31 of each 32 x 32 fragment (the operands are given
  // in reverse), four consecutive columns at a time.  Each wave turns 32 rows
  // at a time through LDS of its own, so that rows leave as whole lines; the
  // 16 bytes of padding per row spread 16 rows over all banks.
  constexpr int W = TN / WN, kPitch = W * 4 + 16, kLanes = W / 4;       // columns, and lanes to a row
  static_assert(NW * 32 * kPitch <= NST * kStage, "the stages' places are free now");
  uint8_t* turn = smem + wave * 32 * kPitch;
  T* out = static_cast<T*>(p.out) + m0 * p.ldo + n0;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<f32x4v*>(turn + r32 * kPitch + (32 * j + 8 * e + 4 * half) * 4) =
            f32x4v{acc[i][j][4 * e], acc[i][j][4 * e + 1], acc[i][j][4 * e + 2], acc[i][j][4 * e + 3]};
#pragma unroll
    for (int k = 0; k < 32 * kLanes / 64; ++k) {
      const int row = k * (64 / kLanes) + lane / kLanes, col = lane % kLanes * 4;
      const f32x4v v = *reinterpret_cast<const f32x4v*>(turn + row * kPitch + col * 4);
      const int r = wm * (TM / WM) + 32 * i + row, c = wn * W + col;
      if (r <= mlast) store4_out(out + r * p.ldo + c, v, nlast + 1 - c, p.accumulate);
    }
  }
}

// Direct kernel, for contractions of at most 12 blocks (whose rows of scale
// bytes are shorter than the tile kernel's requests): 4 x 4 tiles of 16 x 16
// outputs per wave, 2 x 2 waves per workgroup, no LDS.  The scaled 16 x 16 x
// 128 instruction takes from lane l the 32 codes and the scale byte of row l %
// 16, block l / 16 of a step; the operands are given in reverse, so that a lane
// ends with four consecutive outputs of a row.  Bound by its stores and by the
// rows that each request of codes and scale bytes looks up: 8192 x 8192 x 128
// 45 us, x 384 72 us (2 x 2 tiles: 51 and 107; nothing either way up to 1024 x
// 1024).
constexpr int kDirectTiles = 4;
template <typename T>
__global__ void __launch_bounds__(256) mx4_direct_kernel(const Mx4MatmulArgs p) {
  constexpr int F = kDirectTiles, kWave = 16 * F, kTile = 2 * kWave;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint32_t tn = (static_cast<uint32_t>(p.n) + kTile - 1u) / kTile;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x / tn) * kTile + (wave >> 1) * kWave;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x % tn) * kTile + (wave & 1) * kWave;
  const int r16 = lane & 15, kb = lane >> 4;
  const uint8_t *ac[F], *as[F], *bc[F], *bs[F];
#pragma unroll
  for (int i = 0; i < F; ++i) {
    // rows past the end read the last row; their products are not stored
    const int64_t ar = min(m0 + 16 * i + r16, static_cast<int64_t>(p.m) - 1);
    const int64_t br = min(n0 + 16 * i + r16, static_cast<int64_t>(p.n) - 1);
    ac[i] = p.a + ar * p.nb * 16;
    as[i] = p.sa + ar * p.sp;
    bc[i] = p.b + br * p.nb * 16;
    bs[i] = p.sb + br * p.sp;
  }
  f32x4v acc[F][F] = {};
  for (int k = 0; k < p.nb; k += 4) {
    const int b = k + kb;
    u32x4v av[F] = {}, bv[F] = {};
    int asv[F] = {}, bsv[F] = {};
    if (b < p.nb) {
#pragma unroll
      for (int i = 0; i < F; ++i) {
        av[i] = *reinterpret_cast<const u32x4v*>(ac[i] + static_cast<int64_t>(b) * 16);
        bv[i] = *reinterpret_cast<const u32x4v*>(bc[i] + static_cast<int64_t>(b) * 16);
        asv[i] = as[i][b];
        bsv[i] = bs[i][b];
      }
    }
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes8(bv[j]), codes8(av[i]), acc[i][j], 4, 4, 0, bsv[j], 0, asv[i]);
  }
  T* out = static_cast<T*>(p.out);
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) {
      const int64_t r = m0 + 16 * i + r16, c = n0 + 16 * j + 4 * kb;
      if (r < p.m && c < p.n) store4_out(out + r * p.ldo + c, acc[i][j], static_cast<int>(min(p.n - c, int64_t{4})), p.accumulate);
    }
}

// Skinny kernel: MT x 16 rows of A (all of them), 16 rows of B per
// workgroup, whose waves share the contraction and add up through LDS.  B's
// codes go from memory to registers once; the instruction's lane groups take
// adjacent blocks, so a row's 64 bytes of a step are one segment, and 16
// blocks of a row (one scale load) are in flight at a time.  Bound by reading
// B: 1 x 28672 x 8192 (125 MB) 26.3 us, 4.7 TB/s.  The waves' sums are added
// in their order, whatever the run.
template <int MT, typename T>
__global__ void __launch_bounds__(1024) mx4_skinny_kernel(const Mx4MatmulArgs p) {
  extern __shared__ __attribute__((aligned(16))) float part[];     // [waves - 1][MT][64][4]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int r16 = lane & 15, kb = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * 16;
  const int64_t br = min(n0 + r16, static_cast<int64_t>(p.n) - 1);
  const uint8_t* b = p.b + br * p.nb * 16;
  const uint8_t* sb = p.sb + br * p.sp;
  const uint8_t *a[MT], *sa[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t ar = min(16 * i + r16, p.m - 1);
    a[i] = p.a + ar * p.nb * 16;
    sa[i] = p.sa + ar * p.sp;
  }
  f32x4v acc[MT] = {};
  const int groups = (p.nb + 15) / 16;
  for (int g = wave; g < groups; g += waves) {
    const int k0 = g * 16;
    u32x4v bv[4], bsv = {}, av[MT][4], asv[MT];
    const bool whole = k0 + 16 <= p.nb;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int64_t blk = min(k0 + 4 * s + kb, p.nb - 1);
      bv[s] = *reinterpret_cast<const u32x4v*>(b + blk * 16);
#pragma unroll
      for (int i = 0; i < MT; ++i) av[i][s] = *reinterpret_cast<const u32x4v*>(a[i] + blk * 16);
    }
    if (whole) {
      bsv = *reinterpret_cast<const u32x4a4*>(sb + k0);
#pragma unroll
      for (int i = 0; i < MT; ++i) asv[i] = *reinterpret_cast<const u32x4a4*>(sa[i] + k0);
    } else {
      // blocks past the end: the last block's codes under zero scale bytes
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int blk = k0 + 4 * s, left = p.nb - blk;
        const uint32_t keep = left >= 4 ? ~0u : left > 0 ? (1u << (8 * left)) - 1u : 0u;
        bsv[s] = left > 0 ? *reinterpret_cast<const uint32_t*>(sb + blk) & keep : 0u;
#pragma unroll
        for (int i = 0; i < MT; ++i) asv[i][s] = left > 0 ? *reinterpret_cast<const uint32_t*>(sa[i] + blk) & keep : 0u;
      }
    }
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int i = 0; i < MT; ++i)
        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes8(av[i][s]), codes8(bv[s]), acc[i], 4, 4, 0,
                                                                  static_cast<int>(asv[i][s] >> (8 * kb)), 0,
                                                                  static_cast<int>(bsv[s] >> (8 * kb)));
  }
  if (waves > 1) {
    f32x4v* q = reinterpret_cast<f32x4v*>(part);
    if (wave) {
#pragma unroll
      for (int i = 0; i < MT; ++i) q[((wave - 1) * MT + i) * 64 + lane] = acc[i];
    }
    __syncthreads();
    if (wave) return;
    for (int w = 0; w < waves - 1; ++w)
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[i] += q[(w * MT + i) * 64 + lane];
  }
  T* out = static_cast<T*>(p.out);
  if (n0 + r16 < p.n) {
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 16 * i + 4 * kb + e;
        if (r < p.m) store_out(out + r * p.ldo + n0 + r16, acc[i][e], p.accumulate);
      }
  }
}

// A grid holds fewer than 2^32 threads, whichever kernel is taken.
bool mx4_matmul_fits(int64_t m, int64_t n) { return ((m + 63) / 64) * ((n + 63) / 64) <= int64_t{0xffffffff} / 256; }

template <int TM, int TN, int WM, int WN, int NST>
static hipError_t run_tile(int out_dt, Mx4MatmulArgs a, hipStream_t s) {
  a.tiles_m = (a.m + TM - 1) / TM;
  a.tiles_n = (a.n + TN - 1) / TN;
  const int64_t tiles = static_cast<int64_t>(a.tiles_m) * a.tiles_n;
  const dim3 g(static_cast<uint32_t>(tiles));
  if (out_dt == F32) mx4_tile_kernel<TM, TN, WM, WN, NST, float><<<g, 64 * WM * WN, 0, s>>>(a);
  else mx4_tile_kernel<TM, TN, WM, WN, NST, __bf16><<<g, 64 * WM * WN, 0, s>>>(a);
  return hipGetLastError();
}

static hipError_t run_direct(int out_dt, const Mx4MatmulArgs& a, hipStream_t s) {
  constexpr int kTile = 32 * kDirectTiles;
  const int64_t tn = (static_cast<int64_t>(a.n) + kTile - 1) / kTile, tm = (static_cast<int64_t>(a.m) + kTile - 1) / kTile;
  const dim3 g(static_cast<uint32_t>(tn * tm));
  if (out_dt == F32) mx4_direct_kernel<float><<<g, 256, 0, s>>>(a);
  else mx4_direct_kernel<__bf16><<<g, 256, 0, s>>>(a);
  return hipGetLastError();
}

template <int MT>
static hipError_t run_skinny(int out_dt, const Mx4MatmulArgs& a, int waves, hipStream_t s) {
  const dim3 g(static_cast<uint32_t>((a.n + 15) / 16));
  const size_t lds = static_cast<size_t>(waves - 1) * MT * 64 * 16;
  if (out_dt == F32) mx4_skinny_kernel<MT, float><<<g, 64 * waves, lds, s>>>(a);
  else mx4_skinny_kernel<MT, __bf16><<<g, 64 * waves, lds, s>>>(a);
  return hipGetLastError();
}

// Which kernel.  Measured on products of K = 8192 (and, at a quarter to a third
// of these times, K = 2048), in us.  K is not in the rule: where the number of
// stages differs much from 64, the fixed part of each tile weighs differently
// than these figures say.
//  * skinny against 64 tiles: 1 x 2048 5 and 19, 32 x 8192 17 and 19, 8 x 28672
//    31 and 28, 16 x 28672 35 and 29, 32 x 28672 50 and 29: up to 32 rows while
//    each row of A is not read again by too many workgroups (one bound on the
//    outputs; near it, at 8 x 28672, the 64 tiles would be a tenth faster);
//  * 64 tiles: 19 for up to 256 of them, 24 for 512, then in proportion;
//  * 128 tiles: 29 for up to 256, 52 for 512, 81 for 768, 112 for 1024;
//  * 256 tiles: 58 for 128 of them, 76 for 256, 162 for 512: whole rounds, as a
//    CU holds one at a time.
hipError_t launch_mx4_matmul(int out_dt, const Mx4MatmulArgs& a, hipStream_t s) {
  const int64_t m = a.m, n = a.n;
  if (m <= 32 && m * n <= (1 << 18)) {
    // waves per workgroup: enough for about 16 on every CU, none without a
    // group of 16 blocks of its own
    const int64_t wgs = (n + 15) / 16, groups = (a.nb + 15) / 16;
    int waves = 1;
    while (waves < 16 && waves * 2 <= groups && wgs * waves < 4096) waves *= 2;
    return m <= 16 ? run_skinny<1>(out_dt, a, waves, s) : run_skinny<2>(out_dt, a, waves, s);
  }
  if (a.nb <= 12) return run_direct(out_dt, a, s);
  auto tiles = [&](int64_t t) { return static_cast<double>((m + t - 1) / t) * static_cast<double>((n + t - 1) / t); };
  const double t64 = tiles(64), t128 = tiles(128), t256 = tiles(256);
  const double c64 = std::max(19.0, 24.0 * t64 / 512), c128 = std::max(29.0, 26.0 * t128 / 256);
  const double c256 = t256 <= 128 ? 58.0 : 76.0 * std::ceil(t256 / 256);
  if (c256 <= c128 && c256 <= c64) return run_tile<256, 256, 2, 2, 3>(out_dt, a, s);
  if (c128 <= c64) return run_tile<128, 128, 2, 2, 3>(out_dt, a, s);
  return run_tile<64, 64, 2, 2, 3>(out_dt, a, s);
}

}  // namespace mo
