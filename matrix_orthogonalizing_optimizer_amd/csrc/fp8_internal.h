// Internal declarations of the 8-bit (e4m3, a scale per block of 128) kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mo {

// Layout of an image (include/muon.h): nb blocks of 128 columns per row, one
// code byte per column of a block, the row of scale bytes padded to 16.
__host__ __device__ inline int64_t fp8_blocks(int64_t cols) { return (cols + 127) / 128; }
__host__ __device__ inline int64_t fp8_scale_pitch(int64_t cols) { return (fp8_blocks(cols) + 15) / 16 * 16; }

// Quantisation of up to kFp8Group matrices per launch (G of them, or 1, whose
// launch arguments are smaller); tile0 is the first workgroup of the matrix.
constexpr int kFp8Group = 48;
struct Fp8QuantItem {
  const void* src;
  uint8_t *codes, *scales, *codes_t, *scales_t;
  int64_t ld;
  int32_t rows, cols;
  int64_t tile0;
};
template <int G>
struct Fp8QuantArgs {
  Fp8QuantItem item[G];
  int count;
  int square;            // one scale for 128 rows x 128 columns
};

struct Fp8DequantItem {
  const uint8_t *codes, *scales;
  void* dst;
  int32_t rows, cols;
  int64_t tile0;
};
template <int G>
struct Fp8DequantArgs {
  Fp8DequantItem item[G];
  int count;
};

struct Fp8MatmulArgs {
  const uint8_t *a, *sa, *b, *sb;
  void* out;
  int64_t ldo;
  int m, n;
  int nb;                // blocks per row of a and b
  int sp;                // bytes per row of scales
  int accumulate;
};

// A product's 32-bit offsets cover 256 rows of an image.
constexpr int64_t kFp8MaxCols = int64_t{1} << 23;
bool fp8_matmul_fits(int64_t m, int64_t n);

// tiles: the kernel that takes 128 x 128 elements per workgroup (an image of
// the transpose or square scales), not the one that takes rows.
int64_t fp8_quant_tiles(int64_t rows, int64_t cols, bool tiles);
int64_t fp8_dequant_tiles(int dt, int64_t rows, int64_t cols);
template <int G>
hipError_t launch_fp8_quant(int dt, bool tiles, const Fp8QuantArgs<G>& a, int64_t count, hipStream_t s);
template <int G>
hipError_t launch_fp8_dequant(int dt, const Fp8DequantArgs<G>& a, int64_t tiles, hipStream_t s);
hipError_t launch_fp8_matmul(int out_dt, const Fp8MatmulArgs& a, hipStream_t s);

}  // namespace mo
