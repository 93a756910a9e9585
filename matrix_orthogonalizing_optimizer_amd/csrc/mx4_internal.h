// Internal declarations of the MX4 (microscaled 4-bit) kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mo {

// Layout of an image (include/muon.h): nb blocks of 32 columns per row, 16
// code bytes per block, the row of scale bytes padded to whole dwords.
__host__ __device__ inline int64_t mx4_blocks(int64_t cols) { return (cols + 31) / 32; }
__host__ __device__ inline int64_t mx4_scale_pitch(int64_t cols) { return (mx4_blocks(cols) + 3) / 4 * 4; }

// Quantisation of up to kMx4Group matrices per launch (G of them, or 1, whose
// launch arguments are smaller); tile0 is the first workgroup of the matrix.
constexpr int kMx4Group = 48;
struct Mx4QuantItem {
  const void* src;
  uint8_t *codes, *scales, *codes_t, *scales_t;
  int64_t ld;
  int32_t rows, cols;
  int64_t tile0;
};
template <int G>
struct Mx4QuantArgs {
  Mx4QuantItem item[G];
  int count;
};

struct Mx4DequantItem {
  const uint8_t *codes, *scales;
  void* dst;
  int32_t rows, cols;
  int64_t tile0;
};
template <int G>
struct Mx4DequantArgs {
  Mx4DequantItem item[G];
  int count;
};

struct Mx4MatmulArgs {
  const uint8_t *a, *sa, *b, *sb;
  void* out;
  int64_t ldo;
  int m, n;
  int nb;                // blocks per row of a and b
  int sp;                // bytes per row of scales
  int accumulate;
  int tiles_m, tiles_n;  // filled in at the launch
};

// A product's 32-bit offsets cover 256 rows of an image.
constexpr int64_t kMx4MaxCols = int64_t{1} << 25;
bool mx4_matmul_fits(int64_t m, int64_t n);

int64_t mx4_quant_tiles(int64_t rows, int64_t cols, bool cols_image);
int64_t mx4_dequant_tiles(int dt, int64_t rows, int64_t cols);
template <int G>
hipError_t launch_mx4_quant(int dt, bool cols_image, const Mx4QuantArgs<G>& a, int64_t tiles, hipStream_t s);
template <int G>
hipError_t launch_mx4_dequant(int dt, const Mx4DequantArgs<G>& a, int64_t tiles, hipStream_t s);
hipError_t launch_mx4_matmul(int out_dt, const Mx4MatmulArgs& a, hipStream_t s);

}  // namespace mo
