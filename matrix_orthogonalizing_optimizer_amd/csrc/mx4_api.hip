// C ABI of the MX4 entry points (declared in include/muon.h): validation
// (all-or-nothing), grouping into launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <climits>
#include <cstdint>
#include <exception>
#include <vector>

#include "mo_host.h"
#include "mo_internal.h"
#include "muon.h"
#include "mx4_internal.h"

namespace {

using namespace mo;

long long ll(int64_t x) { return static_cast<long long>(x); }

int check_shape(int64_t rows, int64_t cols, const char* what, int64_t i) {
  if (rows < 1 || cols < 1 || rows > INT32_MAX || cols > INT32_MAX || rows > (int64_t{1} << 40) / cols)
    return fail(MO_EINVAL, "%s %lld: rows and cols must be in [1, 2^31) with rows * cols <= 2^40", what, ll(i));
  return MO_OK;
}

size_t code_bytes(int64_t rows, int64_t cols) { return static_cast<size_t>(rows * mx4_blocks(cols) * 16); }
size_t scale_bytes(int64_t rows, int64_t cols) { return static_cast<size_t>(rows * mx4_scale_pitch(cols)); }

// Bytes that a [rows, cols] view with rows `ld` elements apart touches.
size_t view_bytes(int64_t rows, int64_t cols, int64_t ld, int esz) {
  return (static_cast<size_t>(rows - 1) * static_cast<size_t>(ld) + static_cast<size_t>(cols)) * static_cast<size_t>(esz);
}

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

struct Range {
  uintptr_t lo, hi;
  int64_t idx;
  bool out;
};

void add_range(std::vector<Range>& v, const void* p, size_t n, int64_t idx, bool out) {
  if (p && n) v.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + n, idx, out});
}

// No output may share a byte with any other range; inputs may share.
int check_overlap(std::vector<Range>& v, const char* what) {
  std::sort(v.begin(), v.end(), [](const Range& a, const Range& b) { return a.lo < b.lo; });
  uintptr_t end_any = 0, end_out = 0;   // furthest end of the ranges so far
  for (const Range& r : v) {
    if (r.lo < end_out || (r.out && r.lo < end_any))
      return fail(MO_EINVAL, "%s %lld: an output overlaps another buffer of the call", what, ll(r.idx));
    end_any = std::max(end_any, r.hi);
    if (r.out) end_out = std::max(end_out, r.hi);
  }
  return MO_OK;
}

int check_image(const mo_mx4_image& x, const char* what, int64_t i) {
  if (int rc = check_shape(x.rows, x.cols, what, i)) return rc;
  if (!x.codes || !x.scales) return fail(MO_EINVAL, "%s %lld: codes and scales must be non-NULL", what, ll(i));
  if (!aligned(x.codes, 16) || !aligned(x.scales, 4))
    return fail(MO_EINVAL, "%s %lld: codes must be 16-byte and scales 4-byte aligned", what, ll(i));
  return MO_OK;
}

int esz_of(int dt) { return dt == MO_F32 ? 4 : 2; }

// Launches are limited by kMx4Group matrices and by a grid of fewer than
// 2^32 threads.
constexpr int64_t kMaxTiles = 0xffffffff / 512;

// Launches over the matrices that want (or do not want) an image of the
// transpose, up to G per launch.
template <int G>
int quant_group(const mo_mx4_item* items, int64_t count, int dtype, bool cols_image, hipStream_t s) {
  const int esz = esz_of(dtype);
  for (int64_t i = 0; i < count;) {
    Mx4QuantArgs<G> a;
    a.count = 0;
    int64_t tiles = 0;
    double bytes = 0;
    for (; i < count && a.count < G; ++i) {
      const mo_mx4_item& x = items[i];
      if ((x.codes_t != nullptr) != cols_image) continue;
      const int64_t t = mx4_quant_tiles(x.rows, x.cols, cols_image);
      if (a.count && tiles + t > kMaxTiles) break;
      a.item[a.count++] = {x.src, static_cast<uint8_t*>(x.codes), static_cast<uint8_t*>(x.scales),
                           static_cast<uint8_t*>(x.codes_t), static_cast<uint8_t*>(x.scales_t), x.ld,
                           static_cast<int32_t>(x.rows), static_cast<int32_t>(x.cols), tiles};
      tiles += t;
      bytes += static_cast<double>(x.rows) * x.cols * esz;
      if (x.codes) bytes += static_cast<double>(code_bytes(x.rows, x.cols) + scale_bytes(x.rows, x.cols));
      if (x.codes_t) bytes += static_cast<double>(code_bytes(x.cols, x.rows) + scale_bytes(x.cols, x.rows));
    }
    if (!a.count) continue;
    ProfScope ps(MO_K_MX4_QUANT, s, bytes);
    if (int rc = checked(launch_mx4_quant(dtype, cols_image, a, tiles, s), s, "mx4 quantize")) return rc;
  }
  return MO_OK;
}

int quantize(const mo_mx4_item* items, int64_t count, int dtype, hipStream_t s) {
  int rc;
  if ((rc = validate_dtype(dtype, "dtype"))) return rc;
  if (count < 0) return fail(MO_EINVAL, "count must be >= 0");
  if (count > 0 && !items) return fail(MO_EINVAL, "items is NULL");
  const int esz = esz_of(dtype);
  std::vector<Range> ranges;
  for (int64_t i = 0; i < count; ++i) {
    const mo_mx4_item& x = items[i];
    if ((rc = check_shape(x.rows, x.cols, "matrix", i))) return rc;
    if (x.ld < x.cols || x.ld > (int64_t{1} << 40) / x.rows)
      return fail(MO_EINVAL, "matrix %lld: ld must be >= cols, with rows * ld <= 2^40", ll(i));
    if (!x.src || !aligned(x.src, esz))
      return fail(MO_EINVAL, "matrix %lld: src must be non-NULL and aligned to its element", ll(i));
    if (!x.codes != !x.scales || !x.codes_t != !x.scales_t || (!x.codes && !x.codes_t))
      return fail(MO_EINVAL, "matrix %lld: an image needs codes and scales, and one image is needed", ll(i));
    if (!aligned(x.codes, 16) || !aligned(x.codes_t, 16) || !aligned(x.scales, 4) || !aligned(x.scales_t, 4))
      return fail(MO_EINVAL, "matrix %lld: codes must be 16-byte and scales 4-byte aligned", ll(i));
    if (mx4_quant_tiles(x.rows, x.cols, x.codes_t != nullptr) > kMaxTiles)
      return fail(MO_EINVAL, "matrix %lld: too large for one launch", ll(i));
    add_range(ranges, x.src, view_bytes(x.rows, x.cols, x.ld, esz), i, false);
    add_range(ranges, x.codes, code_bytes(x.rows, x.cols), i, true);
    add_range(ranges, x.scales, scale_bytes(x.rows, x.cols), i, true);
    add_range(ranges, x.codes_t, code_bytes(x.cols, x.rows), i, true);
    add_range(ranges, x.scales_t, scale_bytes(x.cols, x.rows), i, true);
  }
  if ((rc = check_overlap(ranges, "matrix"))) return rc;
  if (count == 1) return quant_group<1>(items, count, dtype, items[0].codes_t != nullptr, s);
  // matrices with an image of the transpose, then those without
  for (bool cols_image : {true, false})
    if ((rc = quant_group<kMx4Group>(items, count, dtype, cols_image, s))) return rc;
  return MO_OK;
}

// Launches over the images of one kind, up to G per launch.
template <int G>
int dequant_group(const mo_mx4_image* images, void* const* dst, int64_t count, int dtype, hipStream_t s) {
  const int esz = esz_of(dtype);
  for (int64_t i = 0; i < count;) {
    Mx4DequantArgs<G> a;
    a.count = 0;
    int64_t tiles = 0;
    double bytes = 0;
    while (i < count && a.count < G) {
      const mo_mx4_image& x = images[i];
      const int64_t t = mx4_dequant_tiles(dtype, x.rows, x.cols);
      if (a.count && tiles + t > kMaxTiles) break;
      a.item[a.count++] = {static_cast<const uint8_t*>(x.codes), static_cast<const uint8_t*>(x.scales), dst[i],
                           static_cast<int32_t>(x.rows), static_cast<int32_t>(x.cols), tiles};
      tiles += t;
      bytes += static_cast<double>(x.rows) * x.cols * esz +
               static_cast<double>(code_bytes(x.rows, x.cols) + scale_bytes(x.rows, x.cols));
      ++i;
    }
    ProfScope ps(MO_K_MX4_DEQUANT, s, bytes);
    if (int rc = checked(launch_mx4_dequant(dtype, a, tiles, s), s, "mx4 dequantize")) return rc;
  }
  return MO_OK;
}

int dequantize(const mo_mx4_image* images, void* const* dst, int64_t count, int dtype, hipStream_t s) {
  int rc;
  if ((rc = validate_dtype(dtype, "dtype"))) return rc;
  if (count < 0) return fail(MO_EINVAL, "count must be >= 0");
  if (count > 0 && (!images || !dst)) return fail(MO_EINVAL, "images or dst is NULL");
  const int esz = esz_of(dtype);
  std::vector<Range> ranges;
  for (int64_t i = 0; i < count; ++i) {
    const mo_mx4_image& x = images[i];
    if ((rc = check_image(x, "image", i))) return rc;
    if (!dst[i] || !aligned16(dst[i])) return fail(MO_EINVAL, "image %lld: dst must be non-NULL and 16-byte aligned", ll(i));
    if (mx4_dequant_tiles(dtype, x.rows, x.cols) > kMaxTiles) return fail(MO_EINVAL, "image %lld: too large for one launch", ll(i));
    add_range(ranges, x.codes, code_bytes(x.rows, x.cols), i, false);
    add_range(ranges, x.scales, scale_bytes(x.rows, x.cols), i, false);
    add_range(ranges, dst[i], view_bytes(x.rows, x.cols, x.cols, esz), i, true);
  }
  if ((rc = check_overlap(ranges, "image"))) return rc;
  return count == 1 ? dequant_group<1>(images, dst, count, dtype, s) : dequant_group<kMx4Group>(images, dst, count, dtype, s);
}

int matmul(const mo_mx4_image* a, const mo_mx4_image* b, void* out, int out_dtype, int64_t ldo, int accumulate,
           hipStream_t s) {
  int rc;
  if (!a || !b) return fail(MO_EINVAL, "a or b is NULL");
  if ((rc = validate_dtype(out_dtype, "out_dtype"))) return rc;
  if ((rc = check_image(*a, "operand", 0)) || (rc = check_image(*b, "operand", 1))) return rc;
  if (a->cols != b->cols)
    return fail(MO_EINVAL, "operands have %lld and %lld columns: the contraction needs equal ones", ll(a->cols), ll(b->cols));
  if (a->cols > kMx4MaxCols) return fail(MO_EINVAL, "operands have %lld columns, more than 2^25", ll(a->cols));
  if (!mx4_matmul_fits(a->rows, b->rows)) return fail(MO_EINVAL, "too many output tiles for one launch");
  const int esz = esz_of(out_dtype);
  if (!out || !aligned(out, esz)) return fail(MO_EINVAL, "out must be non-NULL and aligned to its element");
  if (ldo < b->rows || ldo > (int64_t{1} << 40) / a->rows)
    return fail(MO_EINVAL, "ldo must be >= the rows of b, with rows of a * ldo <= 2^40");
  std::vector<Range> ranges;
  for (const mo_mx4_image* x : {a, b}) {
    add_range(ranges, x->codes, code_bytes(x->rows, x->cols), x == a ? 0 : 1, false);
    add_range(ranges, x->scales, scale_bytes(x->rows, x->cols), x == a ? 0 : 1, false);
  }
  add_range(ranges, out, view_bytes(a->rows, b->rows, ldo, esz), 2, true);
  if ((rc = check_overlap(ranges, "operand"))) return rc;
  Mx4MatmulArgs g{};
  g.a = static_cast<const uint8_t*>(a->codes);
  g.sa = static_cast<const uint8_t*>(a->scales);
  g.b = static_cast<const uint8_t*>(b->codes);
  g.sb = static_cast<const uint8_t*>(b->scales);
  g.out = out;
  g.ldo = ldo;
  g.m = static_cast<int>(a->rows);
  g.n = static_cast<int>(b->rows);
  g.nb = static_cast<int>(mx4_blocks(a->cols));
  g.sp = static_cast<int>(mx4_scale_pitch(a->cols));
  g.accumulate = accumulate != 0;
  ProfScope ps(MO_K_MX4_MATMUL, s, 2.0 * static_cast<double>(a->rows) * b->rows * a->cols);
  return checked(launch_mx4_matmul(out_dtype, g, s), s, "mx4 matmul");
}

// No C++ exception may leave a C entry point.
template <typename F>
int guarded(F f) {
  try {
    return f();
  } catch (const std::exception& e) {
    return fail(MO_EINVAL, "host memory: %s", e.what());
  }
}

}  // namespace

extern "C" {

int mo_mx4_image_size(int64_t rows, int64_t cols, size_t* codes, size_t* scales) {
  if (!codes || !scales) return fail(MO_EINVAL, "code_bytes and scale_bytes must be non-NULL");
  if (int rc = check_shape(rows, cols, "image", 0)) return rc;
  *codes = code_bytes(rows, cols);
  *scales = scale_bytes(rows, cols);
  return MO_OK;
}

int mo_mx4_quantize(const mo_mx4_item* items, int64_t count, int dtype, void* stream) {
  return guarded([&] { return quantize(items, count, dtype, static_cast<hipStream_t>(stream)); });
}

int mo_mx4_dequantize(const mo_mx4_image* images, void* const* dst, int64_t count, int dtype, void* stream) {
  return guarded([&] { return dequantize(images, dst, count, dtype, static_cast<hipStream_t>(stream)); });
}

int mo_mx4_matmul(const mo_mx4_image* a, const mo_mx4_image* b, void* out, int out_dtype, int64_t ldo, int accumulate,
                  void* stream) {
  return guarded([&] { return matmul(a, b, out, out_dtype, ldo, accumulate, static_cast<hipStream_t>(stream)); });
}

}  // extern "C"
