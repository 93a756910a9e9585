// Argument checks that several C-ABI translation units share.
#pragma once

#include <algorithm>
#include <cstdint>
#include <exception>
#include <vector>

#include "mo_host.h"
#include "muon.h"

namespace mo {

inline long long ll(int64_t x) { return static_cast<long long>(x); }
inline int esz_of(int dt) { return dt == MO_F32 ? 4 : 2; }
inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Bytes that a [rows, cols] view with rows `ld` elements apart touches.
inline size_t view_bytes(int64_t rows, int64_t cols, int64_t ld, int esz) {
  if (rows < 1 || cols < 1) return 0;
  return (static_cast<size_t>(rows - 1) * static_cast<size_t>(ld) + static_cast<size_t>(cols)) * static_cast<size_t>(esz);
}

struct Range {
  uintptr_t lo, hi;
  int64_t idx;
  bool out;
};

inline void add_range(std::vector<Range>& v, const void* p, size_t n, int64_t idx, bool out) {
  if (p && n) v.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + n, idx, out});
}

// No output may share a byte with any other range; inputs may share.
inline int check_overlap(std::vector<Range>& v, const char* what) {
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

// No C++ exception may leave a C entry point.
template <typename F>
int guarded(F f) {
  try {
    return f();
  } catch (const std::exception& e) {
    return fail(MO_EINVAL, "host memory: %s", e.what());
  }
}

}  // namespace mo
