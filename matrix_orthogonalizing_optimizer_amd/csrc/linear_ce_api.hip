// C ABI of the cross entropy of a linear layer's logits (declared in
// include/muon.h): validation (all-or-nothing) and launches.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>

#include "checks.h"
#include "linear_ce_internal.h"
#include "mo_host.h"
#include "mo_internal.h"
#include "muon.h"

namespace {

using namespace mo;

int check_sizes(int64_t rows, int64_t hidden, int64_t vocab) {
  if (rows < 0 || rows > kCeMaxRows) return fail(MO_EINVAL, "rows must be in [0, 2^20]");
  if (hidden < 1 || hidden > kCeMaxHidden) return fail(MO_EINVAL, "hidden must be in [1, 2^22]");
  if (vocab < 1 || vocab > INT32_MAX) return fail(MO_EINVAL, "vocab must be in [1, 2^31)");
  return MO_OK;
}

int check_matrix(const void* p, int dtype, int64_t rows, int64_t cols, int64_t ld, const char* what) {
  if (!p || !aligned(p, esz_of(dtype))) return fail(MO_EINVAL, "%s must be non-NULL and aligned to its element", what);
  if (ld < cols || ld > (int64_t{1} << 40) / rows)
    return fail(MO_EINVAL, "the row stride of %s must be >= hidden, with rows * stride <= 2^40", what);
  return MO_OK;
}

int linear_ce(const LinearCeArgs& a, int64_t rows, int64_t hidden, int64_t vocab, void* workspace, size_t workspace_bytes, hipStream_t s) {
  int rc;
  if ((rc = validate_dtype(a.x_dt, "x_dtype")) || (rc = validate_dtype(a.w_dt, "w_dtype")) || (rc = validate_dtype(a.dw_dt, "dw_dtype"))) return rc;
  if ((rc = check_sizes(rows, hidden, vocab))) return rc;
  if (a.accumulate && !a.dw) return fail(MO_EINVAL, "accumulate needs dw");
  if (!aligned(a.targets, 8) || !aligned(a.grad_loss, 4) || !aligned(a.loss, 4))
    return fail(MO_EINVAL, "targets, grad_loss and loss must be aligned to their elements");
  if ((rc = check_matrix(a.w, a.w_dt, vocab, hidden, a.ldw, "w"))) return rc;
  if (a.dw && (rc = check_matrix(a.dw, a.dw_dt, vocab, hidden, a.ld_dw, "dw"))) return rc;
  if (rows > 0) {
    if (!a.targets || !a.loss) return fail(MO_EINVAL, "targets and loss must be non-NULL");
    if ((rc = check_matrix(a.x, a.x_dt, rows, hidden, a.ldx, "x"))) return rc;
    if (a.dx && (rc = check_matrix(a.dx, a.x_dt, rows, hidden, a.ld_dx, "dx"))) return rc;
  }
  const size_t need = linear_ce_workspace(rows, hidden, vocab, a.x_dt, a.dw_dt, a.dx != nullptr, a.dw != nullptr);
  if (need && (rc = check_workspace(workspace, workspace_bytes, need))) return rc;
  const size_t n = static_cast<size_t>(rows);
  std::vector<Range> ranges;
  add_range(ranges, a.x, view_bytes(rows, hidden, a.ldx, esz_of(a.x_dt)), 0, false);
  add_range(ranges, a.w, view_bytes(vocab, hidden, a.ldw, esz_of(a.w_dt)), 1, false);
  add_range(ranges, a.targets, n * 8, 2, false);
  add_range(ranges, a.grad_loss, n * 4, 3, false);
  add_range(ranges, a.loss, n * 4, 4, true);
  if (a.dx) add_range(ranges, a.dx, view_bytes(rows, hidden, a.ld_dx, esz_of(a.x_dt)), 5, true);
  if (a.dw) add_range(ranges, a.dw, view_bytes(vocab, hidden, a.ld_dw, esz_of(a.dw_dt)), 6, true);
  add_range(ranges, workspace, need, 7, true);
  if ((rc = check_overlap(ranges, "argument"))) return rc;
  if (rows == 0 && (!a.dw || a.accumulate)) return MO_OK;
  const double products = 1.0 + (a.dx ? 1.0 : 0.0) + (a.dw ? 1.0 : 0.0);
  ProfScope ps(MO_K_LINEAR_CE, s, 2.0 * products * static_cast<double>(rows) * static_cast<double>(hidden) * static_cast<double>(vocab));
  return checked(launch_linear_ce(a, workspace, s), s, "linear cross entropy");
}

}  // namespace

extern "C" {

int mo_linear_ce_workspace_size(int64_t rows, int64_t hidden, int64_t vocab, int x_dtype, int dw_dtype, int want_dx, int want_dw,
                                size_t* bytes) {
  if (!bytes) return fail(MO_EINVAL, "bytes is NULL");
  int rc;
  if ((rc = validate_dtype(x_dtype, "x_dtype")) || (rc = validate_dtype(dw_dtype, "dw_dtype"))) return rc;
  if ((rc = check_sizes(rows, hidden, vocab))) return rc;
  *bytes = linear_ce_workspace(rows, hidden, vocab, x_dtype, dw_dtype, want_dx != 0, want_dw != 0);
  return MO_OK;
}

int mo_linear_ce(const void* x, int x_dtype, int64_t ldx, const void* w, int w_dtype, int64_t ldw, int64_t rows, int64_t hidden,
                 int64_t vocab, const int64_t* targets, const float* grad_loss, float* loss, void* dx, int64_t ld_dx, void* dw,
                 int dw_dtype, int64_t ld_dw, int accumulate, void* workspace, size_t workspace_bytes, void* stream) {
  LinearCeArgs a{};
  a.x = x;
  a.w = w;
  a.x_dt = x_dtype;
  a.w_dt = w_dtype;
  a.dw_dt = dw_dtype;
  a.ldx = ldx;
  a.ldw = ldw;
  a.ld_dx = ld_dx;
  a.ld_dw = ld_dw;
  a.rows = static_cast<int>(rows);
  a.hidden = static_cast<int>(hidden);
  a.vocab = static_cast<int>(vocab);
  a.targets = targets;
  a.grad_loss = grad_loss;
  a.loss = loss;
  a.dx = dx;
  a.dw = dw;
  a.accumulate = accumulate != 0;
  return guarded([&] { return linear_ce(a, rows, hidden, vocab, workspace, workspace_bytes, static_cast<hipStream_t>(stream)); });
}

}  // extern "C"
