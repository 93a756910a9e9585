// C ABI of the router's balance loss (declared in include/muon.h): validation
// (all-or-nothing) and launches.
#include <hip/hip_runtime.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "balance_internal.h"
#include "checks.h"
#include "mo_host.h"
#include "mo_internal.h"
#include "muon.h"

namespace {

using namespace mo;

int check_sizes(int64_t tokens, int64_t experts) {
  if (tokens < 0 || tokens > INT32_MAX) return fail(MO_EINVAL, "tokens must be in [0, 2^31)");
  if (experts < 1 || experts > kMaxExperts) return fail(MO_EINVAL, "experts must be in [1, %d]", kMaxExperts);
  return MO_OK;
}

int check_rows(const void* p, int dtype, int64_t tokens, int64_t experts, int64_t ld, const char* what) {
  if (!p || !aligned(p, esz_of(dtype))) return fail(MO_EINVAL, "%s must be non-NULL and aligned to its element", what);
  if (ld < experts || ld > (int64_t{1} << 40) / tokens)
    return fail(MO_EINVAL, "the row stride of %s must be >= experts, with tokens * stride <= 2^40", what);
  return MO_OK;
}

int balance(int dtype, int64_t experts, int64_t top, BalanceArgs a, void* workspace, size_t workspace_bytes, hipStream_t s) {
  int rc;
  if ((rc = validate_dtype(dtype, "dtype"))) return rc;
  if ((rc = check_sizes(a.tokens, experts))) return rc;
  if (top < 1 || top > kMaxExperts) return fail(MO_EINVAL, "top must be in [1, %d]", kMaxExperts);
  if (!std::isfinite(a.weight)) return fail(MO_EINVAL, "weight must be finite");
  if (!a.loss || !a.counts) return fail(MO_EINVAL, "loss and counts must be non-NULL");
  if (a.accumulate && !a.grad) return fail(MO_EINVAL, "accumulate needs grad");
  if (!aligned(a.index, 8) || !aligned(a.counts, 8) || !aligned(a.loss, 4) || !aligned(a.grad_loss, 4))
    return fail(MO_EINVAL, "index, counts, loss and grad_loss must be aligned to their elements");
  if (a.tokens > 0) {
    if (!a.index) return fail(MO_EINVAL, "index must be non-NULL");
    if ((rc = check_rows(a.logits, dtype, a.tokens, experts, a.ld, "logits"))) return rc;
    if (a.grad && (rc = check_rows(a.grad, dtype, a.tokens, experts, a.ld_grad, "grad"))) return rc;
  }
  a.experts = static_cast<int>(experts);
  a.top = static_cast<int>(top);
  const size_t need = balance_workspace(a.tokens, a.experts);
  if (need && (rc = check_workspace(workspace, workspace_bytes, need))) return rc;
  std::vector<Range> ranges;
  add_range(ranges, a.logits, view_bytes(a.tokens, experts, a.ld, esz_of(dtype)), 0, false);
  add_range(ranges, a.index, static_cast<size_t>(a.tokens) * top * 8, 1, false);
  add_range(ranges, a.grad_loss, 4, 2, false);
  add_range(ranges, a.loss, 4, 3, true);
  add_range(ranges, a.counts, static_cast<size_t>(experts) * 8, 4, true);
  if (a.grad) add_range(ranges, a.grad, view_bytes(a.tokens, experts, a.ld_grad, esz_of(dtype)), 5, true);
  add_range(ranges, workspace, need, 6, true);
  if ((rc = check_overlap(ranges, "argument"))) return rc;
  ProfScope ps(MO_K_BALANCE, s, static_cast<double>(a.tokens) * (static_cast<double>(experts) * esz_of(dtype) * (a.grad ? 2.0 : 1.0) + 8.0 * top));
  return checked(launch_balance(dtype, a, workspace, s), s, "balance loss");
}

}  // namespace

extern "C" {

int mo_balance_loss_workspace_size(int64_t tokens, int64_t experts, size_t* bytes) {
  if (!bytes) return fail(MO_EINVAL, "bytes is NULL");
  if (int rc = check_sizes(tokens, experts)) return rc;
  *bytes = balance_workspace(tokens, static_cast<int>(experts));
  return MO_OK;
}

int mo_balance_loss(const void* logits, int dtype, int64_t tokens, int64_t experts, int64_t ld, const int64_t* index, int64_t top,
                    float weight, const float* grad_loss, float* loss, int64_t* counts, void* grad, int64_t ld_grad, int accumulate,
                    void* workspace, size_t workspace_bytes, void* stream) {
  BalanceArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.ld_grad = ld_grad;
  a.tokens = tokens;
  a.index = index;
  a.weight = weight;
  a.grad_loss = grad_loss;
  a.loss = loss;
  a.counts = counts;
  a.grad = grad;
  a.accumulate = accumulate != 0;
  return guarded([&] { return balance(dtype, experts, top, a, workspace, workspace_bytes, static_cast<hipStream_t>(stream)); });
}

}  // extern "C"
