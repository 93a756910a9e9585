// C ABI of the token log probabilities and of the distillation loss
// (declared in include/muon.h): validation (all-or-nothing) and launches.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>

#include "mo_host.h"
#include "mo_internal.h"
#include "muon.h"
#include "token_internal.h"

namespace {

using namespace mo;

static_assert(kMaxTop == MO_MAX_TOP, "slots per row");

int esz_of(int dt) { return dt == MO_F32 ? 4 : 2; }

bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int check_sizes(int64_t rows, int64_t vocab, int top, int top_min) {
  // a row is one workgroup of at most 1024 threads in a grid of fewer than 2^32
  if (rows < 0 || rows > (int64_t{1} << 22) - 1) return fail(MO_EINVAL, "rows must be in [0, 2^22)");
  if (vocab < 1 || vocab > INT32_MAX) return fail(MO_EINVAL, "vocab must be in [1, 2^31)");
  if (!token_grid_fits(rows, vocab)) return fail(MO_EINVAL, "rows times vocab is too large for one launch");
  if (top < top_min || top > MO_MAX_TOP) return fail(MO_EINVAL, "top must be in [%d, %d] (got %d)", top_min, MO_MAX_TOP, top);
  return MO_OK;
}

// 1 / temperature times log2(e) is finite, and temperature squared, the scale
// of the loss at high temperatures.
int check_temperature(float t) {
  if (!(t >= 0x1p-126f && t <= 0x1p63f)) return fail(MO_EINVAL, "temperature must be in [2^-126, 2^63]");
  return MO_OK;
}

int check_rows(const void* p, int dtype, int64_t rows, int64_t vocab, int64_t ld, const char* what) {
  if (!p || !aligned(p, esz_of(dtype))) return fail(MO_EINVAL, "%s must be non-NULL and aligned to its element", what);
  if (ld < vocab || ld > (int64_t{1} << 40) / rows)
    return fail(MO_EINVAL, "the row stride of %s must be >= vocab, with rows * stride <= 2^40", what);
  return MO_OK;
}

struct Range {
  const void* p;
  size_t n;
  bool out;
  const char* name;
};

template <size_t N>
int check_overlap(const Range (&r)[N]) {
  for (size_t i = 0; i < N; ++i)
    for (size_t j = i + 1; j < N; ++j) {
      if (!r[i].p || !r[j].p || !r[i].n || !r[j].n || !(r[i].out || r[j].out)) continue;
      const uintptr_t x = reinterpret_cast<uintptr_t>(r[i].p), y = reinterpret_cast<uintptr_t>(r[j].p);
      if (x < y + r[j].n && y < x + r[i].n) return fail(MO_EINVAL, "%s and %s overlap", r[i].name, r[j].name);
    }
  return MO_OK;
}

size_t row_bytes(int64_t rows, int64_t vocab, int64_t ld, int dtype) {
  return (static_cast<size_t>(rows - 1) * static_cast<size_t>(ld) + static_cast<size_t>(vocab)) * esz_of(dtype);
}

}  // namespace

extern "C" {

int mo_token_logprobs_workspace_size(int64_t rows, int64_t vocab, int top, size_t* bytes) {
  if (!bytes) return fail(MO_EINVAL, "bytes is NULL");
  if (int rc = check_sizes(rows, vocab, top, 0)) return rc;
  *bytes = logprobs_workspace(rows, vocab, top);
  return MO_OK;
}

int mo_distill_loss_workspace_size(int64_t rows, int64_t vocab, int top, size_t* bytes) {
  if (!bytes) return fail(MO_EINVAL, "bytes is NULL");
  if (int rc = check_sizes(rows, vocab, top, 1)) return rc;
  *bytes = distill_workspace(rows, vocab, top);
  return MO_OK;
}

int mo_token_logprobs(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld, const int64_t* tokens,
                      float temperature, float* logprob, float* entropy, int top, int64_t* top_index,
                      float* top_logprob, void* workspace, size_t workspace_bytes, void* stream) {
  int rc;
  if ((rc = validate_dtype(dtype, "dtype"))) return rc;
  if ((rc = check_sizes(rows, vocab, top, 0))) return rc;
  if (top > vocab) return fail(MO_EINVAL, "top = %d exceeds vocab = %lld", top, static_cast<long long>(vocab));
  if ((rc = check_temperature(temperature))) return rc;
  if (!tokens != !logprob) return fail(MO_EINVAL, "tokens and logprob: both or neither");
  if ((top > 0) != (top_index != nullptr) || (top > 0) != (top_logprob != nullptr))
    return fail(MO_EINVAL, "top_index and top_logprob must be given iff top > 0");
  if (!aligned(tokens, 8) || !aligned(top_index, 8) || !aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(top_logprob, 4))
    return fail(MO_EINVAL, "tokens and outputs must be aligned to their elements");
  if (rows == 0) return MO_OK;
  if ((rc = check_rows(logits, dtype, rows, vocab, ld, "logits"))) return rc;
  const size_t need = logprobs_workspace(rows, vocab, top);
  if (need && (rc = check_workspace(workspace, workspace_bytes, need))) return rc;
  const size_t n = static_cast<size_t>(rows), k = n * static_cast<size_t>(top);
  const Range ranges[] = {{logits, row_bytes(rows, vocab, ld, dtype), false, "logits"},
                          {tokens, n * 8, false, "tokens"},
                          {logprob, n * 4, true, "logprob"},
                          {entropy, n * 4, true, "entropy"},
                          {top_index, k * 8, true, "top_index"},
                          {top_logprob, k * 4, true, "top_logprob"},
                          {workspace, need, true, "the workspace"}};
  if ((rc = check_overlap(ranges))) return rc;
  if (!logprob && !entropy && top == 0) return MO_OK;
  LogprobArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.rows = static_cast<int>(rows);
  a.vocab = static_cast<int>(vocab);
  a.top = top;
  a.inv_tau = 1.0f / temperature;
  a.tokens = tokens;
  a.logprob = logprob;
  a.entropy = entropy;
  a.top_index = top_index;
  a.top_logprob = top_logprob;
  hipStream_t s = static_cast<hipStream_t>(stream);
  ProfScope ps(MO_K_LOGPROBS, s, static_cast<double>(rows) * vocab * esz_of(dtype));
  return checked(launch_logprobs(dtype, a, workspace, s), s, "token logprobs");
}

int mo_distill_loss(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t ld, const int64_t* top_index,
                    const float* top_logit, int top, float temperature, const float* grad_loss, float* loss,
                    void* grad, int64_t ld_grad, void* workspace, size_t workspace_bytes, void* stream) {
  int rc;
  if ((rc = validate_dtype(dtype, "dtype"))) return rc;
  if ((rc = check_sizes(rows, vocab, top, 1))) return rc;
  if ((rc = check_temperature(temperature))) return rc;
  if (rows == 0) return MO_OK;
  if (!loss && !grad) return fail(MO_EINVAL, "loss and grad are both NULL");
  if (!top_index || !top_logit) return fail(MO_EINVAL, "top_index and top_logit must be non-NULL");
  if (!aligned(top_index, 8) || !aligned(top_logit, 4) || !aligned(grad_loss, 4) || !aligned(loss, 4))
    return fail(MO_EINVAL, "top_index, top_logit, grad_loss and loss must be aligned to their elements");
  if ((rc = check_rows(logits, dtype, rows, vocab, ld, "logits"))) return rc;
  if (grad && (rc = check_rows(grad, dtype, rows, vocab, ld_grad, "grad"))) return rc;
  const size_t need = distill_workspace(rows, vocab, top);
  if (need && (rc = check_workspace(workspace, workspace_bytes, need))) return rc;
  const size_t n = static_cast<size_t>(rows), k = n * static_cast<size_t>(top);
  const Range ranges[] = {{logits, row_bytes(rows, vocab, ld, dtype), false, "logits"},
                          {top_index, k * 8, false, "top_index"},
                          {top_logit, k * 4, false, "top_logit"},
                          {grad_loss, n * 4, false, "grad_loss"},
                          {loss, n * 4, true, "loss"},
                          {grad, grad ? row_bytes(rows, vocab, ld_grad, dtype) : 0, true, "grad"},
                          {workspace, need, true, "the workspace"}};
  if ((rc = check_overlap(ranges))) return rc;
  DistillArgs a{};
  a.logits = logits;
  a.ld = ld;
  a.ld_grad = ld_grad;
  a.rows = static_cast<int>(rows);
  a.vocab = static_cast<int>(vocab);
  a.top = top;
  a.tau = temperature;
  a.inv_tau = 1.0f / temperature;
  a.top_index = top_index;
  a.top_logit = top_logit;
  a.grad_loss = grad_loss;
  a.loss = loss;
  a.grad = grad;
  hipStream_t s = static_cast<hipStream_t>(stream);
  ProfScope ps(MO_K_DISTILL, s, static_cast<double>(rows) * vocab * esz_of(dtype) * (grad ? 2.0 : 1.0));
  return checked(launch_distill(dtype, a, workspace, s), s, "distill loss");
}

}  // extern "C"
