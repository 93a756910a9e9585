// Internal declarations of the cross entropy of a linear layer's logits.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mo {

struct LinearCeArgs {
  const void *x, *w;
  int x_dt, w_dt, dw_dt;
  int64_t ldx, ldw, ld_dx, ld_dw;       // elements
  int rows, hidden, vocab;
  const int64_t* targets;
  const float* grad_loss;
  float* loss;
  void *dx, *dw;                        // either or both may be null
  int accumulate;                       // dw += ..
};

// Every size is one of these.
constexpr int64_t kCeMaxRows = int64_t{1} << 20, kCeMaxHidden = int64_t{1} << 22;

size_t linear_ce_workspace(int64_t rows, int64_t hidden, int64_t vocab, int x_dt, int dw_dt, bool dx, bool dw);
hipError_t launch_linear_ce(const LinearCeArgs& a, void* ws, hipStream_t s);

}  // namespace mo
