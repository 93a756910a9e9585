// Internal declarations of the token log-probability and distillation
// kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mo {

constexpr int kMaxTop = 128;

struct LogprobArgs {
  const void* logits;
  int64_t ld;
  int rows, vocab, top;
  float inv_tau;
  const int64_t* tokens;
  float *logprob, *entropy;
  int64_t* top_index;
  float* top_logprob;
  // filled in at the launch: pieces of a row, columns of a piece, and each
  // piece's {m, S, U, -} and sorted keys
  int pieces, piece_len;
  float4* part;
  unsigned long long* part_keys;
};

struct DistillArgs {
  const void* logits;
  int64_t ld, ld_grad;
  int rows, vocab, top;
  float tau, inv_tau;
  const int64_t* top_index;
  const float* top_logit;
  const float* grad_loss;
  float* loss;
  void* grad;
  int pieces, piece_len;   // as above
  float4* part;
};

bool token_grid_fits(int64_t rows, int64_t vocab);
size_t logprobs_workspace(int64_t rows, int64_t vocab, int top);
size_t distill_workspace(int64_t rows, int64_t vocab, int top);
hipError_t launch_logprobs(int dt, const LogprobArgs& a, void* ws, hipStream_t s);
hipError_t launch_distill(int dt, const DistillArgs& a, void* ws, hipStream_t s);

}  // namespace mo
