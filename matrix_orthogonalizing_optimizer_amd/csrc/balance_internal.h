// Internal declarations of the router's balance loss.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mo {

constexpr int kMaxExperts = 4096;

struct BalanceArgs {
  const void* logits;
  int64_t ld, ld_grad;
  int64_t tokens;
  int experts, top;
  const int64_t* index;         // [tokens][top]
  float weight;
  const float* grad_loss;       // or null
  float* loss;
  int64_t* counts;
  void* grad;                   // or null
  int accumulate;
};

size_t balance_workspace(int64_t tokens, int experts);
hipError_t launch_balance(int dt, const BalanceArgs& a, void* ws, hipStream_t s);

}  // namespace mo
