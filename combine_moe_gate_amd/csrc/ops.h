// Host-side launchers of the router's balance loss and of the expert products with an
// epilogue, shared between their kernels and the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "internal.h"

namespace moe {

// ---------------------------------------------------------------------------------
// balance loss

struct BalanceArgs {
  const float* logits;     // [s, e]
  const int32_t* idx;      // [s, k]
  const uint8_t* mask;     // [s] (0: padded token), or null
  const int32_t* groups;   // [g + 1] first token of each group, or null (g = 1: all tokens)
  int32_t s, e, k, g;
};

// Tiles of tokens the forward is cut into, and where their partial sums lie in the
// workspace. A tile and a group that meet own the partial row `tile + group`: both only
// grow along the tokens, so no two meetings share one.
struct BalancePlan {
  int32_t tile, ntiles, pitch, chunks;
  int64_t slots;
  size_t off_probs, off_counts, off_z, off_tokens, off_dots, bytes;
};
BalancePlan balance_plan(int32_t s, int32_t e, int32_t g);

hipError_t launch_balance_loss(const BalanceArgs& a, const BalancePlan& p, char* ws, int32_t* counts,
                               int32_t* tokens, float* probs, float* loss, float* z, hipStream_t stream);
hipError_t launch_balance_loss_backward(const BalanceArgs& a, const int32_t* counts, const int32_t* tokens,
                                        const float* grad_loss, const float* grad_z, float* grad_logits,
                                        hipStream_t stream);

}  // namespace moe
