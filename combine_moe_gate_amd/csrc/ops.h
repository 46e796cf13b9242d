// Host-side launchers of the router's balance loss and of the expert products with an
// epilogue, shared between their kernels and the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "internal.h"

namespace moe {

// Most workgroups of so many threads in one launch: a grid is counted in 32-bit work items.
constexpr int64_t most_workgroups(int threads) { return UINT32_MAX / threads; }

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
  size_t off_probs, off_counts, off_z, off_tokens, off_dots, off_arrived, bytes;
};
BalancePlan balance_plan(int32_t s, int32_t e, int32_t g);

hipError_t launch_balance_loss(const BalanceArgs& a, const BalancePlan& p, char* ws, int32_t* counts,
                               int32_t* tokens, float* probs, float* loss, float* z, hipStream_t stream);
hipError_t launch_balance_loss_backward(const BalanceArgs& a, const int32_t* counts, const int32_t* tokens,
                                        const float* grad_loss, const float* grad_z, float* grad_logits,
                                        hipStream_t stream);

// ---------------------------------------------------------------------------------
// expert products with an epilogue

enum Act : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4 };

// One grouped product out[r] = w_r act(A(r) W[x]^T + b[x]) + residual(r) (gated: act of the
// first n products times the last n). Element types are 16-bit; nz = 2 n if gated, else n.
struct ExpertAct {
  const void* a;            // [s, m] if gather, else [rows, m]
  const void* w;            // [e, nz, m]
  const void* bias;         // [e, nz] (float32 if bias_f32), or null
  const float* route_w;     // [s, k], or null
  const void* residual;     // [s, n] if residual_gather, else [rows, n], or null
  void* preact;             // [rows, nz] (float32 if preact_f32), or null
  void* out;                // [rows, n]
  const int32_t *dst, *src, *kept, *offsets;
  int32_t e, k, m, n, nz, act;
  int64_t rows;
  bool gather, gated, bias_f32, residual_gather, preact_f32;
};
hipError_t launch_expert_act(const LayoutView& L, const ExpertAct& p, int dtype, hipStream_t stream);
bool expert_act_fits(const LayoutView& L, int n, bool gated);  // whether one launch takes its workgroups
// Its input gradient: out[r] = a[r] @ W[x] with W [e, m, n] (m weight rows, n inputs): the
// struct's a = the gradient rows [rows, m], out [rows, n], nz = n; no epilogue.
hipError_t launch_expert_act_dgrad(const LayoutView& L, const ExpertAct& p, int dtype, hipStream_t stream);
bool expert_act_dgrad_fits(const LayoutView& L, int n);

// Its epilogue's backward (n, nz as above).
struct ExpertActBackward {
  const void* grad_out;     // [rows, n]
  const void* preact;       // [rows, nz] (float32 if preact_f32), or null where nothing needs it
  const float* route_w;     // [s, k], or null
  void* grad_preact;        // [rows, nz], or null
  void* grad_bias;          // [e, nz] (float32 if bias_f32), or null
  float* grad_w;            // [s, k], or null
  void* grad_residual;      // [rows, n], or null
  const int32_t *dst, *src, *kept, *offsets;
  int32_t s, e, k, n, nz, act;
  int64_t rows;
  bool gated, bias_f32, preact_f32;
};
// The workspace: a partial bias row per row tile, a partial dot per row and column block.
struct ExpertActBackwardPlan {
  int32_t col_blocks;
  int32_t shift;  // a tile has 1 << shift rows
  int64_t slots, grid;
  size_t off_bias, off_dots, bytes;
};
ExpertActBackwardPlan expert_act_backward_plan(const LayoutView& L, int n, bool gated);
// Whether its launches, the second with the sums of a bias and of route weights, take their workgroups.
bool expert_act_backward_fits(const LayoutView& L, const ExpertActBackwardPlan& plan, int nz, bool bias, bool weights);
hipError_t launch_expert_act_backward(const LayoutView& L, const ExpertActBackward& p,
                                      const ExpertActBackwardPlan& plan, char* ws, int dtype, hipStream_t stream);

}  // namespace moe
