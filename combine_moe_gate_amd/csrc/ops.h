// Host-side launchers of the router's balance loss and of the expert products with an
// epilogue, shared between their kernels and the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

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

constexpr int kZeroBlocks = 64;  // workgroups that clear rows no route fills

// At most this many row tiles of a height, known without reading the layout: a segment of R
// rows has fewer than R / height + 1.
int64_t row_tiles(const LayoutView& L, int height);

// Dynamic LDS above the 64 KiB default needs the kernel's limit raised, once per device.
hipError_t allow_lds(const void* kernel, int bytes, std::atomic<uint64_t>& done);

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
  void* grad_preact;        // [rows, nz], in two parts [rows, 2, nz] bf16, or null
  void* grad_bias;          // [e, nz] (float32 if bias_f32), or null
  float* grad_w;            // [s, k], or null
  void* grad_residual;      // [rows, n], or null
  const int32_t *dst, *src, *kept, *offsets;
  int32_t s, e, k, n, nz, act;
  int32_t parts;            // of grad_preact: 1 or 2
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

// ---------------------------------------------------------------------------------
// microscaled 4-bit floating point (the format stands in mx4.h)

// `blocks` blocks of 32 values: to 16 bytes of codes and a scale byte each, and back.
hipError_t launch_mx4_quantize(const void* x, int64_t blocks, int dtype, void* codes, void* scales, hipStream_t stream);
hipError_t launch_mx4_dequantize(const void* codes, const void* scales, int64_t blocks, int dtype, void* out,
                                 hipStream_t stream);

// An expert product whose weights are 4-bit: w holds codes [e, nz, m / 2]. With a_scales the rows
// are 4-bit as well (a: codes [.., m / 2]), with out_scales the results (out: codes [rows, n / 2]).
struct Mx4Act : ExpertAct {
  const uint8_t* a_scales;  // [s or rows, m / 32], or null
  const uint8_t* w_scales;  // [e, nz, m / 32]
  uint8_t* out_scales;      // [rows, n / 32], or null
};
hipError_t launch_mx4_act(const LayoutView& L, const Mx4Act& p, int dtype, hipStream_t stream);
bool mx4_act_fits(const LayoutView& L, const Mx4Act& p, int dtype);
// Its form for long segments: tiles of at most so many rows, by 256 weight rows.
constexpr int kMx4TileThreads = 512;
int mx4_tile_rows();
hipError_t launch_mx4_tiles(const Mx4Act& p, int dtype, int col_blocks, int64_t grid, hipStream_t stream);
// Its form for few rows: 16 `few` (1, 2 or, of 4 bits, 4) rows by 128 weight rows; m a multiple of 128,
// scales 4-byte aligned.
constexpr int kMx4StreamThreads = 256;
hipError_t launch_mx4_stream(const Mx4Act& p, int dtype, int few, int col_blocks, int64_t grid, hipStream_t stream);
// Its input gradient: out[r] = a[r] @ W[x] with W [e, m, n] (m weight rows, n inputs): the struct's
// a = the gradient rows [rows, m], or in two bf16 parts [rows, 2, m], out [rows, n], nz = n; no
// epilogue.
struct Mx4Dgrad : Mx4Act {
  int32_t parts;            // of the gradient rows: 1, or 2 (bf16)
  int32_t out_type;
};
hipError_t launch_mx4_dgrad(const LayoutView& L, const Mx4Dgrad& p, int dtype, hipStream_t stream);
bool mx4_dgrad_fits(const LayoutView& L, int n);

}  // namespace moe
