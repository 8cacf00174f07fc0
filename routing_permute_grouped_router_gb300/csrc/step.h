// Declarations of the operators that join blocks to a training step: the
// residual path between blocks (residual_norm.cu), gradient clipping
// (clip.cu) and the vocabulary loss (vocab_loss.cu).  Their C entry points
// are in step_api.cu.
#pragma once

#include "../../include/moe.h"
#include "block.h"

namespace moe {

// Kernel kinds of launch accounting, after those of block.h.
enum StepKernelKind : int {
  KK_RESIDUAL_NORM_FWD = KK_ALL,
  KK_RESIDUAL_NORM_BWD,
  KK_RESIDUAL_NORM_REDUCE,
  KK_GRAD_NORM,
  KK_GRAD_CLIP,
  KK_LOSS_ROWS,
  KK_LOSS_LOGITS,
  KK_LOSS_COMBINE,
  KK_LOSS_DLOGITS,
  KK_LOSS_GRADS,
  KK_LOSS_FINISH,
  KK_END
};

// Codes of the device error word, after those of internal.h.
constexpr uint32_t DEV_BAD_LABEL = 6;  // a label >= V

// ---- residual_norm.cu ----
struct JoinArgs {
  moe_residual_norm p;
  const void* x;
  const void* y;
  void* out;         // the backward reads it
  void* h;
  float* rstd_post;  // the backward reads them
  float* rstd_next;
  const void* dh;
  const void* dout;
  void* dx;
  void* dy;
  moe_residual_norm_grads g;
  int accumulate;
  void* ws;
};
size_t join_ws_bytes(int64_t rows, int d);
cudaError_t launch_join_fwd(const JoinArgs& a, uint32_t* err, cudaStream_t st);
cudaError_t launch_join_bwd(const JoinArgs& a, uint32_t* err, cudaStream_t st);

// ---- clip.cu ----
size_t clip_ws_bytes(int count);
cudaError_t launch_clip(const moe_grad* grads, int count, float max_norm, float* norm, void* ws, cudaStream_t st);

// ---- vocab_loss.cu ----
struct LossArgs {
  int T, d, V;
  bool bf16, dw_bf16;
  const void* x;
  const void* W;
  const int32_t* labels;
  float* loss;
  float* lse;         // the backward reads it
  float* total;       // [2] or null
  const float* dloss; // [T] or null
  void* dx;           // or null
  void* dW;           // or null
  int accumulate;
  void* ws;
};
size_t loss_ws_bytes(int T, int d, int V, bool bf16, bool training);
cudaError_t launch_loss_fwd(const LossArgs& a, uint32_t* err, cudaStream_t st);
cudaError_t launch_loss_bwd(const LossArgs& a, uint32_t* err, cudaStream_t st);

}  // namespace moe
