// What the parts of the vocabulary loss share: the token lists and epilogue data
// that vocab_loss.cu prepares, the products of vocab_loss_tc.cu, and the form
// for few tokens.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "step.h"

namespace moe {

constexpr int LOSS_TILE = 256;   // rows and columns of a product's tile
constexpr int LOSS_PART = 128;   // columns of a partial sum of the forward
constexpr int MAX_PARTS = 3;     // bf16 parts of a float32 value

// What logits are measured from in a sum of exponentials: their maximum, or the
// finite value next to it.  So an infinite logit adds infinity (measured from
// itself it would be a NaN), and -inf adds 0 among nothing but -inf too.
__device__ __forceinline__ float base_of(float best) { return fminf(fmaxf(best, -3.402823466e38f), 3.402823466e38f); }

// ---- vocab_loss_few.cu: the forward of at most LOSS_FEW tokens, in the workspace's first bytes ----
constexpr int LOSS_FEW = 64;
bool loss_is_few(int T, int d, bool bf16);  // float32: fewer
size_t loss_few_bytes();
cudaError_t launch_loss_few(const LossArgs& a, uint32_t* err, cudaStream_t st);

// ---- vocab_loss_tc.cu ----
// 2-D tensor map over a row-major [rows, cols] matrix, 128-byte swizzle; what a box
// has past it reads as 0.  maps_ready: the driver's encoder was found.
bool maps_ready();
bool make_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_cols, uint32_t box_rows,
              bool fp32 = false);
// Labelled tokens only, in token order, padded with zero rows to a whole tile.
struct LossWork {
  int32_t* list;    // [T]: the labelled tokens
  int32_t* pos;     // [T]: a token's place among them, -1 for the others
  int32_t* count;   // their number
  int32_t* label;   // [Tp], of the labelled tokens; -1 on padding
  float* picked;    // [Tp]: the label's logit
  float* lse;       // [Tp]
  float* grad;      // [Tp]: the gradient that reaches the token's loss
  float* off;       // [Tp]: what the first part of dz leaves of the label's
  __nv_bfloat16* xp;  // [Tp][parts][ldx]: the labelled rows of x
  const __nv_bfloat16* wp;  // [V][parts][ldw]: W itself, or its parts
  float2* partial;  // [V / LOSS_PART, whole tiles][Tp]: the largest logit and the sum of exp of the distances to it
  __nv_bfloat16* dz;  // [dz parts][Tp][piece]
  float* acc;       // [slices][Tp][d]: dx before its rounding
  int slices;       // of each piece, summed apart where dx alone has too few tiles
  int T, Tp, d, V, parts, ldx, ldw;
  int mean;         // that gradient is 1 / count for every token: dz goes without it, dx and dW get it at the end
  int v0, piece, dzp;  // the piece of the vocabulary in work; bf16 parts of dz
  uint32_t* err;
};

// Logits of all labelled tokens, tile by tile: partial and picked.
cudaError_t tc_loss_logits(const LossWork& w, cudaStream_t st);
// Logits of a piece again, and from them dz.
cudaError_t tc_loss_dlogits(const LossWork& w, cudaStream_t st);
// acc (+)= dz W (dx), dW[piece] (+)= dz^T x (dW not null); acc is overwritten by the first piece.
cudaError_t tc_loss_grads(const LossWork& w, bool dx, void* dW, bool dw_bf16, bool accumulate, cudaStream_t st);

}  // namespace moe
