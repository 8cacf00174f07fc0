// Declarations of the operators around the layer: the whole layer for a few
// tokens (decode.cu, decode_tc.cu), the layer norm (norm.cu) and the
// counter-based dropout (dropout.cu).  Their C entry points are in block_api.cu.
#pragma once

#include "internal.h"

namespace moe {

// Kernel kinds of launch accounting, after those of internal.h.
enum BlockKernelKind : int {
  KK_DECODE = KK_COUNT,
  KK_NORM_FWD,
  KK_NORM_BWD,
  KK_NORM_BWD_REDUCE,
  KK_DROPOUT_ADD,
  KK_DROPOUT_BWD,
  KK_ALL
};

int sm_count();  // of the current device; 152 where there is none (host-side sizing)

// ---- decode.cu: the layer for at most MOE_DECODE_MAX_T tokens in one kernel ----
struct DecodeIo {
  const void* x;
  const float* W_r;
  const float* bias;  // or null
  const void* W1;
  const void* W3;
  const void* W2;
  const void* residual;  // [T, d] added to y, or null
  void* y;
  int32_t* ids;  // [T, k] or null
  float* gates;  // [T, k] or null
};
size_t decode_ws_bytes(const Shape& s);
cudaError_t launch_decode(const Shape& s, const DecodeIo& io, void* ws, uint32_t* err, cudaStream_t st);

// ---- norm.cu ----
cudaError_t launch_norm_fwd(int64_t rows, int d, bool bf16, const void* x, const float* gamma, const float* beta,
                            float eps, void* y, float* mean, float* rstd, uint32_t* err, cudaStream_t st);
size_t norm_ws_bytes(int64_t rows, int d);
cudaError_t launch_norm_bwd(int64_t rows, int d, bool bf16, const void* x, const void* dy, const float* gamma,
                            const float* mean, const float* rstd, const void* dres, void* dx, float* dgamma,
                            float* dbeta, int accumulate, void* ws, uint32_t* err, cudaStream_t st);

// ---- dropout.cu ----
cudaError_t launch_dropout(int kind, int64_t n, bool bf16, const void* y, const void* residual, void* out,
                           uint32_t cut, uint64_t seed, uint64_t offset, cudaStream_t st);

}  // namespace moe
