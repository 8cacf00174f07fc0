// C entry points of the operators around the layer: argument checks and the
// launchers of decode.cu, norm.cu and dropout.cu.  Contracts are in moe.h.
#include <cmath>

#include "../../include/moe.h"
#include "block.h"

namespace moe {

int sm_count() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  if (cached[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 152;
    cached[dev] = n;
  }
  return cached[dev];
}

namespace {

moe_status need(const void* p, size_t a = 16) {
  if (p == nullptr) return MOE_ERR_INVALID_ARG;
  return reinterpret_cast<uintptr_t>(p) % a == 0 ? MOE_OK : MOE_ERR_ALIGNMENT;
}
moe_status may(const void* p, size_t a = 16) { return p == nullptr ? MOE_OK : need(p, a); }

#define MOE_TRY(expr)                                       \
  do {                                                      \
    const moe_status st_ = static_cast<moe_status>(expr);   \
    if (st_ != MOE_OK) return st_;                          \
  } while (0)
#define CUDA_TRY(expr)                              \
  do {                                              \
    if ((expr) != cudaSuccess) return MOE_ERR_CUDA; \
  } while (0)

moe_status decode_shape(const moe_config* cfg, Shape* s) {
  MOE_TRY(validate_config(cfg, s));
  return s->T <= MOE_DECODE_MAX_T ? MOE_OK : MOE_ERR_SHAPE;
}

moe_status rows_shape(int64_t rows, int32_t d, int32_t dtype) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_DTYPE;
  if (rows < 0 || d < 1 || d > (1 << 16) || rows > ((int64_t)1 << 40) / d) return MOE_ERR_SHAPE;
  return MOE_OK;
}

// The 16-bit cut of dropout probability p: draws below it are dropped.
moe_status drop_cut(float p, uint32_t* cut) {
  if (!(p >= 0.f) || !(p < 1.f)) return MOE_ERR_INVALID_ARG;  // NaN too
  *cut = (uint32_t)std::floor((double)p * 65536.0 + 0.5);
  return *cut < 65536u ? MOE_OK : MOE_ERR_INVALID_ARG;  // p rounds to 1: nothing would be kept
}

moe_status elements(int64_t n, int32_t dtype) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_DTYPE;
  return n >= 0 && n <= ((int64_t)1 << 40) ? MOE_OK : MOE_ERR_SHAPE;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_decode_workspace_size(const moe_config* cfg, size_t* bytes) {
  Shape s;
  MOE_TRY(decode_shape(cfg, &s));
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = decode_ws_bytes(s);
  return MOE_OK;
}

moe_status moe_layer_decode(const moe_config* cfg, const moe_weights* w, const void* x, const void* residual, void* y,
                            int32_t* ids, float* gates, void* ws, size_t ws_bytes, moe_stream_t stream) {
  Shape s;
  MOE_TRY(decode_shape(cfg, &s));
  if (w == nullptr) return MOE_ERR_INVALID_ARG;
  if (s.T > 0) {
    MOE_TRY(need(x));
    MOE_TRY(need(y));
  }
  MOE_TRY(need(w->W_r, 4));
  MOE_TRY(may(w->bias, 4));
  MOE_TRY(need(w->W1));
  MOE_TRY(need(w->W3));
  MOE_TRY(need(w->W2));
  MOE_TRY(may(residual));
  MOE_TRY(may(ids, 4));
  MOE_TRY(may(gates, 4));
  if (ws == nullptr || ws_bytes < decode_ws_bytes(s)) return MOE_ERR_WORKSPACE;
  uint32_t* err = nullptr;
  MOE_TRY(current_error_word(&err));
  if (s.T == 0) return MOE_OK;
  const DecodeIo io{x, w->W_r, w->bias, w->W1, w->W3, w->W2, residual, y, ids, gates};
  CUDA_TRY(launch_decode(s, io, ws, err, stream));
  return MOE_OK;
}

moe_status moe_norm_fwd(int64_t rows, int32_t d, int32_t dtype, const void* x, const float* gamma, const float* beta,
                        float eps, void* y, float* mean, float* rstd, moe_stream_t stream) {
  MOE_TRY(rows_shape(rows, d, dtype));
  if (!std::isfinite(eps) || eps < 0.f) return MOE_ERR_INVALID_ARG;
  if (rows > 0) {
    MOE_TRY(need(x));
    MOE_TRY(need(y));
  }
  MOE_TRY(need(gamma, 4));
  MOE_TRY(need(beta, 4));
  MOE_TRY(may(mean, 4));
  MOE_TRY(may(rstd, 4));
  uint32_t* err = nullptr;
  MOE_TRY(current_error_word(&err));
  if (rows == 0) return MOE_OK;
  CUDA_TRY(launch_norm_fwd(rows, d, dtype == MOE_BF16, x, gamma, beta, eps, y, mean, rstd, err, stream));
  return MOE_OK;
}

moe_status moe_norm_workspace_size(int64_t rows, int32_t d, size_t* bytes) {
  MOE_TRY(rows_shape(rows, d, MOE_F32));
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = norm_ws_bytes(rows, d) + 256;
  return MOE_OK;
}

moe_status moe_norm_bwd(int64_t rows, int32_t d, int32_t dtype, const void* x, const void* dy, const float* gamma,
                        const float* mean, const float* rstd, const void* dres, void* dx, float* dgamma, float* dbeta,
                        int accumulate, void* ws, size_t ws_bytes, moe_stream_t stream) {
  MOE_TRY(rows_shape(rows, d, dtype));
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
  if (rows > 0) {
    MOE_TRY(need(x));
    MOE_TRY(need(dy));
    MOE_TRY(need(dx));
    MOE_TRY(need(mean, 4));
    MOE_TRY(need(rstd, 4));
  }
  MOE_TRY(need(gamma, 4));
  MOE_TRY(may(dres));
  MOE_TRY(need(dgamma, 4));
  MOE_TRY(need(dbeta, 4));
  if (ws == nullptr || ws_bytes < norm_ws_bytes(rows, d) + 256) return MOE_ERR_WORKSPACE;
  uint32_t* err = nullptr;
  MOE_TRY(current_error_word(&err));
  if (rows == 0) {
    if (accumulate) return MOE_OK;
    CUDA_TRY(cudaMemsetAsync(dgamma, 0, (size_t)d * 4, stream));
    CUDA_TRY(cudaMemsetAsync(dbeta, 0, (size_t)d * 4, stream));
    return MOE_OK;
  }
  void* base = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(ws) + 255) / 256 * 256);
  CUDA_TRY(launch_norm_bwd(rows, d, dtype == MOE_BF16, x, dy, gamma, mean, rstd, dres, dx, dgamma, dbeta, accumulate,
                           base, err, stream));
  return MOE_OK;
}

moe_status moe_dropout_add(int64_t n, int32_t dtype, const void* y, const void* residual, void* out, float p,
                           uint64_t seed, uint64_t offset, moe_stream_t stream) {
  uint32_t cut = 0, *err = nullptr;
  MOE_TRY(elements(n, dtype));
  MOE_TRY(drop_cut(p, &cut));
  if (n > 0) {
    MOE_TRY(need(y));
    MOE_TRY(need(out));
  }
  MOE_TRY(may(residual));
  MOE_TRY(current_error_word(&err));
  if (n == 0) return MOE_OK;
  CUDA_TRY(launch_dropout(KK_DROPOUT_ADD, n, dtype == MOE_BF16, y, residual, out, cut, seed, offset, stream));
  return MOE_OK;
}

moe_status moe_dropout_bwd(int64_t n, int32_t dtype, const void* dout, void* dy, float p, uint64_t seed,
                           uint64_t offset, moe_stream_t stream) {
  uint32_t cut = 0, *err = nullptr;
  MOE_TRY(elements(n, dtype));
  MOE_TRY(drop_cut(p, &cut));
  if (n > 0) {
    MOE_TRY(need(dout));
    MOE_TRY(need(dy));
  }
  MOE_TRY(current_error_word(&err));
  if (n == 0) return MOE_OK;
  CUDA_TRY(launch_dropout(KK_DROPOUT_BWD, n, dtype == MOE_BF16, dout, nullptr, dy, cut, seed, offset, stream));
  return MOE_OK;
}

}  // extern "C"
