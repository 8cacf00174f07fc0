// C entry points of the operators that join blocks to a training step:
// argument checks and the launchers of residual_norm.cu, clip.cu and
// vocab_loss.cu.  Contracts are in moe.h.
#include <algorithm>
#include <cmath>
#include <mutex>

#include "step.h"

namespace moe {
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

bool known(int32_t dtype) { return dtype == MOE_F32 || dtype == MOE_BF16; }

moe_status rows_shape(int64_t rows, int32_t d) {
  return rows < 0 || d < 1 || d > (1 << 16) || rows > ((int64_t)1 << 40) / d ? MOE_ERR_SHAPE : MOE_OK;
}

moe_status join_shape(const moe_residual_norm* p) {
  if (p == nullptr) return MOE_ERR_INVALID_ARG;
  if (!known(p->dtype)) return MOE_ERR_DTYPE;
  MOE_TRY(rows_shape(p->rows, p->d));
  if (!std::isfinite(p->eps) || p->eps < 0.f || !std::isfinite(p->residual_scale) || !std::isfinite(p->branch_scale))
    return MOE_ERR_INVALID_ARG;
  MOE_TRY(may(p->gamma_post, 4));
  MOE_TRY(may(p->gamma_next, 4));
  MOE_TRY(may(p->gate, 4));
  return may(p->row_gate, 4);
}

// Whether a tensor that is written overlaps another one.
struct Span {
  uintptr_t at, end;
  bool written;
  bool operator<(const Span& o) const { return at < o.at; }
};
// Sorted by merging the ascending runs that are there: lists come in the order of
// their buffers, often two runs (300 tensors: 4 us of a call, std::sort 12).
Span* sort_runs(Span* s, Span* other, int n) {
  for (;;) {
    int at = 0, runs = 0;
    while (at < n) {
      int mid = at + 1;
      while (mid < n && !(s[mid] < s[mid - 1])) ++mid;
      int end = mid < n ? mid + 1 : mid;
      while (end < n && !(s[end] < s[end - 1])) ++end;
      std::merge(s + at, s + mid, s + mid, s + end, other + at);
      at = end;
      ++runs;
    }
    std::swap(s, other);
    if (runs <= 1) return s;
  }
}
// Its lists of spans are the library's own, one set behind a lock (300 tensors hold
// it for 4 us): host memory is not allocated either.  Short lists are on the stack.
constexpr int FEW_SPANS = 32;
Span g_spans[4 * (size_t)MOE_CLIP_MAX_TENSORS];
std::mutex g_spans_mu;
moe_status check_overlap(const moe_grad* g, int32_t count) {
  Span few[4 * FEW_SPANS];
  std::unique_lock<std::mutex> lk(g_spans_mu, std::defer_lock);
  Span* s = few;
  if (count > FEW_SPANS) {
    lk.lock();
    s = g_spans;
  }
  int n = 0;
  bool any = false;
  for (int i = 0; i < count; ++i) {  // the sources, then the destinations
    if (g[i].n == 0) continue;
    const uintptr_t src = reinterpret_cast<uintptr_t>(g[i].src);
    any = any || g[i].dst != nullptr;
    s[n++] = {src, src + (uintptr_t)g[i].n * (g[i].dtype == MOE_BF16 ? 2 : 4), g[i].dst == g[i].src};
  }
  for (int i = 0; i < count; ++i) {
    if (g[i].n == 0 || g[i].dst == nullptr || g[i].dst == g[i].src) continue;
    const uintptr_t dst = reinterpret_cast<uintptr_t>(g[i].dst);
    s[n++] = {dst, dst + (uintptr_t)g[i].n * (g[i].dtype == MOE_BF16 ? 2 : 4), true};
  }
  moe_status st = MOE_OK;
  if (any) {
    const Span* v = sort_runs(s, s + n, n);
    uintptr_t end = 0, written_end = 0;  // of the tensors before, and of the written ones among them
    for (int i = 0; i < n; ++i) {
      if (v[i].at < written_end || (v[i].written && v[i].at < end)) st = MOE_ERR_INVALID_ARG;
      end = std::max(end, v[i].end);
      if (v[i].written) written_end = std::max(written_end, v[i].end);
    }
  }
  return st;
}

moe_status loss_shape(int32_t T, int32_t d, int32_t V, int32_t dtype) {
  if (!known(dtype)) return MOE_ERR_DTYPE;
  if (T < 0 || T > (1 << 24) || V < 1 || V > (1 << 24) || d < 1 || d > (1 << 16)) return MOE_ERR_SHAPE;
  if ((int64_t)T * V > (int64_t)1 << 44) return MOE_ERR_SHAPE;
  return d % (dtype == MOE_BF16 ? 8 : 4) == 0 ? MOE_OK : MOE_ERR_SHAPE;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_residual_norm_fwd(const moe_residual_norm* p, const void* x, const void* y, void* out, void* h,
                                 float* rstd_post, float* rstd_next, moe_stream_t stream) {
  MOE_TRY(join_shape(p));
  // a norm or a gate of a branch that is not there, h without its weight, nothing to write
  if (y == nullptr && p->rows > 0 && (p->gamma_post || p->gate || p->row_gate)) return MOE_ERR_INVALID_ARG;
  if ((!p->gamma_post && rstd_post) || (!p->gamma_next && (rstd_next || h))) return MOE_ERR_INVALID_ARG;
  if (p->rows > 0) {
    MOE_TRY(need(x));
    if (p->gamma_next) MOE_TRY(need(h));
    if (!out && !h) return MOE_ERR_INVALID_ARG;
    if (out == h) return MOE_ERR_INVALID_ARG;
  }
  MOE_TRY(may(y));
  MOE_TRY(may(out));
  MOE_TRY(may(rstd_post, 4));
  MOE_TRY(may(rstd_next, 4));
  uint32_t* err = nullptr;
  MOE_TRY(current_error_word(&err));
  if (p->rows == 0) return MOE_OK;
  JoinArgs a{};
  a.p = *p;
  a.x = x;
  a.y = y;
  a.out = out;
  a.h = h;
  a.rstd_post = rstd_post;
  a.rstd_next = rstd_next;
  CUDA_TRY(launch_join_fwd(a, err, stream));
  return MOE_OK;
}

moe_status moe_residual_norm_workspace_size(int64_t rows, int32_t d, size_t* bytes) {
  MOE_TRY(rows_shape(rows, d));
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = join_ws_bytes(rows, d) + 256;
  return MOE_OK;
}

moe_status moe_residual_norm_bwd(const moe_residual_norm* p, const void* out, const void* y, const void* dh,
                                 const void* dout, const float* rstd_post, const float* rstd_next, void* dx, void* dy,
                                 const moe_residual_norm_grads* grads, int accumulate, void* ws, size_t ws_bytes,
                                 moe_stream_t stream) {
  MOE_TRY(join_shape(p));
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
  const moe_residual_norm_grads g = grads ? *grads : moe_residual_norm_grads{};
  if ((g.dgamma_post && !p->gamma_post) || (g.dgamma_next && !p->gamma_next) || (g.dgate && !p->gate) ||
      (g.drow_gate && !p->row_gate))
    return MOE_ERR_INVALID_ARG;
  if (p->rows > 0) {
    if ((y == nullptr) != (dy == nullptr)) return MOE_ERR_INVALID_ARG;
    if (y == nullptr && (p->gamma_post || p->gate || p->row_gate)) return MOE_ERR_INVALID_ARG;
    if ((p->gamma_next == nullptr) != (dh == nullptr)) return MOE_ERR_INVALID_ARG;
    if (!dh && !dout) return MOE_ERR_INVALID_ARG;
    if (dx && dx == dy) return MOE_ERR_INVALID_ARG;
    if (p->gamma_next) {
      MOE_TRY(need(out));
      MOE_TRY(need(rstd_next, 4));
    }
    if (p->gamma_post) MOE_TRY(need(rstd_post, 4));
    MOE_TRY(may(y));
    MOE_TRY(may(dh));
    MOE_TRY(may(dout));
    MOE_TRY(may(dx));
    MOE_TRY(may(dy));
  }
  MOE_TRY(may(g.dgamma_post, 4));
  MOE_TRY(may(g.dgamma_next, 4));
  MOE_TRY(may(g.dgate, 4));
  MOE_TRY(may(g.drow_gate, 4));
  if (ws == nullptr || ws_bytes < join_ws_bytes(p->rows, p->d) + 256) return MOE_ERR_WORKSPACE;
  uint32_t* err = nullptr;
  MOE_TRY(current_error_word(&err));
  if (p->rows == 0) {
    if (accumulate) return MOE_OK;
    for (float* v : {g.dgamma_post, g.dgamma_next, g.dgate})
      if (v) CUDA_TRY(cudaMemsetAsync(v, 0, (size_t)p->d * 4, stream));
    return MOE_OK;
  }
  JoinArgs a{};
  a.p = *p;
  a.y = y;
  a.out = const_cast<void*>(out);
  a.dh = dh;
  a.dout = dout;
  a.rstd_post = const_cast<float*>(rstd_post);
  a.rstd_next = const_cast<float*>(rstd_next);
  a.dx = dx;
  a.dy = dy;
  a.g = g;
  a.accumulate = accumulate;
  a.ws = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(ws) + 255) / 256 * 256);
  CUDA_TRY(launch_join_bwd(a, err, stream));
  return MOE_OK;
}

moe_status moe_clip_workspace_size(int32_t count, size_t* bytes) {
  if (count < 0 || count > MOE_CLIP_MAX_TENSORS) return MOE_ERR_SHAPE;
  if (bytes == nullptr) return MOE_ERR_INVALID_ARG;
  *bytes = clip_ws_bytes(count) + 256;
  return MOE_OK;
}

moe_status moe_clip_grads(const moe_grad* grads, int32_t count, float max_norm, float* norm, void* ws, size_t ws_bytes,
                          moe_stream_t stream) {
  if (count < 0 || count > MOE_CLIP_MAX_TENSORS) return MOE_ERR_SHAPE;
  if (!(max_norm > 0.f)) return MOE_ERR_INVALID_ARG;  // NaN too
  if (count > 0 && grads == nullptr) return MOE_ERR_INVALID_ARG;
  MOE_TRY(need(norm, 4));
  for (int i = 0; i < count; ++i) {
    if (!known(grads[i].dtype)) return MOE_ERR_DTYPE;
    if (grads[i].n < 0 || grads[i].n > ((int64_t)1 << 40)) return MOE_ERR_SHAPE;
    const size_t es = grads[i].dtype == MOE_BF16 ? 2 : 4;
    if (grads[i].n > 0) {
      MOE_TRY(need(grads[i].src, es));
      MOE_TRY(may(grads[i].dst, es));
    }
  }
  if (ws == nullptr || ws_bytes < clip_ws_bytes(count) + 256) return MOE_ERR_WORKSPACE;
  MOE_TRY(check_overlap(grads, count));
  uint32_t* err = nullptr;
  MOE_TRY(current_error_word(&err));
  void* base = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(ws) + 255) / 256 * 256);
  CUDA_TRY(launch_clip(grads, count, max_norm, norm, base, stream));
  return MOE_OK;
}

moe_status moe_vocab_loss_workspace_size(int32_t T, int32_t d, int32_t V, int32_t dtype, int training, size_t* bytes) {
  MOE_TRY(loss_shape(T, d, V, dtype));
  if (bytes == nullptr || (training != 0 && training != 1)) return MOE_ERR_INVALID_ARG;
  *bytes = loss_ws_bytes(T, d, V, dtype == MOE_BF16, training != 0) + 256;
  return MOE_OK;
}

moe_status moe_vocab_loss_fwd(int32_t T, int32_t d, int32_t V, int32_t dtype, const void* x, const void* W,
                              const int32_t* labels, float* loss, float* lse, float* total, void* ws, size_t ws_bytes,
                              moe_stream_t stream) {
  MOE_TRY(loss_shape(T, d, V, dtype));
  if (T > 0) {
    MOE_TRY(need(x));
    MOE_TRY(need(labels, 4));
    MOE_TRY(need(loss, 4));
    MOE_TRY(need(lse, 4));
  }
  MOE_TRY(need(W));
  MOE_TRY(may(total, 4));
  if (ws == nullptr || ws_bytes < loss_ws_bytes(T, d, V, dtype == MOE_BF16, false) + 256) return MOE_ERR_WORKSPACE;
  uint32_t* err = nullptr;
  MOE_TRY(current_error_word(&err));
  if (T == 0) {
    if (total) CUDA_TRY(cudaMemsetAsync(total, 0, 8, stream));
    return MOE_OK;
  }
  LossArgs a{};
  a.T = T;
  a.d = d;
  a.V = V;
  a.bf16 = dtype == MOE_BF16;
  a.x = x;
  a.W = W;
  a.labels = labels;
  a.loss = loss;
  a.lse = lse;
  a.total = total;
  a.ws = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(ws) + 255) / 256 * 256);
  CUDA_TRY(launch_loss_fwd(a, err, stream));
  return MOE_OK;
}

moe_status moe_vocab_loss_bwd(int32_t T, int32_t d, int32_t V, int32_t dtype, int32_t dw_dtype, const void* x,
                              const void* W, const int32_t* labels, const float* lse, const float* dloss, void* dx,
                              void* dW, int accumulate, void* ws, size_t ws_bytes, moe_stream_t stream) {
  MOE_TRY(loss_shape(T, d, V, dtype));
  if (!known(dw_dtype) || (dtype == MOE_F32 && dw_dtype != MOE_F32)) return MOE_ERR_DTYPE;
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
  if (T > 0) {
    if (dx == nullptr && dW == nullptr) return MOE_ERR_INVALID_ARG;
    MOE_TRY(need(x));
    MOE_TRY(need(labels, 4));
    MOE_TRY(need(lse, 4));
  }
  MOE_TRY(need(W));
  MOE_TRY(may(dloss, 4));
  MOE_TRY(may(dx));
  MOE_TRY(may(dW));
  if (ws == nullptr || ws_bytes < loss_ws_bytes(T, d, V, dtype == MOE_BF16, true) + 256) return MOE_ERR_WORKSPACE;
  uint32_t* err = nullptr;
  MOE_TRY(current_error_word(&err));
  if (T == 0) {
    if (dW && !accumulate) CUDA_TRY(cudaMemsetAsync(dW, 0, (size_t)V * d * (dw_dtype == MOE_BF16 ? 2 : 4), stream));
    return MOE_OK;
  }
  LossArgs a{};
  a.T = T;
  a.d = d;
  a.V = V;
  a.bf16 = dtype == MOE_BF16;
  a.dw_bf16 = dw_dtype == MOE_BF16;
  a.x = x;
  a.W = W;
  a.labels = labels;
  a.lse = const_cast<float*>(lse);
  a.dloss = dloss;
  a.dx = dx;
  a.dW = dW;
  a.accumulate = accumulate;
  a.ws = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(ws) + 255) / 256 * 256);
  CUDA_TRY(launch_loss_bwd(a, err, stream));
  return MOE_OK;
}

}  // extern "C"
