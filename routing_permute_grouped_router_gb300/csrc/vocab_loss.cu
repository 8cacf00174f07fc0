// Softmax cross entropy over a large vocabulary and its gradient, the logits
// formed a piece at a time and never kept; formulas are in moe.h.
//
// The labelled tokens are listed first (ignored ones cost nothing further).
#include "common.cuh"
#include "step.h"

namespace moe {
namespace {

constexpr int LIST_NT = 1024;
constexpr int TM = 64, TN = 64, TK = 16, GEMM_NT = 256;  // a tile: 4 x 4 of it a thread
constexpr int64_t PIECE_VALUES = (int64_t)1 << 26;        // values of dz held at a time

struct LossK {
  const void *x, *W;
  const int32_t* labels;
  float *loss, *lse, *total;
  const float* dloss;
  void *dx, *dW;
  int T, d, V, accumulate, dw_bf16;
  // workspace
  int32_t* list;    // [T]: the labelled tokens
  int32_t* count;   // their number
  float2* partial;  // [T][tiles]: the largest logit of each tile and the sum of exp of the distances to it
  float* picked;    // [T]: the label's logit
  float* dz;        // [T][piece]
  float* acc;       // [T][d]: dx before its rounding
  int v0, piece, tiles;
  uint32_t* err;
};

// The labelled tokens in order, and their number.
__global__ void __launch_bounds__(LIST_NT) loss_rows_kernel(const LossK a) {
  pdl_enter();
  __shared__ int before[32];
  __shared__ int base;
  if (threadIdx.x == 0) base = 0;
  __syncthreads();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  for (int t0 = 0; t0 < a.T; t0 += LIST_NT) {
    const int t = t0 + threadIdx.x;
    const int label = t < a.T ? a.labels[t] : -1;
    if (label >= a.V) report_error(a.err, DEV_BAD_LABEL, (uint32_t)t & 0xFFFFFFu);
    const bool valid = label >= 0 && label < a.V;
    const uint32_t votes = __ballot_sync(0xffffffffu, valid);
    if (lane == 0) before[warp] = __popc(votes);
    __syncthreads();
    int at = base, all = 0;
    for (int w = 0; w < LIST_NT / 32; ++w) {
      at += w < warp ? before[w] : 0;
      all += before[w];
    }
    if (valid) a.list[at + __popc(votes & ((1u << lane) - 1u))] = t;
    __syncthreads();
    if (threadIdx.x == 0) base += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) *a.count = base;
}

// c[4][4] of a 64 x 64 tile of A B, A(m, k) and B(n, k) read through fa and fb (0 outside)
template <typename FA, typename FB>
__device__ __forceinline__ void tile_product(int K, FA fa, FB fb, float (&c)[4][4]) {
  __shared__ float sa[TK][TM + 4], sb[TK][TN + 4];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) c[i][j] = 0.f;
  for (int k0 = 0; k0 < K; k0 += TK) {
    __syncthreads();
#pragma unroll
    for (int e = threadIdx.x; e < TM * TK; e += GEMM_NT) {
      sa[e % TK][e / TK] = k0 + e % TK < K ? fa(e / TK, k0 + e % TK) : 0.f;
      sb[e % TK][e / TK] = k0 + e % TK < K ? fb(e / TK, k0 + e % TK) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < TK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i][j] = fmaf(sa[k][ty * 4 + i], sb[k][tx * 4 + j], c[i][j]);
  }
}

// The logits of a tile: their maximum and sum (GRAD: dz instead).
template <typename T, bool GRAD>
__global__ void __launch_bounds__(GEMM_NT) loss_logits_kernel(const LossK a) {
  pdl_enter();
  const int n = *a.count, r0 = blockIdx.y * TM, c0 = blockIdx.x * TN;  // of the labelled tokens, of the piece
  if (r0 >= n) return;
  const T *x = static_cast<const T*>(a.x), *W = static_cast<const T*>(a.W);
  float c[4][4];
  tile_product(
      a.d,
      [&](int m, int k) { return r0 + m < n ? to_f32(x[(int64_t)a.list[r0 + m] * a.d + k]) : 0.f; },
      [&](int v, int k) { return c0 + v < a.piece && a.v0 + c0 + v < a.V ? to_f32(W[(int64_t)(a.v0 + c0 + v) * a.d + k]) : 0.f; }, c);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = r0 + ty * 4 + i;
    const int t = r < n ? a.list[r] : 0, label = r < n ? a.labels[t] : -1;
    if (GRAD) {
      const float g = r < n ? (a.dloss ? a.dloss[t] : 1.f / (float)n) : 0.f, lse = r < n ? a.lse[t] : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int v = c0 + tx * 4 + j;
        if (r < n && v < a.piece)
          a.dz[(int64_t)r * a.piece + v] =
              a.v0 + v < a.V ? g * (expf(c[i][j] - lse) - (a.v0 + v == label ? 1.f : 0.f)) : 0.f;
      }
    } else {
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int v = c0 + tx * 4 + j;
        if (v >= a.V) continue;
        top = fmaxf(top, c[i][j]);
        if (v == label) a.picked[r] = c[i][j];
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      const float from = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c0 + tx * 4 + j < a.V) sum += expf(c[i][j] - from);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (tx == 0 && r < n) a.partial[(int64_t)r * a.tiles + blockIdx.x] = make_float2(top, sum);
    }
  }
}

// A warp for each labelled token: its tiles' sums, its loss.
__global__ void __launch_bounds__(256) loss_combine_kernel(const LossK a) {
  pdl_enter();
  const int n = *a.count, lane = threadIdx.x % 32;
  for (int r = (blockIdx.x * 256 + threadIdx.x) / 32; r < n; r += gridDim.x * 8) {
    const float2* p = a.partial + (int64_t)r * a.tiles;
    float top = -INFINITY, sum = 0.f;
    for (int i = lane; i < a.tiles; i += 32) top = fmaxf(top, p[i].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    for (int i = lane; i < a.tiles; i += 32) sum += p[i].x == -INFINITY ? p[i].y : p[i].y * expf(p[i].x - top);
    sum = warp_sum(sum);
    if (lane == 0) {
      const int t = a.list[r];
      const float lse = top + logf(sum);
      a.lse[t] = lse;
      a.loss[t] = lse - a.picked[r];
    }
  }
}

// 0 for the ignored tokens; the sum of the losses and the number of the labelled ones.
__global__ void __launch_bounds__(LIST_NT) loss_total_kernel(const LossK a) {
  pdl_enter();
  __shared__ double scratch[32];
  double s = 0.0;
  for (int t = threadIdx.x; t < a.T; t += LIST_NT) {
    const int label = a.labels[t];
    if (label < 0 || label >= a.V) a.loss[t] = a.lse[t] = 0.f;
    else s += a.loss[t];
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (threadIdx.x % 32 == 0) scratch[threadIdx.x / 32] = s;
  __syncthreads();
  if (threadIdx.x == 0 && a.total) {
    s = 0.0;
    for (int i = 0; i < LIST_NT / 32; ++i) s += scratch[i];
    a.total[0] = (float)s;
    a.total[1] = (float)*a.count;
  }
}

// acc (+)= dz W over the piece
template <typename T>
__global__ void __launch_bounds__(GEMM_NT) loss_dx_kernel(const LossK a) {
  pdl_enter();
  const int n = *a.count, r0 = blockIdx.y * TM, c0 = blockIdx.x * TN;
  if (r0 >= n) return;
  const T* W = static_cast<const T*>(a.W);
  float c[4][4];
  const int K = a.V - a.v0 < a.piece ? a.V - a.v0 : a.piece;
  tile_product(
      K, [&](int m, int k) { return r0 + m < n ? a.dz[(int64_t)(r0 + m) * a.piece + k] : 0.f; },
      [&](int i, int k) { return c0 + i < a.d ? to_f32(W[(int64_t)(a.v0 + k) * a.d + c0 + i]) : 0.f; }, c);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = r0 + ty * 4 + i, col = c0 + tx * 4 + j;
      if (r >= n || col >= a.d) continue;
      float* p = a.acc + (int64_t)r * a.d + col;
      *p = a.v0 == 0 ? c[i][j] : *p + c[i][j];
    }
}
// dW (+)= dz^T x of the piece's rows
template <typename T, typename TW>
__global__ void __launch_bounds__(GEMM_NT) loss_dw_kernel(const LossK a) {
  pdl_enter();
  const int n = *a.count, r0 = blockIdx.y * TM, c0 = blockIdx.x * TN;
  const T* x = static_cast<const T*>(a.x);
  float c[4][4];
  tile_product(
      n, [&](int m, int k) { return r0 + m < a.piece ? a.dz[(int64_t)k * a.piece + r0 + m] : 0.f; },
      [&](int i, int k) { return c0 + i < a.d ? to_f32(x[(int64_t)a.list[k] * a.d + c0 + i]) : 0.f; }, c);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = r0 + ty * 4 + i, col = c0 + tx * 4 + j;
      if (r >= a.piece || a.v0 + r >= a.V || col >= a.d) continue;
      TW* p = static_cast<TW*>(a.dW) + (int64_t)(a.v0 + r) * a.d + col;
      *p = from_f32<TW>(a.accumulate ? to_f32(*p) + c[i][j] : c[i][j]);
    }
}
// dx of the labelled tokens from acc, 0 for the others
template <typename T>
__global__ void __launch_bounds__(256) loss_dx_zero_kernel(const LossK a) {
  pdl_enter();
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int label = a.labels[t];
    if (label >= 0 && label < a.V) continue;
    for (int i = threadIdx.x; i < a.d; i += 256) static_cast<T*>(a.dx)[(int64_t)t * a.d + i] = from_f32<T>(0.f);
  }
}
template <typename T>
__global__ void __launch_bounds__(256) loss_dx_store_kernel(const LossK a) {
  pdl_enter();
  const int n = *a.count;
  for (int r = blockIdx.x; r < n; r += gridDim.x)
    for (int i = threadIdx.x; i < a.d; i += 256)
      static_cast<T*>(a.dx)[(int64_t)a.list[r] * a.d + i] = from_f32<T>(a.acc[(int64_t)r * a.d + i]);
}

size_t up(size_t n) { return (n + 255) / 256 * 256; }
int piece_of(int T, int V) {
  int64_t p = PIECE_VALUES / (T > 0 ? T : 1) / TN * TN;
  const int64_t all = ((int64_t)V + TN - 1) / TN * TN;
  if (p < TN) p = TN;
  return (int)(p < all ? p : all);
}
struct Layout {
  size_t list, count, picked, partial, dz, acc, end;
};
Layout layout(int T, int d, int V, bool training) {
  Layout l{};
  const size_t t = T;
  l.list = 0;
  l.count = l.list + up(t * 4);
  l.picked = l.count + 256;
  l.partial = l.picked + up(t * 4);
  l.end = l.partial + up(t * ((V + TN - 1) / TN) * 8);
  if (training) {  // the backward's share the place of the forward's
    l.dz = l.picked;
    l.acc = l.dz + up(t * piece_of(T, V) * 4);
    const size_t e = l.acc + up(t * d * 4);
    l.end = l.end > e ? l.end : e;
  }
  return l;
}
LossK kernel_args(const LossArgs& a, bool training, uint32_t* err) {
  const Layout l = layout(a.T, a.d, a.V, training);
  char* ws = static_cast<char*>(a.ws);
  LossK k{};
  k.x = a.x;
  k.W = a.W;
  k.labels = a.labels;
  k.loss = a.loss;
  k.lse = a.lse;
  k.total = a.total;
  k.dloss = a.dloss;
  k.dx = a.dx;
  k.dW = a.dW;
  k.T = a.T;
  k.d = a.d;
  k.V = a.V;
  k.accumulate = a.accumulate;
  k.list = reinterpret_cast<int32_t*>(ws + l.list);
  k.count = reinterpret_cast<int32_t*>(ws + l.count);
  k.picked = reinterpret_cast<float*>(ws + l.picked);
  k.partial = reinterpret_cast<float2*>(ws + l.partial);
  k.dz = reinterpret_cast<float*>(ws + l.dz);
  k.acc = reinterpret_cast<float*>(ws + l.acc);
  k.tiles = (a.V + TN - 1) / TN;
  k.err = err;
  return k;
}
#define LAUNCH(kind, ...)                            \
  do {                                               \
    LaunchScope ls(kind, st);                        \
    const cudaError_t e = launch_pdl(__VA_ARGS__);   \
    if (e != cudaSuccess) return e;                  \
  } while (0)

template <typename T>
cudaError_t fwd_t(const LossArgs& args, uint32_t* err, cudaStream_t st) {
  LossK a = kernel_args(args, false, err);
  a.piece = a.tiles * TN;
  LAUNCH(KK_LOSS_ROWS, loss_rows_kernel, dim3(1), dim3(LIST_NT), 0, st, a);
  LAUNCH(KK_LOSS_LOGITS, loss_logits_kernel<T, false>, dim3(a.tiles, (a.T + TM - 1) / TM), dim3(GEMM_NT), 0, st, a);
  LAUNCH(KK_LOSS_COMBINE, loss_combine_kernel, dim3((a.T + 7) / 8), dim3(256), 0, st, a);
  LAUNCH(KK_LOSS_FINISH, loss_total_kernel, dim3(1), dim3(LIST_NT), 0, st, a);
  return cudaSuccess;
}
template <typename T>
cudaError_t bwd_t(const LossArgs& args, uint32_t* err, cudaStream_t st) {
  LossK a = kernel_args(args, true, err);
  a.piece = piece_of(a.T, a.V);
  const int rows = (a.T + TM - 1) / TM, cols = (a.d + TN - 1) / TN;
  LAUNCH(KK_LOSS_ROWS, loss_rows_kernel, dim3(1), dim3(LIST_NT), 0, st, a);
  for (a.v0 = 0; a.v0 < a.V; a.v0 += a.piece) {
    LAUNCH(KK_LOSS_DLOGITS, loss_logits_kernel<T, true>, dim3(a.piece / TN, rows), dim3(GEMM_NT), 0, st, a);
    if (a.dx) LAUNCH(KK_LOSS_GRADS, loss_dx_kernel<T>, dim3(cols, rows), dim3(GEMM_NT), 0, st, a);
    const dim3 grid(cols, a.piece / TM);
    if (a.dW && args.dw_bf16) LAUNCH(KK_LOSS_GRADS, loss_dw_kernel<T, __nv_bfloat16>, grid, dim3(GEMM_NT), 0, st, a);
    else if (a.dW) LAUNCH(KK_LOSS_GRADS, loss_dw_kernel<T, float>, grid, dim3(GEMM_NT), 0, st, a);
  }
  if (!a.dx) return cudaSuccess;
  const unsigned ctas = a.T < 65536 ? a.T : 65536;
  LAUNCH(KK_LOSS_FINISH, loss_dx_zero_kernel<T>, dim3(ctas), dim3(256), 0, st, a);
  LAUNCH(KK_LOSS_FINISH, loss_dx_store_kernel<T>, dim3(ctas), dim3(256), 0, st, a);
  return cudaSuccess;
}

}  // namespace

size_t loss_ws_bytes(int T, int d, int V, bool bf16, bool training) {
  (void)bf16;
  return layout(T, d, V, training).end;
}
cudaError_t launch_loss_fwd(const LossArgs& a, uint32_t* err, cudaStream_t st) {
  return a.bf16 ? fwd_t<__nv_bfloat16>(a, err, st) : fwd_t<float>(a, err, st);
}
cudaError_t launch_loss_bwd(const LossArgs& a, uint32_t* err, cudaStream_t st) {
  return a.bf16 ? bwd_t<__nv_bfloat16>(a, err, st) : bwd_t<float>(a, err, st);
}

}  // namespace moe
