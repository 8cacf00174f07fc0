// Layer norm of the rows in front of the layer, forward and backward.
//
//   forward   mean = sum(x) / d,  rstd = 1 / sqrt(sum((x - mean)^2) / d + eps)
//             y = (x - mean) * rstd * gamma + beta
//   backward  n = (x - mean) * rstd,  v = dy * gamma
//             dx = rstd * (v - sum(v) / d - n * sum(v n) / d)  [+ dres]
//             dgamma = sum over rows of dy * n,  dbeta = sum over rows of dy
//
// Both passes are bound by HBM: the forward reads and writes a row once, the
// backward reads x, dy (and dres) and writes dx.  A row is held in registers
// between the load and the store: `tpr` threads share it, each with NV vectors
// of VN elements, so the variance is the sum of squared distances from the
// mean (no cancellation of large means) without a second read.  A CTA walks
// rows in a grid stride and keeps its columns' gamma, beta and, in the
// backward, its dgamma and dbeta sums in registers; the sums of the CTAs are
// added in CTA order by a second kernel, so results do not depend on timing.
// All statistics and sums are fp32.
//
// Rows that are not a multiple of 16 bytes (odd d) are loaded element by
// element, coalesced; rows of more than 8192 elements are walked in a loop
// (the wide kernels) and read again from cache.
#include "block.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int MAX_TPR = 512;   // most threads that share a row held in registers
constexpr int EPT = 16;        // most elements of a row a thread holds
constexpr int NT = 256;        // threads a CTA when tpr <= 256
constexpr int WIDE_NT = 512;   // threads a CTA of the wide kernels
constexpr int RED_COLS = 32, RED_STRIPS = 16;

template <typename T, int VN>
__device__ __forceinline__ void ld_vec(const T* p, float* v) {
  if constexpr (VN == 1) {
    v[0] = to_f32(*p);
  } else {
    float w[Vec<T>::N];
    unpack(*reinterpret_cast<const uint4*>(p), w);
#pragma unroll
    for (int i = 0; i < VN; ++i) v[i] = w[i];
  }
}
template <typename T, int VN>
__device__ __forceinline__ void st_vec(T* p, const float* v) {
  if constexpr (VN == 1) {
    *p = from_f32<T>(v[0]);
  } else {
    float w[Vec<T>::N];
#pragma unroll
    for (int i = 0; i < VN; ++i) w[i] = v[i];
    stg16(p, pack(w));
  }
}
template <int VN>
__device__ __forceinline__ void ld_f32(const float* p, float* v) {
#pragma unroll
  for (int i = 0; i < VN; ++i) v[i] = __ldg(p + i);
}

// Sum over the tpr threads of a row; scratch holds one float2 a warp, twice
// (used in turn, so one barrier a reduction).
__device__ __forceinline__ float2 row_sum(float2 s, int tpr, float2* scratch, int& turn) {
  s.x = warp_sum(s.x);
  s.y = warp_sum(s.y);
  if (tpr > 32) {
    const int warp = threadIdx.x / 32, nw = blockDim.x / 32;
    float2* buf = scratch + turn * nw;
    turn ^= 1;
    if (threadIdx.x % 32 == 0) buf[warp] = s;
    __syncthreads();
    const int w0 = warp & ~(tpr / 32 - 1);
    s = make_float2(0.f, 0.f);
    for (int i = 0; i < tpr / 32; ++i) {
      s.x += buf[w0 + i].x;
      s.y += buf[w0 + i].y;
    }
  }
  return s;
}

struct NormArgs {
  const void* x;
  const void* dy;
  const void* dres;
  const float* gamma;
  const float* beta;
  const float* mean_in;
  const float* rstd_in;
  void* out;  // y or dx
  float* mean;
  float* rstd;
  float* partial;  // [CTAs][2][d]: dgamma, dbeta
  float* dgamma;
  float* dbeta;
  int64_t rows;
  int d, tpr, parts, accumulate;
  float eps;
};

template <typename T, int VN, int NV>
__global__ void __launch_bounds__(MAX_TPR) norm_fwd_kernel(const NormArgs a) {
  pdl_enter();  // see pdl_wait: no global access before this
  __shared__ float2 scratch[2 * MAX_TPR / 32];
  int turn = 0;
  const T* x = static_cast<const T*>(a.x);
  T* y = static_cast<T*>(a.out);
  const int groups = blockDim.x / a.tpr, g = threadIdx.x / a.tpr, r = threadIdx.x % a.tpr;
  const int nvec = a.d / VN;
  const float inv = 1.f / (float)a.d;
  float ga[NV * VN], be[NV * VN];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int q = r + i * a.tpr;
#pragma unroll
    for (int j = 0; j < VN; ++j) ga[i * VN + j] = be[i * VN + j] = 0.f;
    if (q < nvec) {
      ld_f32<VN>(a.gamma + (size_t)q * VN, ga + i * VN);
      ld_f32<VN>(a.beta + (size_t)q * VN, be + i * VN);
    }
  }
  // every group of the CTA makes the same number of turns (row_sum has a barrier)
  for (int64_t row0 = (int64_t)blockIdx.x * groups; row0 < a.rows; row0 += (int64_t)gridDim.x * groups) {
    const int64_t row = row0 + g;
    const bool live = row < a.rows;
    const T* xr = x + row * a.d;
    float v[NV * VN];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int q = r + i * a.tpr;
#pragma unroll
      for (int j = 0; j < VN; ++j) v[i * VN + j] = 0.f;
      if (live && q < nvec) ld_vec<T, VN>(xr + (size_t)q * VN, v + i * VN);
    }
#pragma unroll
    for (int i = 0; i < NV * VN; ++i) s += v[i];
    const float mean = row_sum(make_float2(s, 0.f), a.tpr, scratch, turn).x * inv;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (r + i * a.tpr < nvec) {
#pragma unroll
        for (int j = 0; j < VN; ++j) {
          v[i * VN + j] -= mean;
          s = fmaf(v[i * VN + j], v[i * VN + j], s);
        }
      }
    const float var = row_sum(make_float2(s, 0.f), a.tpr, scratch, turn).x * inv;
    const float rstd = 1.f / sqrtf(var + a.eps);
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int q = r + i * a.tpr;
      if (q < nvec) {
#pragma unroll
        for (int j = 0; j < VN; ++j) v[i * VN + j] = fmaf(v[i * VN + j] * rstd, ga[i * VN + j], be[i * VN + j]);
        st_vec<T, VN>(y + row * a.d + (size_t)q * VN, v + i * VN);
      }
    }
    if (r == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

template <typename T, int VN, int NV, bool RES>
__global__ void __launch_bounds__(MAX_TPR) norm_bwd_kernel(const NormArgs a) {
  pdl_enter();
  __shared__ float2 scratch[2 * MAX_TPR / 32];
  extern __shared__ float dsum[];  // [2][d]: the CTA's dgamma and dbeta (groups > 1)
  int turn = 0;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  const T* res = static_cast<const T*>(a.dres);
  T* dx = static_cast<T*>(a.out);
  const int groups = blockDim.x / a.tpr, g = threadIdx.x / a.tpr, r = threadIdx.x % a.tpr;
  const int nvec = a.d / VN;
  const float inv = 1.f / (float)a.d;
  float ga[NV * VN], dg[NV * VN], db[NV * VN];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int q = r + i * a.tpr;
#pragma unroll
    for (int j = 0; j < VN; ++j) ga[i * VN + j] = dg[i * VN + j] = db[i * VN + j] = 0.f;
    if (q < nvec) ld_f32<VN>(a.gamma + (size_t)q * VN, ga + i * VN);
  }
  for (int64_t row0 = (int64_t)blockIdx.x * groups; row0 < a.rows; row0 += (int64_t)gridDim.x * groups) {
    const int64_t row = row0 + g;
    const bool live = row < a.rows;
    const float mean = live ? a.mean_in[row] : 0.f, rstd = live ? a.rstd_in[row] : 0.f;
    float n[NV * VN], v[NV * VN];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int q = r + i * a.tpr;
#pragma unroll
      for (int j = 0; j < VN; ++j) n[i * VN + j] = v[i * VN + j] = 0.f;
      if (live && q < nvec) {
        ld_vec<T, VN>(x + row * a.d + (size_t)q * VN, n + i * VN);
        ld_vec<T, VN>(dy + row * a.d + (size_t)q * VN, v + i * VN);
      }
    }
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (live && r + i * a.tpr < nvec) {
#pragma unroll
        for (int j = 0; j < VN; ++j) {
          const int c = i * VN + j;
          n[c] = (n[c] - mean) * rstd;
          dg[c] = fmaf(v[c], n[c], dg[c]);
          db[c] += v[c];
          v[c] *= ga[c];
          s.x += v[c];
          s.y = fmaf(v[c], n[c], s.y);
        }
      }
    s = row_sum(s, a.tpr, scratch, turn);
    const float m1 = s.x * inv, m2 = s.y * inv;
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int q = r + i * a.tpr;
      if (q < nvec) {
        float o[VN], rr[VN];
        if (RES) ld_vec<T, VN>(res + row * a.d + (size_t)q * VN, rr);
#pragma unroll
        for (int j = 0; j < VN; ++j) {
          const int c = i * VN + j;
          o[j] = (v[c] - m1 - n[c] * m2) * rstd;
          if (RES) o[j] += rr[j];
        }
        st_vec<T, VN>(dx + row * a.d + (size_t)q * VN, o);
      }
    }
  }
  // the CTA's sums: the groups in turn, then one row pair of the partials
  float* out = a.partial + (size_t)blockIdx.x * 2 * a.d;
  for (int t = 0; t < groups; ++t) {
    if (groups > 1) __syncthreads();
    if (g != t) continue;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int q = r + i * a.tpr;
      if (q < nvec) {
#pragma unroll
        for (int j = 0; j < VN; ++j) {
          const int c = i * VN + j, col = q * VN + j;
          float u = dg[c], w = db[c];
          if (t > 0) {
            u += dsum[col];
            w += dsum[a.d + col];
          }
          if (t == groups - 1) {
            out[col] = u;
            out[a.d + col] = w;
          } else {
            dsum[col] = u;
            dsum[a.d + col] = w;
          }
        }
      }
    }
  }
}

// dgamma and dbeta from the partials [parts][2][d], added in part order within
// RED_STRIPS interleaved strips and then over the strips.
__global__ void __launch_bounds__(RED_COLS * RED_STRIPS) norm_bwd_reduce_kernel(const NormArgs a) {
  pdl_enter();
  __shared__ float tile[RED_STRIPS][RED_COLS + 1];
  const int c = threadIdx.x % RED_COLS, strip = threadIdx.x / RED_COLS;
  const int col = blockIdx.x * RED_COLS + c;  // of the 2 d columns
  float s = 0.f;
  if (col < 2 * a.d)
    for (int p = strip; p < a.parts; p += RED_STRIPS) s += a.partial[(size_t)p * 2 * a.d + col];
  tile[strip][c] = s;
  __syncthreads();
  if (strip == 0 && col < 2 * a.d) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < RED_STRIPS; ++i) s += tile[i][c];
    float* dst = col < a.d ? a.dgamma + col : a.dbeta + (col - a.d);
    *dst = a.accumulate ? *dst + s : s;
  }
}

// ---- rows of more than MAX_TPR * EPT elements: one CTA a row, walked in a loop ----
__device__ __forceinline__ float2 cta_sum(float2 s, float2* scratch, int& turn) {
  return row_sum(s, WIDE_NT, scratch, turn);
}

template <typename T>
__global__ void __launch_bounds__(WIDE_NT) norm_fwd_wide_kernel(const NormArgs a) {
  pdl_enter();
  __shared__ float2 scratch[2 * WIDE_NT / 32];
  int turn = 0;
  const float inv = 1.f / (float)a.d;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* xr = static_cast<const T*>(a.x) + row * a.d;
    T* yr = static_cast<T*>(a.out) + row * a.d;
    float s = 0.f;
    for (int i = threadIdx.x; i < a.d; i += WIDE_NT) s += to_f32(xr[i]);
    const float mean = cta_sum(make_float2(s, 0.f), scratch, turn).x * inv;
    s = 0.f;
    for (int i = threadIdx.x; i < a.d; i += WIDE_NT) {
      const float c = to_f32(xr[i]) - mean;
      s = fmaf(c, c, s);
    }
    const float rstd = 1.f / sqrtf(cta_sum(make_float2(s, 0.f), scratch, turn).x * inv + a.eps);
    for (int i = threadIdx.x; i < a.d; i += WIDE_NT)
      yr[i] = from_f32<T>(fmaf((to_f32(xr[i]) - mean) * rstd, __ldg(a.gamma + i), __ldg(a.beta + i)));
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// dx of the rows row = blockIdx.x, + gridDim.x, ... and the sums of the same rows
template <typename T>
__global__ void __launch_bounds__(WIDE_NT) norm_bwd_wide_kernel(const NormArgs a) {
  pdl_enter();
  __shared__ float2 scratch[2 * WIDE_NT / 32];
  int turn = 0;
  const float inv = 1.f / (float)a.d;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  const T* res = static_cast<const T*>(a.dres);
  T* dx = static_cast<T*>(a.out);
  float* part = a.partial + (size_t)blockIdx.x * 2 * a.d;
  bool first = true;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float mean = a.mean_in[row], rstd = a.rstd_in[row];
    const int64_t at = row * a.d;
    float2 s = make_float2(0.f, 0.f);
    for (int i = threadIdx.x; i < a.d; i += WIDE_NT) {
      const float v = to_f32(dy[at + i]) * __ldg(a.gamma + i);
      s.x += v;
      s.y = fmaf(v, (to_f32(x[at + i]) - mean) * rstd, s.y);
    }
    s = cta_sum(s, scratch, turn);
    const float m1 = s.x * inv, m2 = s.y * inv;
    for (int i = threadIdx.x; i < a.d; i += WIDE_NT) {
      const float g = to_f32(dy[at + i]), n = (to_f32(x[at + i]) - mean) * rstd;
      float o = (g * __ldg(a.gamma + i) - m1 - n * m2) * rstd;
      if (res) o += to_f32(res[at + i]);
      dx[at + i] = from_f32<T>(o);
      part[i] = first ? g * n : fmaf(g, n, part[i]);
      part[a.d + i] = first ? g : part[a.d + i] + g;
    }
    first = false;
  }
}

bool wide(int d) { return d > MAX_TPR * EPT; }

// Threads that share a row: as few as hold it in EPT elements each.
int threads_per_row(int d, int vn, int nv) {
  int tpr = 32;
  while ((int64_t)tpr * vn * nv < d) tpr *= 2;
  return tpr;
}
bool whole_vectors(int d, bool bf16) { return d % (bf16 ? 8 : 4) == 0; }

// CTAs of the backward, each with its own partial sums: at most two an SM
int bwd_ctas(int64_t rows, int d, int groups) {
  const int64_t need = (rows + groups - 1) / groups, most = (int64_t)sm_count() * 2;
  return (int)(need < most ? need : most);
}
// groups of a CTA for the vector and the element path (the partials are sized for either)
int groups_of(int tpr) { return tpr < NT ? NT / tpr : 1; }

template <typename T, int VN, int NV>
cudaError_t fwd_n(NormArgs& a, cudaStream_t st) {
  a.tpr = threads_per_row(a.d, VN, NV);
  const int groups = groups_of(a.tpr), threads = a.tpr < NT ? NT : a.tpr;
  const int64_t need = (a.rows + groups - 1) / groups, most = (int64_t)sm_count() * (2048 / threads);
  return launch_pdl(norm_fwd_kernel<T, VN, NV>, dim3((unsigned)(need < most ? need : most)), dim3(threads), 0, st, a);
}
template <typename T, int VN, int NV>
cudaError_t bwd_n(NormArgs& a, cudaStream_t st) {
  a.tpr = threads_per_row(a.d, VN, NV);
  const int groups = groups_of(a.tpr), threads = a.tpr < NT ? NT : a.tpr;
  a.parts = bwd_ctas(a.rows, a.d, groups);
  const size_t smem = groups > 1 ? (size_t)2 * a.d * 4 : 0;
  return a.dres ? launch_pdl(norm_bwd_kernel<T, VN, NV, true>, dim3(a.parts), dim3(threads), smem, st, a)
                : launch_pdl(norm_bwd_kernel<T, VN, NV, false>, dim3(a.parts), dim3(threads), smem, st, a);
}
template <typename T>
cudaError_t fwd_t(NormArgs& a, cudaStream_t st) {
  constexpr int VN = Vec<T>::N;
  if (wide(a.d)) {
    const int64_t most = (int64_t)sm_count() * 4;
    return launch_pdl(norm_fwd_wide_kernel<T>, dim3((unsigned)(a.rows < most ? a.rows : most)), dim3(WIDE_NT), 0, st, a);
  }
  if (a.d % VN == 0) return fwd_n<T, VN, EPT / VN>(a, st);
  return fwd_n<T, 1, EPT>(a, st);
}
template <typename T>
cudaError_t bwd_t(NormArgs& a, cudaStream_t st) {
  constexpr int VN = Vec<T>::N;
  if (wide(a.d)) {
    a.parts = bwd_ctas(a.rows, a.d, 1);
    return launch_pdl(norm_bwd_wide_kernel<T>, dim3(a.parts), dim3(WIDE_NT), 0, st, a);
  }
  if (a.d % VN == 0) return bwd_n<T, VN, EPT / VN>(a, st);
  return bwd_n<T, 1, EPT>(a, st);
}

}  // namespace

cudaError_t launch_norm_fwd(int64_t rows, int d, bool bf16, const void* x, const float* gamma, const float* beta,
                            float eps, void* y, float* mean, float* rstd, cudaStream_t st) {
  NormArgs a{};
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.eps = eps;
  a.out = y;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.d = d;
  LaunchScope ls(KK_NORM_FWD, st);
  return bf16 ? fwd_t<__nv_bfloat16>(a, st) : fwd_t<float>(a, st);
}

size_t norm_ws_bytes(int64_t rows, int d) {
  return (size_t)bwd_ctas(rows, d, 1) * 2 * d * 4;  // one group a CTA makes the most CTAs
}

cudaError_t launch_norm_bwd(int64_t rows, int d, bool bf16, const void* x, const void* dy, const float* gamma,
                            const float* mean, const float* rstd, const void* dres, void* dx, float* dgamma,
                            float* dbeta, int accumulate, void* ws, cudaStream_t st) {
  NormArgs a{};
  a.x = x;
  a.dy = dy;
  a.dres = dres;
  a.gamma = gamma;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.out = dx;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.partial = static_cast<float*>(ws);
  a.rows = rows;
  a.d = d;
  a.accumulate = accumulate;
  {
    LaunchScope ls(KK_NORM_BWD, st);
    const cudaError_t e = bf16 ? bwd_t<__nv_bfloat16>(a, st) : bwd_t<float>(a, st);
    if (e != cudaSuccess) return e;
  }
  LaunchScope ls(KK_NORM_BWD_REDUCE, st);
  return launch_pdl(norm_bwd_reduce_kernel, dim3((2 * d + RED_COLS - 1) / RED_COLS), dim3(RED_COLS * RED_STRIPS), 0,
                    st, a);
}

}  // namespace moe
