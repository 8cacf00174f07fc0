// The residual path between two blocks with the norms on either side of it.
//
//   u   = y ry gamma_post,  out = rs x + bs row_gate gate u,  h = out ro gamma_next
//
// and its backward; formulas are in moe.h.
//
// A row has one CTA and is walked in a loop, again from cache for each pass.
// The columns' sums are taken in a pass of their own before anything is written
// (dx and dy may be dh or dout).  All statistics and sums are fp32.
#include "common.cuh"
#include "step.h"

namespace moe {
namespace {

constexpr int WIDE_NT = 512;   // threads of a row's CTA
constexpr int COL_NT = 128;
constexpr int RED_COLS = 32, RED_STRIPS = 32;

struct JoinK {
  const void *x, *y, *dh, *dout;
  void *out, *h, *dx, *dy;
  const float *gamma_post, *gamma_next, *gate, *row_gate;
  float *rstd_post, *rstd_next;
  float *dgamma_post, *dgamma_next, *dgate, *drow_gate;
  float* mean_vn;  // [rows]: sum(v n) / d
  float* partial;  // [parts][2][d]: sums of dh n, and of row_gate D m
  int64_t rows;
  int d, parts, accumulate;
  float rs, bs, eps;
  uint32_t* err;
};

__device__ __forceinline__ float row_sum(float v, float* scratch, int& turn) {
  v = warp_sum(v);
  if (threadIdx.x % 32 == 0) scratch[turn * 16 + threadIdx.x / 32] = v;
  __syncthreads();
  v = warp_sum(threadIdx.x % 32 < WIDE_NT / 32 ? scratch[turn * 16 + threadIdx.x % 32] : 0.f);
  turn ^= 1;
  return v;
}
template <typename T, int VN>
__device__ __forceinline__ void ld_n(const T* p, float (&v)[VN]) {
  if constexpr (VN == 1) v[0] = to_f32(*p);
  else unpack(*reinterpret_cast<const uint4*>(p), v);
}
template <typename T, int VN>
__device__ __forceinline__ void st_n(T* p, const float (&v)[VN]) {
  if constexpr (VN == 1) *p = from_f32<T>(v[0]);
  else stg16(p, pack(v));
}
// a weight of each channel, 1 where there is none (vectors need not be aligned)
template <int VN>
__device__ __forceinline__ void ld_w(const float* p, int i, float (&v)[VN]) {
#pragma unroll
  for (int j = 0; j < VN; ++j) v[j] = p == nullptr ? 1.f : __ldg(p + i + j);
}

template <typename T, int VN>
__global__ void __launch_bounds__(WIDE_NT) join_fwd_wide_kernel(const JoinK a) {
  pdl_enter();
  __shared__ float scratch[2 * 16];
  int turn = 0;
  const float inv = 1.f / (float)a.d;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.d;
    const T* y = static_cast<const T*>(a.y) + (a.y ? row * a.d : 0);
    float ry = 1.f, ro = 0.f;
    if (a.gamma_post) {
      float s = 0.f;
      for (int i = threadIdx.x * VN; i < a.d; i += WIDE_NT * VN) {
        float v[VN];
        ld_n<T, VN>(y + i, v);
#pragma unroll
        for (int j = 0; j < VN; ++j) s = fmaf(v[j], v[j], s);
      }
      ry = rsqrtf(fmaf(row_sum(s, scratch, turn), inv, a.eps));
    }
    const float by = a.bs * (a.row_gate ? a.row_gate[row] : 1.f) * ry;
    auto joined = [&](int i, float (&o)[VN]) {
      ld_n<T, VN>(x + i, o);
#pragma unroll
      for (int j = 0; j < VN; ++j) o[j] *= a.rs;
      if (a.y) {
        float v[VN], g[VN], w[VN];
        ld_n<T, VN>(y + i, v);
        ld_w<VN>(a.gamma_post, i, g);
        ld_w<VN>(a.gate, i, w);
#pragma unroll
        for (int j = 0; j < VN; ++j) o[j] = fmaf(v[j] * by, g[j] * w[j], o[j]);
      }
    };
    if (a.gamma_next) {
      float s = 0.f;
      for (int i = threadIdx.x * VN; i < a.d; i += WIDE_NT * VN) {
        float o[VN];
        joined(i, o);
#pragma unroll
        for (int j = 0; j < VN; ++j) s = fmaf(o[j], o[j], s);
      }
      ro = rsqrtf(fmaf(row_sum(s, scratch, turn), inv, a.eps));
    }
    for (int i = threadIdx.x * VN; i < a.d; i += WIDE_NT * VN) {
      float o[VN];
      joined(i, o);
      if (a.out) st_n<T, VN>(static_cast<T*>(a.out) + row * a.d + i, o);
      if (a.gamma_next) {
        float g[VN];
        ld_w<VN>(a.gamma_next, i, g);
#pragma unroll
        for (int j = 0; j < VN; ++j) o[j] *= ro * g[j];
        st_n<T, VN>(static_cast<T*>(a.h) + row * a.d + i, o);
      }
    }
    if (threadIdx.x == 0) {
      if (a.rstd_post) a.rstd_post[row] = ry;
      if (a.rstd_next) a.rstd_next[row] = ro;
    }
  }
}

// D of VN elements of a row, from the mean of v n
template <typename T, int VN>
__device__ __forceinline__ void stream_grad(const JoinK& a, int64_t row, int i, float ro, float mvn, float (&D)[VN]) {
  if (a.dout) {
    ld_n<T, VN>(static_cast<const T*>(a.dout) + row * a.d + i, D);
  } else {
#pragma unroll
    for (int j = 0; j < VN; ++j) D[j] = 0.f;
  }
  if (a.gamma_next) {
    float n[VN], v[VN], g[VN];
    ld_n<T, VN>(static_cast<const T*>(a.out) + row * a.d + i, n);
    ld_n<T, VN>(static_cast<const T*>(a.dh) + row * a.d + i, v);
    ld_w<VN>(a.gamma_next, i, g);
#pragma unroll
    for (int j = 0; j < VN; ++j) D[j] = fmaf(ro, fmaf(v[j], g[j], -(n[j] * ro) * mvn), D[j]);
  }
}

// sum(v n) / d of each row
template <typename T, int VN>
__global__ void __launch_bounds__(WIDE_NT) join_bwd_stats_kernel(const JoinK a) {
  pdl_enter();
  __shared__ float scratch[2 * 16];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float s = 0.f;
    if (a.gamma_next) {
      for (int i = threadIdx.x * VN; i < a.d; i += WIDE_NT * VN) {
        float n[VN], v[VN], g[VN];
        ld_n<T, VN>(static_cast<const T*>(a.out) + row * a.d + i, n);
        ld_n<T, VN>(static_cast<const T*>(a.dh) + row * a.d + i, v);
        ld_w<VN>(a.gamma_next, i, g);
#pragma unroll
        for (int j = 0; j < VN; ++j) s = fmaf(v[j] * g[j], n[j], s);
      }
      s = row_sum(s, scratch, turn) * a.rstd_next[row] / (float)a.d;
    }
    if (threadIdx.x == 0) a.mean_vn[row] = s;
  }
}

// The sums of VN columns a thread over the rows blockIdx.y, + gridDim.y, ...
template <typename T, int VN>
__global__ void __launch_bounds__(COL_NT) join_bwd_columns_kernel(const JoinK a) {
  pdl_enter();
  const int i = (blockIdx.x * COL_NT + threadIdx.x) * VN;
  if (i >= a.d) return;
  float sn[VN], sm[VN];
#pragma unroll
  for (int j = 0; j < VN; ++j) sn[j] = sm[j] = 0.f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float ro = a.gamma_next ? a.rstd_next[row] : 0.f;
    if (a.gamma_next) {
      float n[VN], v[VN];
      ld_n<T, VN>(static_cast<const T*>(a.out) + row * a.d + i, n);
      ld_n<T, VN>(static_cast<const T*>(a.dh) + row * a.d + i, v);
#pragma unroll
      for (int j = 0; j < VN; ++j) sn[j] = fmaf(v[j], n[j] * ro, sn[j]);
    }
    if (a.y) {
      const float by = (a.row_gate ? a.row_gate[row] : 1.f) * (a.gamma_post ? a.rstd_post[row] : 1.f);
      float D[VN], m[VN];
      stream_grad<T, VN>(a, row, i, ro, a.mean_vn[row], D);
      ld_n<T, VN>(static_cast<const T*>(a.y) + row * a.d + i, m);
#pragma unroll
      for (int j = 0; j < VN; ++j) sm[j] = fmaf(D[j], m[j] * by, sm[j]);
    }
  }
  float* out = a.partial + (size_t)blockIdx.y * 2 * a.d;
#pragma unroll
  for (int j = 0; j < VN; ++j) {
    out[i + j] = sn[j];
    out[a.d + i + j] = sm[j];
  }
}

template <typename T, int VN>
__global__ void __launch_bounds__(WIDE_NT) join_bwd_wide_kernel(const JoinK a) {
  pdl_enter();
  __shared__ float scratch[2 * 16];
  int turn = 0;
  const float inv = 1.f / (float)a.d;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float ro = a.gamma_next ? a.rstd_next[row] : 0.f, ry = a.gamma_post ? a.rstd_post[row] : 1.f;
    const float mvn = a.mean_vn[row], rg = a.row_gate ? a.row_gate[row] : 1.f;
    const T* y = static_cast<const T*>(a.y) + (a.y ? row * a.d : 0);
    float mwm = 0.f;
    if (a.gamma_post || a.drow_gate) {
      float s = 0.f;  // sum of bs gate gamma_post D m
      for (int i = threadIdx.x * VN; i < a.d; i += WIDE_NT * VN) {
        float D[VN], m[VN], g[VN], w[VN];
        stream_grad<T, VN>(a, row, i, ro, mvn, D);
        ld_n<T, VN>(y + i, m);
        ld_w<VN>(a.gate, i, g);
        ld_w<VN>(a.gamma_post, i, w);
#pragma unroll
        for (int j = 0; j < VN; ++j) s = fmaf(a.bs * D[j] * g[j] * w[j], m[j] * ry, s);
      }
      s = row_sum(s, scratch, turn);
      if (a.drow_gate && threadIdx.x == 0) a.drow_gate[row] = s;
      mwm = s * rg * inv;
    }
    for (int i = threadIdx.x * VN; i < a.d; i += WIDE_NT * VN) {
      float D[VN], o[VN], m[VN], g[VN], w[VN];
      stream_grad<T, VN>(a, row, i, ro, mvn, D);
      if (a.y) {
        ld_n<T, VN>(y + i, m);
        ld_w<VN>(a.gate, i, g);
        ld_w<VN>(a.gamma_post, i, w);
#pragma unroll
        for (int j = 0; j < VN; ++j) {
          const float G = a.bs * rg * g[j] * D[j];
          o[j] = a.gamma_post ? ry * fmaf(G, w[j], -(m[j] * ry) * mwm) : G;
        }
      }
#pragma unroll
      for (int j = 0; j < VN; ++j) D[j] *= a.rs;
      if (a.dx) st_n<T, VN>(static_cast<T*>(a.dx) + row * a.d + i, D);
      if (a.dy) st_n<T, VN>(static_cast<T*>(a.dy) + row * a.d + i, o);
    }
  }
}

// The parameters' gradients from the partials [parts][2][d], added in part
// order within RED_STRIPS interleaved strips and then over the strips.  The sum
// S of row_gate D m gives both that of gamma_post and that of the gate.
__global__ void __launch_bounds__(RED_COLS * RED_STRIPS) join_bwd_reduce_kernel(const JoinK a) {
  pdl_enter();
  __shared__ float tile[RED_STRIPS][RED_COLS + 1];
  const int c = threadIdx.x % RED_COLS, strip = threadIdx.x / RED_COLS;
  const int col = blockIdx.x * RED_COLS + c;  // of the 2 d columns
  float s = 0.f;
  if (col < 2 * a.d) {
#pragma unroll 1
    for (int p = strip; p < a.parts; p += 8 * RED_STRIPS) {  // eight loads at once
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = p + j * RED_STRIPS < a.parts ? a.partial[(size_t)(p + j * RED_STRIPS) * 2 * a.d + col] : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[j];
    }
  }
  tile[strip][c] = s;
  __syncthreads();
  if (strip != 0 || col >= 2 * a.d) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < RED_STRIPS; ++i) s += tile[i][c];
  auto give = [&](float* dst, float v) { *dst = a.accumulate ? *dst + v : v; };
  if (col < a.d) {
    if (a.dgamma_next) give(a.dgamma_next + col, s);
    return;
  }
  const int i = col - a.d;
  s *= a.bs;
  if (a.dgamma_post) give(a.dgamma_post + i, a.gate ? s * a.gate[i] : s);
  if (a.dgate) give(a.dgate + i, a.gamma_post ? s * a.gamma_post[i] : s);
}

JoinK kernel_args(const JoinArgs& a, uint32_t* err) {
  JoinK k{};
  k.x = a.x;
  k.y = a.y;
  k.dh = a.dh;
  k.dout = a.dout;
  k.out = a.out;
  k.h = a.h;
  k.dx = a.dx;
  k.dy = a.dy;
  k.gamma_post = a.p.gamma_post;
  k.gamma_next = a.p.gamma_next;
  k.gate = a.p.gate;
  k.row_gate = a.p.row_gate;
  k.rstd_post = a.rstd_post;
  k.rstd_next = a.rstd_next;
  k.dgamma_post = a.g.dgamma_post;
  k.dgamma_next = a.g.dgamma_next;
  k.dgate = a.g.dgate;
  k.drow_gate = a.g.drow_gate;
  k.rows = a.p.rows;
  k.d = a.p.d;
  k.accumulate = a.accumulate;
  k.rs = a.p.residual_scale;
  k.bs = a.p.branch_scale;
  k.eps = a.p.eps;
  k.err = err;
  return k;
}

unsigned row_ctas(int64_t rows) {
  const int64_t most = (int64_t)sm_count() * 4;
  return (unsigned)(rows < most ? rows : most);
}
// Row slices of the columns' sums: about 16 CTAs an SM
int wide_slices(int64_t rows, int d) {
  const int64_t tiles = (d + COL_NT * 8 - 1) / (COL_NT * 8), most = ((int64_t)sm_count() * 16 + tiles - 1) / tiles;
  return (int)(rows < most ? rows : most);
}

template <typename T, int VN>
cudaError_t fwd_wide(const JoinK& a, cudaStream_t st) {
  return launch_pdl(join_fwd_wide_kernel<T, VN>, dim3(row_ctas(a.rows)), dim3(WIDE_NT), 0, st, a);
}
template <typename T, int VN>
cudaError_t bwd_wide(JoinK& a, cudaStream_t st) {
  a.parts = wide_slices(a.rows, a.d);
  cudaError_t e = launch_pdl(join_bwd_stats_kernel<T, VN>, dim3(row_ctas(a.rows)), dim3(WIDE_NT), 0, st, a);
  if (e != cudaSuccess) return e;
  e = launch_pdl(join_bwd_columns_kernel<T, VN>, dim3((a.d + COL_NT * VN - 1) / (COL_NT * VN), a.parts), dim3(COL_NT), 0,
                 st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(join_bwd_wide_kernel<T, VN>, dim3(row_ctas(a.rows)), dim3(WIDE_NT), 0, st, a);
}
template <typename T>
cudaError_t fwd_t(const JoinK& a, cudaStream_t st) {
  return a.d % Vec<T>::N == 0 ? fwd_wide<T, Vec<T>::N>(a, st) : fwd_wide<T, 1>(a, st);
}
template <typename T>
cudaError_t bwd_t(JoinK& a, cudaStream_t st) {
  return a.d % Vec<T>::N == 0 ? bwd_wide<T, Vec<T>::N>(a, st) : bwd_wide<T, 1>(a, st);
}
size_t partial_bytes(int64_t rows, int d) { return (size_t)wide_slices(rows, d) * 2 * d * 4; }

}  // namespace

size_t join_ws_bytes(int64_t rows, int d) {
  return rows == 0 ? 0 : (partial_bytes(rows, d) + 255) / 256 * 256 + (size_t)rows * 4;
}

cudaError_t launch_join_fwd(const JoinArgs& args, uint32_t* err, cudaStream_t st) {
  const JoinK a = kernel_args(args, err);
  LaunchScope ls(KK_RESIDUAL_NORM_FWD, st);
  return args.p.dtype == MOE_BF16 ? fwd_t<__nv_bfloat16>(a, st) : fwd_t<float>(a, st);
}

cudaError_t launch_join_bwd(const JoinArgs& args, uint32_t* err, cudaStream_t st) {
  JoinK a = kernel_args(args, err);
  a.partial = static_cast<float*>(args.ws);
  a.mean_vn = reinterpret_cast<float*>(static_cast<char*>(args.ws) + (partial_bytes(a.rows, a.d) + 255) / 256 * 256);
  {
    LaunchScope ls(KK_RESIDUAL_NORM_BWD, st);
    const cudaError_t e = args.p.dtype == MOE_BF16 ? bwd_t<__nv_bfloat16>(a, st) : bwd_t<float>(a, st);
    if (e != cudaSuccess) return e;
  }
  if (!a.dgamma_post && !a.dgamma_next && !a.dgate) return cudaSuccess;
  LaunchScope ls(KK_RESIDUAL_NORM_REDUCE, st);
  return launch_pdl(join_bwd_reduce_kernel, dim3((2 * a.d + RED_COLS - 1) / RED_COLS), dim3(RED_COLS * RED_STRIPS), 0,
                    st, a);
}

}  // namespace moe
