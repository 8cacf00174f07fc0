// The 2-norm of many gradient tensors together, and the gradients clipped to it.
//
//   norm = sqrt(sum_i sum g_i^2),  out_i = g_i * min(1, max_norm / norm)
//
// Two kernels over one list of chunks, which is passed by value with the
// launch (no copy to the device, and a captured graph keeps its own).  The first sums
// squares; the second adds the CTAs' sums, each CTA all of them in the same
// order, and scales.  It walks the chunks backwards, so what the first kernel
// read last comes from L2, and where nothing is clipped in place it ends at
// once.  Both are bound by HBM.
//
// Chunks begin on 16 bytes of the source whatever the tensor's own alignment;
// the first and last vector of a tensor are read element by element.
#include <cmath>
#include <cstring>

#include "common.cuh"
#include "step.h"

namespace moe {
namespace {

constexpr int CLIP_NT = 256;                  // threads of a chunk
constexpr int GROUPS = 4;                     // chunks that an SM has in work
constexpr int VECS = 8;                       // 16-byte vectors of a chunk that a thread holds
constexpr int CHUNK_BYTES = CLIP_NT * VECS * 16;
constexpr int FEW = 96, MANY = 768;           // tensors of a launch: parameters of 3 KB, or of 24 KB for long lists

// A tensor's entry is one line of the constant cache: a miss there is a latency
// of its own (fields in arrays of their own: 700 small tensors 20 us, both kernels).
struct alignas(32) ClipEntry {
  const void* src;
  void* dst;
  int64_t n;
  int64_t first_bf16;  // twice the tensor's first chunk, plus 1 for bf16
};
template <int N>
struct ClipList {
  ClipEntry t[N + 1];  // the last one's first chunk is the number of chunks
  int count;
  __host__ __device__ int64_t first(int i) const { return t[i].first_bf16 >> 1; }
};
struct ClipScale {
  const double* partial;
  int parts;
  float max_norm;
  float* norm;  // or null: another launch writes it
};

// Chunks of a tensor of n elements of es bytes at p, counted from the 16-byte boundary at or before it.
int64_t chunks_of(const void* p, int64_t n, int es) {
  if (n == 0) return 0;
  return ((int64_t)(reinterpret_cast<uintptr_t>(p) & 15) + n * es + CHUNK_BYTES - 1) / CHUNK_BYTES;
}

// The tensor of a chunk: searched from where it would be among tensors of equal
// length, in growing steps (each look at the list is a latency of its own: 300
// small tensors 20.7 us by halving, both kernels).
template <int N>
__device__ __forceinline__ int tensor_of(const ClipList<N>& l, int64_t chunk) {
  int lo = (int)((float)chunk / (float)l.first(l.count) * (float)l.count), hi, step = 1;
  if (lo >= l.count) lo = l.count - 1;
  if (l.first(lo) <= chunk) {
    while (lo + step < l.count && l.first(lo + step) <= chunk) {
      lo += step;
      step *= 2;
    }
    hi = lo + step < l.count ? lo + step : l.count;
  } else {
    hi = lo;
    while (hi - step > 0 && l.first(hi - step) > chunk) {
      hi -= step;
      step *= 2;
    }
    lo = hi - step > 0 ? hi - step : 0;
  }
  while (lo + 1 < hi) {  // first[lo] <= chunk < first[hi]
    const int mid = (lo + hi) >> 1;
    if (l.first(mid) <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

// A thread's part of a chunk: VECS vectors, CLIP_NT apart.  e0 is the element
// index (in the tensor) of vector j's first element; it may be negative in the
// first vector and reach past n in the last.
template <typename T>
struct Part {
  const T* src;   // the tensor's first element
  int64_t n, e0;  // of the thread's first vector
  static constexpr int VN = Vec<T>::N;
  __device__ __forceinline__ Part(const void* p, int64_t n_, int64_t chunk) : src(static_cast<const T*>(p)), n(n_) {
    const int before = (int)(reinterpret_cast<uintptr_t>(p) & 15) / (int)sizeof(T);
    e0 = chunk * (CHUNK_BYTES / (int)sizeof(T)) + (int)(threadIdx.x % CLIP_NT) * VN - before;
  }
  __device__ __forceinline__ int64_t at(int j) const { return e0 + (int64_t)j * CLIP_NT * VN; }
  __device__ __forceinline__ bool whole(int j) const { return at(j) >= 0 && at(j) + VN <= n; }
  __device__ __forceinline__ void load(uint4 (&u)[VECS]) const {
#pragma unroll
    for (int j = 0; j < VECS; ++j) {
      if (whole(j)) {
        u[j] = *reinterpret_cast<const uint4*>(src + at(j));
      } else {
        T w[VN];
#pragma unroll
        for (int i = 0; i < VN; ++i) w[i] = at(j) + i >= 0 && at(j) + i < n ? src[at(j) + i] : from_f32<T>(0.f);
        memcpy(&u[j], w, 16);
      }
    }
  }
};

// The sum of squares of a thread's part of a chunk in 64 bits, read again.
template <typename T>
__device__ __noinline__ double squares64(const void* src, int64_t n, int64_t chunk) {
  constexpr int VN = Vec<T>::N;
  const Part<T> p(src, n, chunk);
  double d = 0.0;
  for (int j = 0; j < VECS; ++j)
    for (int i = 0; i < VN; ++i) {
      const int64_t at = p.at(j) + i;
      const double v = at >= 0 && at < n ? (double)to_f32(p.src[at]) : 0.0;
      d += v * v;
    }
  return d;
}
// The same, in fp32 where that is exact enough: where the largest value is
// within 2^50 of 1 either way nothing that counts underflows and nothing
// overflows.  Beyond that no trained model is.  A NaN is left out by the maximum
// and makes either sum a NaN.
template <typename T>
__device__ __forceinline__ double squares(const void* src, int64_t n, int64_t chunk) {
  constexpr int VN = Vec<T>::N;
  uint4 u[VECS];
  Part<T>(src, n, chunk).load(u);
  float top = 0.f, s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < VECS; ++j) {
    float v[VN];
    unpack(u[j], v);
#pragma unroll
    for (int i = 0; i < VN; ++i) {
      top = fmaxf(top, fabsf(v[i]));
      s[i & 3] = fmaf(v[i], v[i], s[i & 3]);
    }
  }
  if (top > 0x1p50f || (top < 0x1p-50f && top != 0.f)) return squares64<T>(src, n, chunk);
  return (double)((s[0] + s[1]) + (s[2] + s[3]));
}

// Sums in 64 bits are few and made by one warp: the SM adds two doubles a clock
// (with all threads in a tree, and CTAs of 256, 700 small tensors took 20 us).
__device__ __forceinline__ double warp_sum64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// CTAs of a chunk at a time (one of four: 350 us for 604 M float32, not 337)
template <int N>
__global__ void __launch_bounds__(CLIP_NT, GROUPS) grad_norm_kernel(const __grid_constant__ ClipList<N> l, double* partial) {
  pdl_enter();
  __shared__ double each[CLIP_NT];
  const int64_t total = l.first(l.count);
  double sum = 0.0;
#pragma unroll 1
  for (int64_t c = blockIdx.x; c < total; c += gridDim.x) {
    const ClipEntry& e = l.t[tensor_of(l, c)];
    sum += (e.first_bf16 & 1) ? squares<__nv_bfloat16>(e.src, e.n, c - (e.first_bf16 >> 1))
                              : squares<float>(e.src, e.n, c - (e.first_bf16 >> 1));
  }
  each[threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  sum = 0.0;
#pragma unroll
  for (int i = 0; i < CLIP_NT; i += 32) sum += each[i + threadIdx.x];
  sum = warp_sum64(sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const void* src, void* dst_, int64_t n, int64_t chunk, float scale) {
  constexpr int VN = Vec<T>::N;
  const Part<T> p(src, n, chunk);
  T* dst = static_cast<T*>(dst_);
  const bool aligned = ((reinterpret_cast<uintptr_t>(src) ^ reinterpret_cast<uintptr_t>(dst_)) & 15) == 0;
  uint4 u[VECS];
  p.load(u);
#pragma unroll
  for (int j = 0; j < VECS; ++j) {
    float v[VN];
    unpack(u[j], v);
#pragma unroll
    for (int i = 0; i < VN; ++i) v[i] *= scale;
    if (aligned && p.whole(j)) {
      stg16(dst + p.at(j), pack(v));
    } else {
#pragma unroll
      for (int i = 0; i < VN; ++i)
        if (p.at(j) + i >= 0 && p.at(j) + i < n) dst[p.at(j) + i] = from_f32<T>(v[i]);
    }
  }
}

// The same by a scale that is no normal float32 or near to it, an element at a
// time in 64 bits.
constexpr float SMALL_SCALE = 0x1p-100f;
template <typename T>
__device__ __noinline__ void scale_chunk64(const void* src, void* dst_, int64_t n, int64_t chunk, double scale) {
  constexpr int VN = Vec<T>::N;
  const Part<T> p(src, n, chunk);
  T* dst = static_cast<T*>(dst_);
#pragma unroll 1
  for (int j = 0; j < VECS; ++j)
#pragma unroll 1
    for (int i = 0; i < VN; ++i) {
      const int64_t at = p.at(j) + i;
      if (at >= 0 && at < n) dst[at] = from_f32<T>((float)((double)to_f32(p.src[at]) * scale));
    }
}

// One CTA an SM: each makes the norm for itself.  (64 registers for 1024 threads: 54
// bytes are spilled beside the eight vectors that a thread has in work.)
template <int N>
__global__ void __launch_bounds__(CLIP_NT* GROUPS, 1) grad_clip_kernel(const __grid_constant__ ClipList<N> l, const ClipScale s) {
  pdl_enter();
  __shared__ double by;
  __shared__ bool clip;
  if (threadIdx.x < 32) {
    double sum = 0.0;
#pragma unroll 4
    for (int i = threadIdx.x; i < s.parts; i += 32) sum += s.partial[i];
    sum = warp_sum64(sum);
    if (threadIdx.x == 0) {
      const double norm = sqrt(sum);
      const float as_float = (float)norm;
      if (s.norm != nullptr && blockIdx.x == 0) *s.norm = as_float;
      clip = isfinite(as_float) && as_float > s.max_norm;
      by = clip ? (double)s.max_norm / norm : 1.0;
    }
  }
  __syncthreads();
  const bool clips = clip;
  const float scale = (float)by;
  const int64_t total = l.first(l.count);
#pragma unroll 1
  for (int64_t c = total - 1 - blockIdx.x - (int64_t)(threadIdx.x / CLIP_NT) * gridDim.x; c >= 0; c -= GROUPS * gridDim.x) {
    const ClipEntry& e = l.t[tensor_of(l, c)];
    if (e.dst == nullptr || (!clips && e.dst == e.src)) continue;
    if (scale < SMALL_SCALE) {
      if (e.first_bf16 & 1) scale_chunk64<__nv_bfloat16>(e.src, e.dst, e.n, c - (e.first_bf16 >> 1), by);
      else scale_chunk64<float>(e.src, e.dst, e.n, c - (e.first_bf16 >> 1), by);
      continue;
    }
    if (e.first_bf16 & 1) scale_chunk<__nv_bfloat16>(e.src, e.dst, e.n, c - (e.first_bf16 >> 1), scale);
    else scale_chunk<float>(e.src, e.dst, e.n, c - (e.first_bf16 >> 1), scale);
  }
}

// The list of tensors [from, from + N) of the call; its chunks.
template <int N>
int64_t fill(ClipList<N>* l, const moe_grad* g, int count, int from) {
  int k = 0;
  int64_t chunks = 0;
  for (int i = from; i < count && i < from + N; ++i) {
    const int es = g[i].dtype == MOE_BF16 ? 2 : 4;
    if (g[i].n == 0) continue;
    l->t[k++] = {g[i].src, g[i].dst, g[i].n, chunks * 2 + (es == 2)};
    chunks += chunks_of(g[i].src, g[i].n, es);
  }
  l->t[k].first_bf16 = chunks * 2;
  l->count = k;
  return chunks;
}
unsigned ctas(int64_t chunks, int an_sm) {
  const int64_t most = (int64_t)sm_count() * an_sm;
  return (unsigned)(chunks < most ? chunks : most);
}

template <int N>
cudaError_t clip_lists(const moe_grad* g, int count, float max_norm, float* norm, double* partial, cudaStream_t st) {
  ClipList<N> l;
  int parts = 0;
  for (int from = 0; from < count; from += N) {
    const int64_t chunks = fill(&l, g, count, from);
    if (chunks == 0) continue;
    LaunchScope ls(KK_GRAD_NORM, st);
    const cudaError_t e = launch_pdl(grad_norm_kernel<N>, dim3(ctas(chunks, GROUPS)), dim3(CLIP_NT), 0, st, l,
                                     partial + parts);
    if (e != cudaSuccess) return e;
    parts += (int)ctas(chunks, GROUPS);
  }
  bool writes = false;
  for (int i = 0; i < count; ++i)
    writes = writes || (g[i].n > 0 && g[i].dst != nullptr && (g[i].dst != g[i].src || !std::isinf(max_norm)));
  ClipScale s{partial, parts, max_norm, norm};
  const int last = writes ? (count - 1) / N * N : 0;
  for (int from = last; from >= 0; from -= N) {  // backwards, as the chunks are
    int64_t chunks = fill(&l, g, count, from);
    if (!writes) {
      l.count = 0;
      l.t[0].first_bf16 = 0;
      chunks = 1;  // the norm alone
    } else if (chunks == 0 && s.norm == nullptr) {
      continue;
    }
    LaunchScope ls(KK_GRAD_CLIP, st);
    const cudaError_t e = launch_pdl(grad_clip_kernel<N>, dim3(ctas(chunks < 1 ? 1 : chunks, 1)),
                                     dim3(CLIP_NT * GROUPS), 0, st, l, s);
    if (e != cudaSuccess) return e;
    s.norm = nullptr;
  }
  return cudaSuccess;
}

}  // namespace

size_t clip_ws_bytes(int count) {
  const int per = count <= FEW ? FEW : MANY;
  return (size_t)((count + per - 1) / per + 1) * sm_count() * GROUPS * sizeof(double);
}

cudaError_t launch_clip(const moe_grad* grads, int count, float max_norm, float* norm, void* ws, cudaStream_t st) {
  double* partial = static_cast<double*>(ws);
  return count <= FEW ? clip_lists<FEW>(grads, count, max_norm, norm, partial, st)
                      : clip_lists<MANY>(grads, count, max_norm, norm, partial, st);
}

}  // namespace moe
