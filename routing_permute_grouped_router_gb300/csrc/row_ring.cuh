// What kernels over rows in shared memory share: the layout of a row over the
// threads that share it, packed fp32 pairs, groups of threads with a barrier of
// their own, and the ring that plain copies bring rows into.  Each translation
// unit gets its own copy in an anonymous namespace.
//
// A copy has to begin and end on 16 bytes.  Rows of another length are copied
// with up to 15 bytes more on either side and read from shared memory element
// by element; what that would read past the tensor's end is loaded directly.
#pragma once

#include "common.cuh"

namespace moe {
namespace {

constexpr int MAX_TPR = 512;   // most threads that share a row held in registers
constexpr int EPT = 16;        // elements of a row a thread holds
constexpr int SMEM_SM = 220 * 1024;             // shared memory of an SM that the rings may take
constexpr int RING = 4;        // most rows on their way to a group of threads

// Element c (of EPT) of thread r of tpr, in whole vectors of VN or one by one.
template <int VN>
__device__ __forceinline__ int column(int r, int tpr, int c) {
  return (r + c / VN * tpr) * VN + c % VN;
}
// whether it is one of the row's d (d is a multiple of VN)
template <int VN>
__device__ __forceinline__ bool in_row(int r, int tpr, int c, int d) {
  return (r + c / VN * tpr) * VN < d;
}

// Two fp32 operations in one instruction; each half rounds as the scalar one does.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// A group of threads: `warps` warps that share a row, the g-th of its CTA.
// (SEVERAL: the CTA may have several groups of more than a warp.)
template <bool SEVERAL>
struct Group {
  int g, r, tpr, warps;
  __device__ __forceinline__ explicit Group(int tpr_) : g(threadIdx.x / tpr_), r(threadIdx.x % tpr_), tpr(tpr_), warps(tpr_ / 32) {}
  __device__ __forceinline__ void sync() const {
    if (warps == 1) __syncwarp();
    else if (SEVERAL) asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(tpr) : "memory");
    else __syncthreads();
  }
  // Every warp gives one float4; after sync() each thread gets that of warp
  // lane % warps, so xor shuffles over the warps (a power of two) finish a
  // sum.  scratch has two rows of 16, used in turn.
  __device__ __forceinline__ void give(float4 v, float4* scratch, int turn) const {
    if (threadIdx.x % 32 == 0) scratch[turn * 16 + threadIdx.x / 32] = v;
  }
  __device__ __forceinline__ float4 get(const float4* scratch, int turn) const {
    return scratch[turn * 16 + g * warps + (threadIdx.x & (warps - 1))];
  }
};
// Two sums over a warp: of a in the lower half of its lanes, of b in the upper half.
__device__ __forceinline__ float half_sums(float a, float b, bool upper) {
  float v = upper ? b : a;
  v += __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float sum_over(float v, int n) {  // n a power of two up to 16
#pragma unroll
  for (int o = 1; o <= 8; o *= 2)
    if (o < n) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---- the ring ----
__device__ __forceinline__ uint32_t sm_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy_row(uint32_t dst, const char* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ bool ring_ready(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for the barrier's phase, two seconds at most.
__device__ __noinline__ void ring_wait(uint32_t bar, uint32_t parity, uint32_t* err) {
  uint64_t t0 = 0;
  for (uint32_t i = 0; i < (1u << 30); ++i) {
    if (ring_ready(bar, parity)) return;
    if ((i & 255u) == 255u) {
      uint64_t t;
      asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
      if (t0 == 0) t0 = t;
      if (t - t0 > 2000000000ull) break;
    }
  }
  report_error(err, DEV_TIMEOUT, 760);
}

// Where a row's copy begins and how long it is: the row itself, or the 16-byte
// units that hold it, cut off at the end of the tensor.
struct Span {
  int64_t at;       // byte offset of the copy in the tensor
  int skip, bytes;  // bytes before the row's first element; bytes of the copy
  bool whole;       // it has all of the row
};
template <typename T, bool WHOLE>
__device__ __forceinline__ Span row_span(int64_t row, int64_t rows, int d) {
  const int64_t b0 = row * d * (int64_t)sizeof(T), b1 = b0 + d * (int64_t)sizeof(T);
  if (WHOLE) return {b0, 0, (int)(b1 - b0), true};
  const int64_t total = rows * d * (int64_t)sizeof(T), a0 = b0 & ~(int64_t)15;
  int64_t a1 = (b1 + 15) & ~(int64_t)15;
  if (a1 > total) a1 = total & ~(int64_t)15;
  return {a0, (int)(b0 - a0), a1 > a0 ? (int)(a1 - a0) : 0, a1 >= b1};
}

// A thread's elements come in chunks, pairs of fp32: a vector of the row, or
// eight single elements where rows are not whole vectors.
template <typename T, bool WHOLE>
struct Chunk {
  static constexpr int N = WHOLE ? Vec<T>::N : 8;
};

// Chunk i of a row, from the ring.  Past the row's end come zeros, or `fill`
// where rows are not whole vectors.
template <typename T, bool WHOLE>
__device__ __forceinline__ void take(const char* stage, const Span& sp, const T* tensor, int r, int tpr, int d, int i,
                                     float2 (&v)[Chunk<T, WHOLE>::N / 2], float fill = 0.f) {
  if constexpr (WHOLE) {
    const int q = r + i * tpr;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (q * Vec<T>::N < d) u = *reinterpret_cast<const uint4*>(stage + q * 16);
    float w[Vec<T>::N];
    unpack(u, w);
#pragma unroll
    for (int j = 0; j < Vec<T>::N; j += 2) v[j / 2] = make_float2(w[j], w[j + 1]);
  } else {
    const int step = tpr * (int)sizeof(T), left = ((d - r + tpr - 1) >> (31 - __clz(tpr))) - i * 8;  // the thread's elements from here on
    int at = sp.skip + (r + i * 8 * tpr) * (int)sizeof(T);
    if (sp.whole) {
      const char* p = stage + at;
#pragma unroll
      for (int j = 0; j < 8; ++j, p += step) {
        const float w = j < left ? to_f32(*reinterpret_cast<const T*>(p)) : fill;
        (j & 1 ? v[j / 2].y : v[j / 2].x) = w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j, at += step) {
        float w = fill;
        if (j < left)
          w = to_f32(at < sp.bytes ? *reinterpret_cast<const T*>(stage + at) : tensor[(sp.at + at) / (int64_t)sizeof(T)]);
        (j & 1 ? v[j / 2].y : v[j / 2].x) = w;
      }
    }
  }
}
template <typename T, bool WHOLE>
__device__ __forceinline__ void put(T* row, int r, int tpr, int d, int i, const float2 (&v)[Chunk<T, WHOLE>::N / 2]) {
  if constexpr (WHOLE) {
    const int q = r + i * tpr;
    float w[Vec<T>::N];
#pragma unroll
    for (int j = 0; j < Vec<T>::N; j += 2) {
      w[j] = v[j / 2].x;
      w[j + 1] = v[j / 2].y;
    }
    if (q * Vec<T>::N < d) stg16(row + (size_t)q * Vec<T>::N, pack(w));
  } else {
    const int left = ((d - r + tpr - 1) >> (31 - __clz(tpr))) - i * 8;
    T* p = row + r + i * 8 * tpr;
#pragma unroll
    for (int j = 0; j < 8; ++j, p += tpr)
      if (j < left) *p = from_f32<T>(j & 1 ? v[j / 2].y : v[j / 2].x);
  }
}

// The columns' weights, in pairs (0 past the row's end).
template <int VN>
__device__ __forceinline__ void take_weights(const float* w, int r, int tpr, int d, float2 (&v)[EPT / 2]) {
#pragma unroll
  for (int c = 0; c < EPT; ++c) {
    const float u = in_row<VN>(r, tpr, c, d) ? __ldg(w + column<VN>(r, tpr, c)) : 0.f;
    (c & 1 ? v[c / 2].y : v[c / 2].x) = u;
  }
}

// VN elements: a 16-byte vector, or one
template <typename T, int VN>
__device__ __forceinline__ void ld_n(const T* p, float (&v)[VN]) {
  if constexpr (VN == 1) v[0] = to_f32(*p);
  else unpack(*reinterpret_cast<const uint4*>(p), v);
}
template <int VN>
__device__ __forceinline__ void ld_w(const float* p, float (&v)[VN]) {  // of the weights
  if constexpr (VN == 1) {
    v[0] = __ldg(p);
  } else {
#pragma unroll
    for (int j = 0; j < VN; j += 4) {
      const float4 w = __ldg(reinterpret_cast<const float4*>(p + j));
      v[j] = w.x;
      v[j + 1] = w.y;
      v[j + 2] = w.z;
      v[j + 3] = w.w;
    }
  }
}
template <typename T, int VN>
__device__ __forceinline__ void st_n(T* p, const float (&v)[VN]) {
  if constexpr (VN == 1) *p = from_f32<T>(v[0]);
  else stg16(p, pack(v));
}

// Threads that share a row: as few as hold it, a warp at least.
int threads_per_row(int d) {
  int tpr = 32;
  while (tpr * EPT < d) tpr *= 2;
  return tpr;
}
}  // namespace
}  // namespace moe
