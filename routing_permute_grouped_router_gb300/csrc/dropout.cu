// Dropout whose mask is drawn from a counter and never stored, with the
// residual added in the same pass; the backward draws the same mask again.
//
// The generator is Philox-4x32-10 (J. Salmon, M. Moraes, R. Dror, D. Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011).  The block
// b = i / 8 of element i has the counter (b, offset), two 64-bit numbers, and
// the key is the seed; the 128 bits of a block are eight draws of 16 bits, low
// half of a word first.  Element i is kept when its draw is at least
// cut = round(65536 p), and scaled by 65536 / (65536 - cut).
//
// A draw has 16 bits rather than 32 so that one block serves eight elements, a
// 16-byte vector of bf16: half the integer work an element.  p is then
// realised to within 2^-17, and the scale is the inverse of the realised rate,
// so the expectation of the output is exact.
#include "block.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int DROP_THREADS = 256;

struct DropArgs {
  const void* y;
  const void* residual;
  void* out;
  int64_t n;
  uint64_t seed, offset;
  uint32_t cut;
  float scale, scale_lo;  // 65536 / (65536 - cut) in two parts
};

__device__ __forceinline__ uint4 philox(uint64_t block, uint64_t offset, uint64_t seed) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)p1;
    c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p0;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

__device__ __forceinline__ uint32_t draw_of(const uint4& u, int i) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  return (i & 1) ? w[i / 2] >> 16 : w[i / 2] & 0xFFFFu;
}
// res + y * (scale + lo), rounded once: the product's and the sum's rounding
// errors are formed exactly (two-sum) and added back, so a float32 output keeps
// its 24 bits where the residual and the scaled value cancel.  The rounded
// intrinsics keep the compiler from fusing the steps.
__device__ __forceinline__ float add_scaled(float res, float y, float scale, float lo) {
  const float p = __fmul_rn(y, scale), pe = __fmaf_rn(y, scale, -p);
  const float s = __fadd_rn(res, p), b = __fsub_rn(s, res);
  const float se = __fadd_rn(__fsub_rn(res, __fsub_rn(s, b)), __fsub_rn(p, b));
  return isfinite(s) ? __fadd_rn(s, __fadd_rn(se, __fmaf_rn(y, lo, pe))) : s;
}
// Keep or drop the eight values of a block and add the residual's; a dropped
// value is 0 whatever it was (infinities and NaN too).
template <typename T, bool RES>
__device__ __forceinline__ void drop8(float (&v)[8], const float (&r)[8], const uint4& u, const DropArgs& a) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const bool keep = draw_of(u, i) >= a.cut;
    if (RES && sizeof(T) == 4) {
      v[i] = keep ? add_scaled(r[i], v[i], a.scale, a.scale_lo) : r[i];
    } else {
      v[i] = keep ? v[i] * a.scale : 0.f;
      if (RES) v[i] += r[i];
    }
  }
}

// the eight values of a block's vectors (loaded plainly, not on the read-only path: out may be y or the residual)
template <typename T>
__device__ __forceinline__ void expand(const uint4 (&u)[8 / Vec<T>::N], float (&v)[8]) {
#pragma unroll
  for (int q = 0; q < 8 / Vec<T>::N; ++q) {
    float w[Vec<T>::N];
    unpack(u[q], w);
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) v[q * Vec<T>::N + i] = w[i];
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
#pragma unroll
  for (int q = 0; q < 8 / Vec<T>::N; ++q) {
    float w[Vec<T>::N];
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) w[i] = v[q * Vec<T>::N + i];
    stg16(p + q * Vec<T>::N, pack(w));
  }
}

// How a direction walks its blocks.  With a residual the next block is loaded
// before this one is drawn for, whose loads take about as long as the draws
// (2^27 bf16 values: 121 us; two blocks loaded and then drawn for: 136.  2^26
// float32 values: 121 and 131).  Without one two blocks are loaded together:
// the 32-bit products of the draws bound bf16 (2^27 values: 98 us; the next
// blocks loaded ahead: 103), and float32 is at HBM's rate either way.
template <typename T, bool RES>
struct Walk {
  static constexpr bool AHEAD = RES;
  static constexpr int B = AHEAD ? 1 : 2;
  static constexpr int RESIDENT = AHEAD ? (sizeof(T) == 2 ? 6 : 4) : 1;  // CTAs an SM that the registers leave room for
  static constexpr int CTAS = AHEAD ? 12 : 8;                            // launched an SM
};

template <typename T, bool RES>
__global__ void __launch_bounds__(DROP_THREADS, Walk<T, RES>::RESIDENT) dropout_kernel(const DropArgs a) {
  pdl_enter();  // see pdl_wait: no global access before this
  constexpr int Q = 8 / Vec<T>::N, B = Walk<T, RES>::B;
  constexpr bool AHEAD = Walk<T, RES>::AHEAD;
  const T* y = static_cast<const T*>(a.y);
  const T* res = static_cast<const T*>(a.residual);
  T* out = static_cast<T*>(a.out);
  const int64_t whole = a.n / 8, step = (int64_t)gridDim.x * DROP_THREADS;
  auto load = [&](const T* p, int64_t b, uint4 (&u)[B][Q]) {
#pragma unroll
    for (int j = 0; j < B; ++j)
      if (b + j * step < whole) {
#pragma unroll
        for (int q = 0; q < Q; ++q) u[j][q] = *reinterpret_cast<const uint4*>(p + (b + j * step) * 8 + q * Vec<T>::N);
      }
  };
  int64_t b0 = (int64_t)blockIdx.x * DROP_THREADS + threadIdx.x;
  uint4 u[B][Q], w[B][Q], u1[B][Q], w1[B][Q];
  if (AHEAD) {
    load(y, b0, u);
    if (RES) load(res, b0, w);
  }
#pragma unroll 1
  for (; b0 < whole; b0 += B * step) {
    load(y, AHEAD ? b0 + B * step : b0, AHEAD ? u1 : u);
    if (RES) load(res, AHEAD ? b0 + B * step : b0, AHEAD ? w1 : w);
#pragma unroll
    for (int j = 0; j < B; ++j) {
      const int64_t b = b0 + j * step;
      if (b < whole) {
        const uint4 draws = philox((uint64_t)b, a.offset, a.seed);
        float v[8], r[8];
        expand<T>(u[j], v);
        if (RES) expand<T>(w[j], r);
        drop8<T, RES>(v, r, draws, a);
        store8(out + b * 8, v);
      }
      if (AHEAD) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          u[j][q] = u1[j][q];
          w[j][q] = w1[j][q];
        }
      }
    }
  }
  // the last, short block
  if (a.n % 8 != 0 && blockIdx.x == 0 && threadIdx.x == 0) {
    const int64_t i0 = whole * 8;
    const int m = (int)(a.n - i0);
    float v[8], r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = i < m ? to_f32(y[i0 + i]) : 0.f;
      r[i] = RES && i < m ? to_f32(res[i0 + i]) : 0.f;
    }
    drop8<T, RES>(v, r, philox((uint64_t)whole, a.offset, a.seed), a);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < m) out[i0 + i] = from_f32<T>(v[i]);
  }
}

template <typename T, bool RES>
cudaError_t launch_drop(const DropArgs& a, cudaStream_t st) {
  using W = Walk<T, RES>;
  const int64_t need = ((a.n + 7) / 8 + DROP_THREADS - 1) / DROP_THREADS, most = (int64_t)sm_count() * W::CTAS;
  return launch_pdl(dropout_kernel<T, RES>, dim3((unsigned)(need < most ? need : most)), dim3(DROP_THREADS), 0, st, a);
}

}  // namespace

cudaError_t launch_dropout(int kind, int64_t n, bool bf16, const void* y, const void* residual, void* out,
                           uint32_t cut, uint64_t seed, uint64_t offset, cudaStream_t st) {
  const double scale = 65536.0 / (65536.0 - cut);
  const DropArgs a{y, residual, out, n, seed, offset, cut, (float)scale, (float)(scale - (float)scale)};
  LaunchScope ls(kind, st);
  if (bf16) return residual ? launch_drop<__nv_bfloat16, true>(a, st) : launch_drop<__nv_bfloat16, false>(a, st);
  return residual ? launch_drop<float, true>(a, st) : launch_drop<float, false>(a, st);
}

}  // namespace moe
