// Shared by the two kernels that run the whole layer for a few tokens
// (decode.cu: fp32 weights on the FMA units, decode_tc.cu: bf16 weights on the
// tensor cores): their arguments, the router, the row lists of the experts and
// the split of the weights over the CTAs.
#pragma once

#include <cooperative_groups.h>
#include <float.h>
#include <math.h>

#include "block.h"
#include "common.cuh"

namespace moe {

struct DecodeArgs {
  DecodeIo io;
  float* score_part;  // [groups][slices][DEC_TG][E] partial logits
  uint32_t* ctr;      // [2 G + 1]: arrivals at the split tiles of the up and the down product, and of the whole grid
  void* h;            // rows of the experts, gate * silu(a) * b: [T k][f] fp32, or [T k][hi f | lo f] bf16
  float* up_part;     // [G][2][T][2 * DEC_N] a and b of a split tile
  float* down_part;   // [G][2][T][DEC_N]
  uint32_t* err;
  int T, d, f, E, k, cap;
  int groups, slices;  // of the scores: groups of DEC_TG tokens, slices of d
};
// decode_tc.cu: bf16 layers, G CTAs
cudaError_t launch_decode_tc(const Shape& s, const DecodeArgs& args, int G, cudaStream_t st);

namespace {

constexpr int DEC_T = 64;          // most tokens (MOE_DECODE_MAX_T)
constexpr int DEC_K = 8;           // most picks a token
constexpr int DEC_ROWS = DEC_T * DEC_K;
constexpr int DEC_E = 128;
constexpr int DEC_N = 128;         // output columns of a weight tile
constexpr int DEC_TG = 8;          // tokens scored together
constexpr uint64_t DEC_WAIT_NS = 2000000000ull;  // a wait for another CTA gives up after 2 s

// What a CTA knows of the routing: every CTA derives the same.
struct alignas(16) Routing {
  int ids[DEC_ROWS];     // [T, k]
  float gates[DEC_ROWS];  // [T, k]
  int slot[DEC_ROWS];    // in visiting order: choice-major, then token
  int cnt[DEC_E];        // kept rows of each expert
  int base[DEC_E];       // first row of each expert
  int act[DEC_E];        // experts with rows
  int tok[DEC_ROWS];     // token of each row
  float gate[DEC_ROWS];  // gate of each row
  int nact;
};

__device__ __forceinline__ uint64_t dec_now() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void red_release(uint32_t* p) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(p) : "memory");
}
// One thread waits until `want` CTAs have arrived.  All CTAs are resident (a
// cooperative launch), so the limit is reached only if one of them gave up.
__device__ __forceinline__ bool wait_count(const uint32_t* p, uint32_t want, uint32_t* err, uint32_t where) {
  if (ld_acquire(p) >= want) return true;
  const uint64_t t0 = dec_now();
  for (uint32_t i = 1; i < (1u << 30); ++i) {
    if (ld_acquire(p) >= want) return true;
    if ((i & 63u) == 0 && dec_now() - t0 > DEC_WAIT_NS) break;
  }
  report_error(err, DEV_TIMEOUT, where);
  return false;
}

// ---- the split of the weights ----
// U equal units in order; the first G CTAs (all, or one a unit where there are
// fewer units) take [c U / G, (c + 1) U / G), the others nothing.  A tile of
// several units can begin in one CTA and end in another, so every CTA streams
// the same bytes to within a unit whatever the number of tiles.
struct Split {
  int64_t U;
  int G;
  __device__ __forceinline__ Split(int64_t units, int ctas) : U(units), G((int)(units < ctas ? units : ctas)) {}
  __device__ __forceinline__ int64_t begin(int c) const { return c < G ? c * U / G : U; }
  __device__ __forceinline__ int owner(int64_t u) const { return (int)(((u + 1) * G + U - 1) / U) - 1; }
};

// ---- scores ----
// Partial logits of DEC_TG tokens over one slice of d: W_r's rows are read
// once a group, the sum runs in a fixed order.
struct ScoreScratch {
  float x[256][DEC_TG];
  float red[256 * DEC_TG];
};
template <typename T, int NT>
__device__ __forceinline__ void score_slice(const DecodeArgs& a, ScoreScratch& s) {
  const int unit = blockIdx.x;
  if (unit >= a.groups * a.slices) return;
  const int grp = unit / a.slices, sl = unit % a.slices, t0 = grp * DEC_TG;
  const int r0 = (int)((int64_t)sl * a.d / a.slices), r1 = (int)((int64_t)(sl + 1) * a.d / a.slices);
  const T* x = static_cast<const T*>(a.io.x);
  int ep = 1;
  while (ep < a.E) ep *= 2;
  const int subs = 256 / ep, e = threadIdx.x % ep, sub = threadIdx.x / ep;  // sub rows at a time
  const bool on = threadIdx.x < 256 && e < a.E;
  float acc[DEC_TG];
#pragma unroll
  for (int t = 0; t < DEC_TG; ++t) acc[t] = 0.f;
  for (int c0 = r0; c0 < r1; c0 += 256) {
    const int n = r1 - c0 < 256 ? r1 - c0 : 256;
    __syncthreads();
    for (int i = threadIdx.x; i < n * DEC_TG; i += NT) {
      const int t = i / n, r = i % n;
      s.x[r][t] = t0 + t < a.T ? to_f32(x[(int64_t)(t0 + t) * a.d + c0 + r]) : 0.f;
    }
    __syncthreads();
    if (on) {
#pragma unroll 8
      for (int r = sub; r < n; r += subs) {
        const float w = __ldg(a.io.W_r + (int64_t)(c0 + r) * a.E + e);
#pragma unroll
        for (int t = 0; t < DEC_TG; ++t) acc[t] = fmaf(s.x[r][t], w, acc[t]);
      }
    }
  }
  if (on) {
#pragma unroll
    for (int t = 0; t < DEC_TG; ++t) s.red[(sub * DEC_TG + t) * ep + e] = acc[t];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < DEC_TG * a.E; i += NT) {
    const int t = i / a.E, ee = i % a.E;
    float v = 0.f;
    for (int q = 0; q < subs; ++q) v += s.red[(q * DEC_TG + t) * ep + ee];
    a.score_part[(int64_t)unit * DEC_TG * a.E + i] = v;
  }
}

// Softmax and top-k of every token (a warp a token), as router_topk_kernel
// does them: NaN scores count as -inf, ties go to the lower expert.
template <int NT>
__device__ __forceinline__ void pick_experts(const DecodeArgs& a, Routing& R) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int t = warp; t < a.T; t += NT / 32) {
    const float* part = a.score_part + ((int64_t)(t / DEC_TG) * a.slices * DEC_TG + t % DEC_TG) * a.E;
    float v[DEC_E / 32];
    float mx = -INFINITY;
#pragma unroll
    for (int c = 0; c < DEC_E / 32; ++c) {
      const int e = lane + 32 * c;
      float s = -INFINITY;
      if (e < a.E) {
        s = 0.f;
#pragma unroll 8
        for (int q = 0; q < a.slices; ++q) s += __ldcg(part + (int64_t)q * DEC_TG * a.E + e);
        if (a.io.bias) s += __ldg(a.io.bias + e);
        if (isnan(s)) s = -INFINITY;
      }
      v[c] = s;
      mx = fmaxf(mx, s);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    uint32_t taken = 0;
    float first = 0.f, den = 0.f, mine = 0.f;  // lane j keeps the j-th pick's exponential
    for (int j = 0; j < a.k; ++j) {
      float bv = -INFINITY;
      int be = 0x7fffffff;
#pragma unroll
      for (int c = 0; c < DEC_E / 32; ++c) {
        const int e = lane + 32 * c;
        if (e < a.E && !((taken >> c) & 1u) && (v[c] > bv || (v[c] == bv && e < be))) {
          bv = v[c];
          be = e;
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
        const int oe = __shfl_xor_sync(0xffffffffu, be, o);
        if (ov > bv || (ov == bv && oe < be)) {
          bv = ov;
          be = oe;
        }
      }
      if ((be & 31) == lane) taken |= 1u << (be >> 5);
      if (j == 0) first = bv;
      const float ex = a.k == 1 ? expf(bv - mx) : expf(bv - first);
      den += ex;
      if (lane == j) {
        mine = ex;
        R.ids[t * a.k + j] = be;
      }
    }
    if (a.k == 1) {  // one pick: its probability over all experts
      den = 0.f;
#pragma unroll
      for (int c = 0; c < DEC_E / 32; ++c)
        if (lane + 32 * c < a.E) den += expf(v[c] - mx);
      den = warp_sum(den);
    }
    if (lane < a.k) R.gates[t * a.k + lane] = mine / den;
  }
}

// Row lists of the experts: assignments are visited choice-major and then in
// token order, an expert keeps its first `cap`; its rows follow each other,
// without padding.
template <int NT>
__device__ __forceinline__ void list_rows(const DecodeArgs& a, Routing& R) {
  const int Tk = a.T * a.k, lane = threadIdx.x % 32;
  for (int e = threadIdx.x; e < DEC_E; e += NT) R.cnt[e] = 0;
  __syncthreads();
  if (threadIdx.x < 32) {
    for (int i0 = 0; i0 < Tk; i0 += 32) {
      const int i = i0 + lane;
      const bool on = i < Tk;
      const int e = on ? R.ids[(i % a.T) * a.k + i / a.T] : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      const int rank = __popc(same & ((1u << lane) - 1u));
      const int before = on ? R.cnt[e] : 0;
      if (on) R.slot[i] = before + rank;
      __syncwarp();
      if (on && rank == 0) R.cnt[e] = before + __popc(same);
      __syncwarp();
    }
    // kept rows, their first rows and the experts that have any
    int rows = 0, nact = 0;
#pragma unroll
    for (int c = 0; c < DEC_E / 32; ++c) {
      const int e = c * 32 + lane;
      int n = R.cnt[e];
      n = n < a.cap ? n : a.cap;
      int pre = n;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int u = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += u;
      }
      const uint32_t live = __ballot_sync(0xffffffffu, n > 0);
      R.cnt[e] = n;
      R.base[e] = rows + pre - n;
      if (n > 0) R.act[nact + __popc(live & ((1u << lane) - 1u))] = e;
      rows += __shfl_sync(0xffffffffu, pre, 31);
      nact += __popc(live);
    }
    if (lane == 0) R.nact = nact;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < Tk; i += NT) {
    const int t = i % a.T, j = i / a.T, e = R.ids[t * a.k + j];
    if (R.slot[i] < R.cnt[e]) {
      const int row = R.base[e] + R.slot[i];
      R.tok[row] = t;
      R.gate[row] = R.gates[t * a.k + j];
    }
  }
  if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i < Tk; i += NT) {
      if (a.io.ids) a.io.ids[i] = R.ids[i];
      if (a.io.gates) a.io.gates[i] = R.gates[i];
    }
  }
  __syncthreads();
}

// Scores, picks and row lists; every thread of every CTA takes part.
template <typename T, int NT>
__device__ __forceinline__ void route(const DecodeArgs& a, ScoreScratch& s, Routing& R) {
  if (blockIdx.x == gridDim.x - 1)
    for (int i = threadIdx.x; i < 2 * (int)gridDim.x + 1; i += NT) a.ctr[i] = 0;
  score_slice<T, NT>(a, s);
  cooperative_groups::this_grid().sync();
  pick_experts<NT>(a, R);
  __syncthreads();
  list_rows<NT>(a, R);
}

// expf: the error of __expf grows with |z|, and h feeds a float32 output
__device__ __forceinline__ float dec_silu(float z) { return z / (1.f + expf(-z)); }

}  // namespace
}  // namespace moe
