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
  int32_t* ids;       // [T, k] picks and their gates, from the CTA that made them to the others
  float* gates;
  uint32_t* ctr;      // [2 G + 3]: arrivals at split tiles and grid barriers
  void* h;            // rows of the experts, gate * silu(a) * b: [T k][f] fp32, or tiles of bf16 (decode_tc.cu)
  float* up_part;     // [2][G][2][T][2 * DEC_N] a and b of split tiles
  float* up_whole;    // [T k][f / DEC_N][2 * DEC_N] a and b of tiles that are not split (decode_tc.cu, few rows)
  float* down_part;   // [2][G + column tiles][T][DEC_N] sums of the CTAs over their part of a column tile
  uint32_t* err;
  int T, d, f, E, k, cap;
  int groups, slices;  // of the scores: groups of DEC_TG tokens, slices of d
};
// decode_tc.cu: bf16 layers, G CTAs
size_t decode_tc_h_bytes(const Shape& s);
size_t decode_tc_whole_bytes(const Shape& s);
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
  float gates[DEC_ROWS];  // [T, k]
  float gate[DEC_ROWS];   // gate of each row
  int16_t slot[DEC_ROWS];  // in visiting order: choice-major, then token
  uint8_t ids[DEC_ROWS];   // [T, k]
  uint8_t tok[DEC_ROWS];   // token of each row
  int cnt[DEC_E];          // kept rows of each expert
  int16_t base[DEC_E];     // first row of each expert
  int16_t block[DEC_E];    // first block of 16 rows of each expert, where each begins a block (bf16: rows of h)
  uint8_t act[DEC_E];      // experts with rows
  int nact, rows;          // experts with rows, and all their rows
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
// U equal units in order: the first U % G CTAs take one more than the others,
// so with fewer units than CTAs the last ones take none.  A tile of several
// units can begin in one CTA and end in another, so every CTA streams the same
// bytes to within a unit whatever the number of tiles.  U < 2^28 by the limits
// on d, f and E.
struct Split {
  int base, more;
  __device__ __forceinline__ Split(int U, int G) : base(U / G), more(U % G) {}
  __device__ __forceinline__ int begin(int c) const { return c * base + (c < more ? c : more); }
  __device__ __forceinline__ int owner(int u) const {
    const int big = more * (base + 1);
    return u < big ? u / (base + 1) : more + (u - big) / base;
  }
};

// Few rows: the partial sums of the up product go straight to the CTAs of the
// down product, which add them and make h for themselves.  That repeats the
// sums in every column tile of y but saves an exchange: the CTAs of a split
// tile add a share of its parts each and write h, and all wait for that (a
// fence, a wait and a barrier of some 2 us each under load).
// One token of a dropless top-4 layer of 32 experts: 39 us, and 44 with the
// exchange; 8 tokens of it, three rows an expert: 91 and 75.
constexpr int DEC_DIRECT = 64;  // most picks of such a call
__device__ __forceinline__ bool few_rows(const DecodeArgs& a, const Routing& R) {
  return a.T * a.k <= DEC_DIRECT && R.nact > 0 && R.rows <= 2 * R.nact;
}

// ---- scores ----
// The kernel runs once through most of its code, and every 128-byte line of
// it that is not yet in an SM's instruction cache costs an L2 or DRAM latency:
// the loops from here on are kept rolled and the bodies short (the unrolled
// forms of the score, pick and epilogue loops cost a one-token step 20 us).
struct alignas(16) ScoreScratch {
  float w[8192];            // rows of W_r
  float x[256 * DEC_TG];    // the same columns of the tokens
  float red[256 * DEC_TG];
};
__device__ __forceinline__ void copy4(float* dst, const float* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ int pow2_at_least(int e) { return e <= 1 ? 1 : 1 << (32 - __clz(e - 1)); }

// Partial logits of DEC_TG tokens over one slice of d, so W_r is read once a
// group.  256 threads take `subs` rows at a time; the sums run in a fixed order.
template <typename T, int NT>
__device__ __forceinline__ void score_slice(const DecodeArgs& a, ScoreScratch& s) {
  const int unit = blockIdx.x;
  if (unit >= a.groups * a.slices) return;
  const int grp = unit / a.slices, sl = unit - grp * a.slices, t0 = grp * DEC_TG;
  const int r0 = (int)((int64_t)sl * a.d / a.slices), r1 = (int)((int64_t)(sl + 1) * a.d / a.slices);
  const int ep = pow2_at_least(a.E), subs = 256 / ep;
  const int e = threadIdx.x & (ep - 1), sub = threadIdx.x / ep, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const bool on = threadIdx.x < 256 && e < a.E;
  const int most = 8192 / a.E < 256 ? 8192 / a.E : 256;
  float acc[DEC_TG];
#pragma unroll
  for (int t = 0; t < DEC_TG; ++t) acc[t] = 0.f;
#pragma unroll 1
  for (int c0 = r0; c0 < r1; c0 += most) {
    const int n = r1 - c0 < most ? r1 - c0 : most;
    __syncthreads();
    const float* W = a.io.W_r + (int64_t)c0 * a.E;
    const T* x = static_cast<const T*>(a.io.x) + (int64_t)(t0 + warp) * a.d + c0;
    const bool live = warp < DEC_TG && t0 + warp < a.T;
    // all loads at once: W_r by asynchronous copies, x in a guarded batch (the
    // rest of an unrolled loop would take them one latency at a time)
#pragma unroll 2
    for (int i = threadIdx.x; i < n * a.E; i += NT) copy4(s.w + i, W + i);
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = live && lane + 32 * j < n ? to_f32(x[lane + 32 * j]) : 0.f;
    if (warp < DEC_TG) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s.x[(lane + 32 * j) * DEC_TG + warp] = v[j];
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    if (on) {
#pragma unroll 2
      for (int r = sub; r < n; r += subs) {
        const float w = s.w[r * a.E + e];
        const float4 p = *reinterpret_cast<const float4*>(s.x + r * DEC_TG);
        const float4 q = *reinterpret_cast<const float4*>(s.x + r * DEC_TG + 4);
        acc[0] = fmaf(p.x, w, acc[0]);
        acc[1] = fmaf(p.y, w, acc[1]);
        acc[2] = fmaf(p.z, w, acc[2]);
        acc[3] = fmaf(p.w, w, acc[3]);
        acc[4] = fmaf(q.x, w, acc[4]);
        acc[5] = fmaf(q.y, w, acc[5]);
        acc[6] = fmaf(q.z, w, acc[6]);
        acc[7] = fmaf(q.w, w, acc[7]);
      }
    }
  }
  if (on) {
#pragma unroll
    for (int t = 0; t < DEC_TG; ++t) s.red[(t * subs + sub) * ep + e] = acc[t];
  }
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < DEC_TG * ep; i += NT) {
    const int t = i / ep, ee = i & (ep - 1);
    if (ee >= a.E || t0 + t >= a.T) continue;
    float v = 0.f;
#pragma unroll 4
    for (int q = 0; q < subs; ++q) v += s.red[(t * subs + q) * ep + ee];
    a.score_part[((int64_t)unit * DEC_TG + t) * a.E + ee] = v;
  }
}

// Logits of `n` <= DEC_TG tokens of one group from token t0 on, added over the
// slices; token t0 + i is then picked for by warp i, as router_topk_kernel
// does it: NaN scores count as -inf, ties go to the lower expert.  put(t, j,
// expert, gate) is called once for each pick.
template <int NT, typename Put>
__device__ __forceinline__ void pick_experts(const DecodeArgs& a, ScoreScratch& s, int t0, int n, Put put) {
  const int ep = pow2_at_least(a.E), np = pow2_at_least(n), warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int pairs = np * ep, subs = pairs < 256 ? 256 / pairs : 1;  // threads that share a sum
  const float* part = a.score_part + ((int64_t)(t0 / DEC_TG) * a.slices * DEC_TG + t0 % DEC_TG) * a.E;
  const int step = DEC_TG * a.E;
#pragma unroll 1
  for (int i = threadIdx.x; i < pairs * subs; i += NT) {
    const int e = i & (ep - 1), t = (i / ep) & (np - 1), sub = i / pairs;
    float v = 0.f;
    if (e < a.E && t < n) {
#pragma unroll 1
      for (int q0 = sub; q0 < a.slices; q0 += 8 * subs) {
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = q0 + j * subs < a.slices ? __ldcg(part + (q0 + j * subs) * step + t * a.E + e) : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) v += w[j];
      }
    }
    s.red[(t * subs + sub) * ep + e] = v;
  }
  __syncthreads();
  if (warp >= n) return;
  float* lg = s.x + warp * DEC_E;  // the token's logits
  uint32_t key[DEC_E / 32];        // ordered as the logits are; 0 for what cannot be picked
#pragma unroll
  for (int c = 0; c < DEC_E / 32; ++c) {
    const int e = lane + 32 * c;
    key[c] = 0;
    if (e < a.E) {
      float sc = a.io.bias ? __ldg(a.io.bias + e) : 0.f;
#pragma unroll 1
      for (int q = 0; q < subs; ++q) sc += s.red[(warp * subs + q) * ep + e];
      sc = isnan(sc) ? -INFINITY : sc + 0.f;  // -0 as 0
      lg[e] = sc;
      const uint32_t u = __float_as_uint(sc);
      key[c] = u & 0x80000000u ? ~u : u | 0x80000000u;
    }
  }
  float mx = 0.f, mine = 0.f;  // lane j keeps the j-th pick and its logit
  int pick = 0;
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    uint32_t bk = 0;
    int be = 0x7fffffff;
#pragma unroll
    for (int c = 0; c < DEC_E / 32; ++c)
      if (key[c] > bk) {
        bk = key[c];
        be = lane + 32 * c;
      }
    const uint32_t top = __reduce_max_sync(0xffffffffu, bk);
    be = __reduce_min_sync(0xffffffffu, bk == top ? be : 0x7fffffff);
#pragma unroll
    for (int c = 0; c < DEC_E / 32; ++c)
      if (be == lane + 32 * c) key[c] = 0;
    const float v = __uint_as_float(top & 0x80000000u ? top & 0x7fffffffu : ~top);
    if (j == 0) mx = v;
    if (lane == j) {
      mine = v;
      pick = be;
    }
  }
  // one pick: its probability over all experts; several: over the picks
  float ex = lane < a.k ? expf(mine - mx) : 0.f, den = ex;
  if (a.k == 1) {
    den = 0.f;
#pragma unroll 1
    for (int e = lane; e < a.E; e += 32) den += expf(lg[e] - mx);
  }
#pragma unroll 1
  for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  if (lane < a.k) put(t0 + warp, lane, pick, ex / den);
}

// Row lists of the experts: assignments are visited choice-major and then in
// token order, an expert keeps its first `cap`; its rows follow each other,
// without padding.
template <int NT>
__device__ __forceinline__ void list_rows(const DecodeArgs& a, Routing& R) {
  const int Tk = a.T * a.k, lane = threadIdx.x % 32;
  if (threadIdx.x < 32) {
    reinterpret_cast<int4*>(R.cnt)[lane] = make_int4(0, 0, 0, 0);
    __syncwarp();
#pragma unroll 1
    for (int i0 = 0; i0 < Tk; i0 += 32) {
      const int i = i0 + lane;
      const bool on = i < Tk;
      const int j = i / a.T, e = on ? R.ids[(i - j * a.T) * a.k + j] : -1;
      const uint32_t same = __match_any_sync(0xffffffffu, e);
      const int rank = __popc(same & ((1u << lane) - 1u));
      const int before = on ? R.cnt[e] : 0;
      if (on) R.slot[i] = (int16_t)(before + rank);
      __syncwarp();
      if (on && rank == 0) R.cnt[e] = before + __popc(same);
      __syncwarp();
    }
    // kept rows, their first rows and the experts that have any: four experts a lane
    const int4 c4 = reinterpret_cast<const int4*>(R.cnt)[lane];
    const int c[4] = {min(c4.x, a.cap), min(c4.y, a.cap), min(c4.z, a.cap), min(c4.w, a.cap)};
    reinterpret_cast<int4*>(R.cnt)[lane] = make_int4(c[0], c[1], c[2], c[3]);
    int own = 0;  // rows, and experts in the upper half
#pragma unroll
    for (int q = 0; q < 4; ++q) own += c[q] + (c[q] > 0 ? 1 << 16 : 0);
    int pre = own;
#pragma unroll 1
    for (int o = 1; o < 32; o *= 2) {
      const int u = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane >= o) pre += u;
    }
    const int nact = __shfl_sync(0xffffffffu, pre, 31) >> 16;
    if (lane == 31) {
      R.nact = nact;
      R.rows = pre & 0xffff;
    }
    pre -= own;
    // The r-th expert with rows is the (r * stride mod nact)-th of the list,
    // stride near 0.618 nact and without a common divisor: experts of
    // neighbouring indices, which can all be popular and cost a CTA more for
    // their rows, end up spread over the list, and so over the CTAs.  (64 tokens
    // of the Zipf-routed dropless layer: 150 us with a stride of 37.)
    int stride = 1;
    if (nact > 8) {
      int p = nact * 158 / 256 + lane, q = nact;
      while (q != 0) {
        const int t = p % q;
        p = q;
        q = t;
      }
      stride = nact * 158 / 256 + __ffs(__ballot_sync(0xffffffffu, p == 1)) - 1;
    }
    int blocks = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) blocks += (c[q] + 15) / 16;
    int at = blocks;
#pragma unroll 1
    for (int o = 1; o < 32; o *= 2) {
      const int u = __shfl_up_sync(0xffffffffu, at, o);
      if (lane >= o) at += u;
    }
    at -= blocks;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      R.block[lane * 4 + q] = (int16_t)at;
      at += (c[q] + 15) / 16;
      R.base[lane * 4 + q] = (int16_t)(pre & 0xffff);
      if (c[q] > 0) {
        R.act[(pre >> 16) * stride % nact] = (uint8_t)(lane * 4 + q);
        pre += c[q] + (1 << 16);
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < Tk; i += NT) {
    const int j = i / a.T, t = i - j * a.T, e = R.ids[t * a.k + j];
    if (R.slot[i] < R.cnt[e]) {
      const int row = R.base[e] + R.slot[i];
      R.tok[row] = (uint8_t)t;
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

// Scores, picks and row lists; every thread of every CTA takes part.  Up to
// DEC_TG tokens every CTA adds the slices and picks for itself; for more, one
// CTA a token does, and a second grid barrier hands the picks to the others.
template <typename T, int NT>
__device__ __forceinline__ void route(const DecodeArgs& a, ScoreScratch& s, Routing& R) {
  if (blockIdx.x == gridDim.x - 1)
    for (int i = threadIdx.x; i < 2 * (int)gridDim.x + 3; i += NT) a.ctr[i] = 0;
  score_slice<T, NT>(a, s);
  cooperative_groups::this_grid().sync();
  if (a.T <= DEC_TG) {
    pick_experts<NT>(a, s, 0, a.T, [&](int t, int j, int e, float g) {
      R.ids[t * a.k + j] = (uint8_t)e;
      R.gates[t * a.k + j] = g;
    });
    __syncthreads();
  } else {
    for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
      __syncthreads();
      pick_experts<NT>(a, s, t, 1, [&](int tt, int j, int e, float g) {
        a.ids[tt * a.k + j] = e;
        a.gates[tt * a.k + j] = g;
      });
    }
    cooperative_groups::this_grid().sync();
    for (int i = threadIdx.x; i < a.T * a.k; i += NT) {
      R.ids[i] = (uint8_t)__ldcg(a.ids + i);
      R.gates[i] = __ldcg(a.gates + i);
    }
    __syncthreads();
  }
  list_rows<NT>(a, R);
}

// expf: the error of __expf grows with |z|, and h feeds a float32 output
__device__ __forceinline__ float dec_silu(float z) { return z / (1.f + expf(-z)); }

}  // namespace
}  // namespace moe
