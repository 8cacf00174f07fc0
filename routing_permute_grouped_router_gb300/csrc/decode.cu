// The whole layer for a few tokens in one kernel: host side, and the kernel
// for fp32 weights.
//
//   y[t] = residual[t] + sum over kept picks j of
//          g_tj * (silu(x_t W1_e) * (x_t W3_e)) W2_e,   e = ids[t, j]
//
// With few tokens the layer is bound by reading the picked experts' weights
// once from HBM, and everything else has to stay out of the way.  One
// cooperative launch, one CTA an SM (two for fp32 weights), in three steps:
//   1. the CTAs score slices of d for groups of tokens, meet at a grid
//      barrier, and each derives the same picks and row lists;
//   2. up product: the W1 and W3 tiles (128 columns, all of d) of the experts
//      that have rows, split evenly over the CTAs in units of rows of d; the
//      CTAs that share a tile add their fp32 partial sums in CTA order, each a
//      share of them, and write h = g * silu(a) * b;
//   3. after a second grid barrier the down product, its W2 tiles (128 columns
//      of y, all experts in turn) split the same way; a CTA adds its experts'
//      rows to the tokens in shared memory, and the CTAs that share a column
//      tile add their sums in CTA order and write y.
// Where rows are few, step 3 makes h from the partial sums itself (few_rows).
// Nothing is summed in an order that depends on timing.
// Measured for fp32: seven tokens of a layer with d 1024, f 4096, eight experts,
// top-2 (352 MB of weights), 84 us; the SMs get unequal shares of HBM, and the
// CTAs wait for the slowest between the products.  Handing the parts out while
// the kernel runs took 95 us: shorter parts cost more at their ends than the
// waits they save.
#include <stddef.h>

#include "decode.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int SM_NT = 256, SM_WARPS = SM_NT / 32;
constexpr int SM_CTAS = 2;   // CTAs an SM: one streams while the other stages or reduces
constexpr int SM_KR = 32;    // rows of a unit
constexpr int SM_KC = 512;   // rows whose inputs are staged at a time
constexpr int SM_TOK = 8;    // most tokens at a time

struct SimtSmem {
  Routing R;
  float yacc[DEC_T][DEC_N];
  union {
    ScoreScratch score;
    float in[SM_KC * SM_TOK];                  // [row][token]
    float red[SM_WARPS * SM_TOK * 2 * DEC_N];  // [warp][token][matrix][column]
  };
};
static_assert(offsetof(SimtSmem, red) % 16 == 0 && offsetof(SimtSmem, score) % 16 == 0, "read as float4");

// out(m, c, sums) for each of n <= TOK inputs and the 128 columns at c0 of MATS
// matrices (`width` columns wide): the sums over rows k0..k1 of in(m, k) *
// W[i][k][c].  The warps take rows in turn, a batch of them loaded at once
// (guarded: the rest of an unrolled loop would wait for each row), and add up
// through shared memory.
template <int TOK, int MATS, typename In, typename Out>
__device__ __forceinline__ void thin_product(SimtSmem& S, const float* const (&W)[2], int width, int c0, int k0, int k1,
                                             int n, In in, Out out) {
  constexpr int RB = 4;  // rows of a batch; eight only lengthen HBM's queue (float32 layer, seven tokens: 93 us, not 87)
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, c = c0 + lane * 4;
  float acc[TOK][MATS][4];
#pragma unroll
  for (int m = 0; m < TOK; ++m)
#pragma unroll
    for (int i = 0; i < MATS; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[m][i][j] = 0.f;
#pragma unroll 1
  for (int kc = k0; kc < k1; kc += SM_KC) {
    const int nk = k1 - kc < SM_KC ? k1 - kc : SM_KC;
    const int padded = (nk + SM_WARPS * RB - 1) / (SM_WARPS * RB) * (SM_WARPS * RB);
    __syncthreads();
#pragma unroll 1
    for (int r = threadIdx.x; r < padded; r += SM_NT) {
      float v[TOK];
#pragma unroll
      for (int m = 0; m < TOK; ++m) v[m] = m < n && r < nk ? in(m, kc + r) : 0.f;
#pragma unroll
      for (int m = 0; m < TOK; ++m) S.in[r * TOK + m] = v[m];
    }
    __syncthreads();
    if (c < width) {
#pragma unroll 1
      for (int r0 = warp; r0 < nk; r0 += SM_WARPS * RB) {
        float w[RB][MATS][4];
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          const int r = r0 + b * SM_WARPS;
#pragma unroll
          for (int i = 0; i < MATS; ++i) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (r < nk) u = ldg16(W[i] + (int64_t)(kc + r) * width + c);
            unpack(u, w[b][i]);
          }
        }
#pragma unroll
        for (int b = 0; b < RB; ++b)
#pragma unroll
          for (int m = 0; m < TOK; ++m) {
            const float x = S.in[(r0 + b * SM_WARPS) * TOK + m];
#pragma unroll
            for (int i = 0; i < MATS; ++i)
#pragma unroll
              for (int j = 0; j < 4; ++j) acc[m][i][j] = fmaf(x, w[b][i][j], acc[m][i][j]);
          }
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < TOK; ++m)
#pragma unroll
    for (int i = 0; i < MATS; ++i)
      *reinterpret_cast<float4*>(S.red + ((warp * TOK + m) * MATS + i) * DEC_N + lane * 4) =
          make_float4(acc[m][i][0], acc[m][i][1], acc[m][i][2], acc[m][i][3]);
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < n * DEC_N; i += SM_NT) {
    const int m = i / DEC_N, col = i % DEC_N;
    float v[2] = {0.f, 0.f};
#pragma unroll
    for (int w = 0; w < SM_WARPS; ++w)
#pragma unroll
      for (int q = 0; q < MATS; ++q) v[q] += S.red[((w * TOK + m) * MATS + q) * DEC_N + col];
    if (c0 + col < width) out(m, col, v);
  }
}

// The product for n rows, as many at a time as fit the registers.
template <int MATS, typename In, typename Out>
__device__ __forceinline__ void thin_products(SimtSmem& S, const float* const (&W)[2], int width, int c0, int k0, int k1,
                                              int n, In in, Out out) {
#pragma unroll 1
  for (int m0 = 0; m0 < n;) {
    const int left = n - m0;
    auto in0 = [&](int m, int k) { return in(m0 + m, k); };
    auto out0 = [&](int m, int col, const float (&v)[2]) { out(m0 + m, col, v); };
    if (left > 4) {
      thin_product<8, MATS>(S, W, width, c0, k0, k1, left < 8 ? left : 8, in0, out0);
      m0 += 8;
    } else if (left > 2) {
      thin_product<4, MATS>(S, W, width, c0, k0, k1, left, in0, out0);
      m0 += 4;
    } else {
      thin_product<2, MATS>(S, W, width, c0, k0, k1, left, in0, out0);
      m0 += 2;
    }
  }
}

__global__ void __launch_bounds__(SM_NT, SM_CTAS) decode_kernel(const __grid_constant__ DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  SimtSmem& S = *reinterpret_cast<SimtSmem*>(smem_raw);
  Routing& R = S.R;
  route<float, SM_NT>(a, S.score, R);
  const int G = gridDim.x, c = blockIdx.x, tid = threadIdx.x;
  const float* x = static_cast<const float*>(a.io.x);
  float* h = static_cast<float*>(a.h);
  const int FT = (a.f + DEC_N - 1) / DEC_N, DT = (a.d + DEC_N - 1) / DEC_N;
  const int KU = (a.d + SM_KR - 1) / SM_KR, KD = (a.f + SM_KR - 1) / SM_KR;

  // ---- up product ----
  const int64_t pslot = (int64_t)a.T * 2 * DEC_N;
  const int per = R.nact * KD;  // units of a column tile of y: all experts' rows of W2
  const Split up(R.nact * FT * KU, G), down(per * DT, G);
  const bool direct = few_rows(a, R);
  // the sums of the parts
  auto add_parts = [&](int first, int segs, int i, float& va, float& vb) {
    for (int s = 0; s < segs; ++s) {
      const float* p = a.up_part + ((int64_t)(first + s) * 2 + (s > 0 ? 0 : 1)) * pslot + i;
      va += __ldcg(p);
      vb += __ldcg(p + DEC_N);
    }
  };
  // h of the sums i0..i1 of a tile (row, column) from the parts of its `segs` CTAs
  auto finish_up = [&](int tile, int first, int segs, int i0, int i1) {
    const int f0 = tile % FT * DEC_N, base = R.base[R.act[tile / FT]];
    for (int i = i0 + tid; i < i1; i += SM_NT) {
      const int m = i / DEC_N, col = i % DEC_N;
      float va = 0.f, vb = 0.f;
      add_parts(first, segs, m * 2 * DEC_N + col, va, vb);
      if (f0 + col < a.f) h[(int64_t)(base + m) * a.f + f0 + col] = R.gate[base + m] * dec_silu(va) * vb;
    }
  };
  if (R.nact > 0) {
    const int u0 = up.begin(c), u1 = up.begin(c + 1);
    for (int u = u0; u < u1;) {
      const int tile = u / KU;
      const int kb0 = u - tile * KU, kb1 = u1 - tile * KU < KU ? u1 - tile * KU : KU;
      const int e = R.act[tile / FT], f0 = tile % FT * DEC_N, n = R.cnt[e], base = R.base[e];
      const int k0 = kb0 * SM_KR, k1 = kb1 * SM_KR < a.d ? kb1 * SM_KR : a.d;
      float* part = a.up_part + ((int64_t)c * 2 + (kb0 > 0 ? 0 : 1)) * pslot;
      const float* const W[2] = {static_cast<const float*>(a.io.W1) + (int64_t)e * a.d * a.f,
                                 static_cast<const float*>(a.io.W3) + (int64_t)e * a.d * a.f};
      thin_products<2>(S, W, a.f, f0, k0, k1, n, [&](int m, int k) { return x[(int64_t)R.tok[base + m] * a.d + k]; },
                       [&](int m, int col, const float (&v)[2]) {
                         part[(int64_t)m * 2 * DEC_N + col] = v[0];
                         part[(int64_t)m * 2 * DEC_N + DEC_N + col] = v[1];
                       });
      if (kb0 == 0 && kb1 == KU) {
        __syncthreads();
        finish_up(tile, c, 1, 0, n * DEC_N);
      }
      u += kb1 - kb0;
    }
    // The other CTAs of the first and the last tile are told at the end: a
    // release in between would hold everyone up for as long as HBM's queue is.
    __syncthreads();
    if (tid == 0 && !direct) {
      for (int u = u0; u < u1;) {
        const int tile = u / KU, end = (tile + 1) * KU, first = up.owner(tile * KU);
        if (up.owner(end - 1) > first) red_release(a.ctr + first);
        u = end < u1 ? end : u1;
      }
    }
    if (tid == 0 && direct) red_release(a.ctr + 2 * G);
    // a share of each tile that other CTAs have a part of
    for (int u = u0; u < u1 && !direct;) {
      const int tile = u / KU, end = (tile + 1) * KU;
      const int first = up.owner(tile * KU), segs = up.owner(end - 1) - first + 1;
      if (segs > 1) {
        __syncthreads();
        if (tid == 0) wait_count(a.ctr + first, segs, a.err, 700);
        __syncthreads();
        const int N = R.cnt[R.act[tile / FT]] * DEC_N;
        finish_up(tile, first, segs, (int)((int64_t)(c - first) * N / segs), (int)((int64_t)(c - first + 1) * N / segs));
      }
      u = end < u1 ? end : u1;
    }
  }
  if (direct) {
    if (tid == 0) wait_count(a.ctr + 2 * G, G, a.err, 702);
    __syncthreads();
  } else {
    cg::this_grid().sync();
  }

  // ---- down product ----
  const int64_t dslot = (int64_t)a.T * DEC_N;
  const float* res = static_cast<const float*>(a.io.residual);
  float* y = static_cast<float*>(a.io.y);
  if (R.nact == 0) {  // every assignment was dropped
    for (int64_t i = (int64_t)c * SM_NT + tid; i < (int64_t)a.T * a.d; i += (int64_t)G * SM_NT)
      y[i] = res ? res[i] : 0.f;
    return;
  }
  // y of the sums i0..i1 (token, column) of a column tile: eight threads a sum, each some of the parts
  auto finish_down = [&](int dt, int first, int segs, int i0, int i1) {
    const int sub = tid % 8;
#pragma unroll 1
    for (int ib = i0; ib < i1; ib += SM_NT / 8) {
      const int i = ib + tid / 8, t = i / DEC_N, col = dt * DEC_N + i % DEC_N;
      float v = 0.f;
#pragma unroll 1
      for (int s0 = sub; s0 < segs; s0 += 64) {
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
          w[j] = i < i1 && s0 + 8 * j < segs ? __ldcg(a.down_part + (int64_t)(first + s0 + 8 * j + dt) * dslot + i) : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) v += w[j];
      }
#pragma unroll
      for (int o = 1; o < 8; o *= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (sub == 0 && i < i1 && col < a.d) {
        const int64_t o = (int64_t)t * a.d + col;
        y[o] = res ? v + res[o] : v;
      }
    }
  };
  const int u0 = down.begin(c), u1 = down.begin(c + 1);
  for (int u = u0; u < u1;) {
    const int dt = u / per, end = (dt + 1) * per < u1 ? (dt + 1) * per : u1;
    const int d0 = dt * DEC_N;
    __syncthreads();
    for (int i = tid; i < a.T * DEC_N; i += SM_NT) (&S.yacc[0][0])[i] = 0.f;
    __syncthreads();
    float* part = a.down_part + (c + dt) * dslot;
    const bool whole = u == dt * per && end == (dt + 1) * per;
    while (u < end) {
      const int q = u - dt * per, ai = q / KD, kb0 = q - ai * KD;
      const int kb1 = end - u < KD - kb0 ? kb0 + end - u : KD;
      const int e = R.act[ai], n = R.cnt[e], base = R.base[e];
      const int k0 = kb0 * SM_KR, k1 = kb1 * SM_KR < a.f ? kb1 * SM_KR : a.f;
      const float* const W[2] = {static_cast<const float*>(a.io.W2) + (int64_t)e * a.f * a.d, nullptr};
      auto in = [&](int m, int k) {
        if (direct) {
          const int tile = ai * FT + k / DEC_N, first = up.owner(tile * KU), segs = up.owner(tile * KU + KU - 1) - first + 1;
          if (segs > 1) {
            float va = 0.f, vb = 0.f;
            add_parts(first, segs, m * 2 * DEC_N + k % DEC_N, va, vb);
            return R.gate[base + m] * dec_silu(va) * vb;
          }
        }
        return __ldcg(h + (int64_t)(base + m) * a.f + k);
      };
      thin_products<1>(S, W, a.d, d0, k0, k1, n, in,
                       [&](int m, int col, const float (&v)[2]) { S.yacc[R.tok[base + m]][col] += v[0]; });
      u += kb1 - kb0;
    }
    __syncthreads();
    for (int i = tid; i < a.T * DEC_N; i += SM_NT) part[i] = (&S.yacc[0][0])[i];
    if (whole) {
      __syncthreads();
      finish_down(dt, c, 1, 0, a.T * DEC_N);
    }
  }
  __syncthreads();
  if (tid == 0) {
    for (int u = u0; u < u1;) {
      const int dt = u / per, end = (dt + 1) * per, first = down.owner(dt * per);
      if (down.owner(end - 1) > first) red_release(a.ctr + G + first);
      u = end < u1 ? end : u1;
    }
  }
  for (int u = u0; u < u1;) {
    const int dt = u / per, end = (dt + 1) * per;
    const int first = down.owner(dt * per), segs = down.owner(end - 1) - first + 1;
    if (segs > 1) {
      __syncthreads();
      if (tid == 0) wait_count(a.ctr + G + first, segs, a.err, 701);
      __syncthreads();
      const int N = a.T * DEC_N;
      finish_down(dt, first, segs, (int)((int64_t)(c - first) * N / segs),
                  (int)((int64_t)(c - first + 1) * N / segs));
    }
    u = end < u1 ? end : u1;
  }
}

// ------------------------------ host side --------------------------------- //
int decode_ctas(const Shape& s) { return sm_count() * (s.bf16 ? 1 : SM_CTAS); }
inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct DecodeWs {
  size_t score, ids, gates, ctr, h, up, whole, down, total;
};
DecodeWs decode_ws(const Shape& s) {
  const size_t G = decode_ctas(s), T = s.T, DT = (s.d + DEC_N - 1) / DEC_N;
  DecodeWs w{};
  w.score = 0;
  w.ids = w.score + up256(G * DEC_TG * s.E * 4);
  w.gates = w.ids + up256(T * s.k * 4);
  w.ctr = w.gates + up256(T * s.k * 4);
  w.h = w.ctr + up256((2 * G + 3) * 4);
  w.up = w.h + up256(s.bf16 ? decode_tc_h_bytes(s) : T * s.k * s.f * 4);
  w.whole = w.up + up256(2 * G * 2 * T * 2 * DEC_N * 4);
  w.down = w.whole + up256(s.bf16 ? decode_tc_whole_bytes(s) : 0);
  w.total = w.down + up256(2 * (G + DT) * T * DEC_N * 4);
  return w;
}

cudaError_t launch_simt(DecodeArgs a, int G, cudaStream_t st) {
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  if (!attr_done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)sizeof(SimtSmem));
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  void* args[] = {&a};
  LaunchScope ls(KK_DECODE, st);
  return cudaLaunchCooperativeKernel((const void*)decode_kernel, dim3(G), dim3(SM_NT), args, sizeof(SimtSmem), st);
}

}  // namespace

size_t decode_ws_bytes(const Shape& s) { return decode_ws(s).total + 256; }

cudaError_t launch_decode(const Shape& s, const DecodeIo& io, void* ws, uint32_t* err, cudaStream_t st) {
  char* base = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(ws) + 255) / 256 * 256);
  const DecodeWs w = decode_ws(s);
  const int G = decode_ctas(s);
  DecodeArgs a{};
  a.io = io;
  a.score_part = reinterpret_cast<float*>(base + w.score);
  a.ids = reinterpret_cast<int32_t*>(base + w.ids);
  a.gates = reinterpret_cast<float*>(base + w.gates);
  a.ctr = reinterpret_cast<uint32_t*>(base + w.ctr);
  a.h = base + w.h;
  a.up_part = reinterpret_cast<float*>(base + w.up);
  a.up_whole = reinterpret_cast<float*>(base + w.whole);
  a.down_part = reinterpret_cast<float*>(base + w.down);
  a.err = err;
  a.T = s.T;
  a.d = s.d;
  a.f = s.f;
  a.E = s.E;
  a.k = s.k;
  a.cap = s.cap;
  a.groups = (s.T + DEC_TG - 1) / DEC_TG;
  // slices of one batch of W_r loads (eight a thread), of at least 32 rows, and no more of them than CTAs
  const int rows = 2048 / s.E < 32 ? 32 : (2048 / s.E > 256 ? 256 : 2048 / s.E);
  a.slices = (s.d + rows - 1) / rows;
  if (a.slices > G / a.groups) a.slices = G / a.groups;
  return s.bf16 ? launch_decode_tc(s, a, G, st) : launch_simt(a, G, st);
}

}  // namespace moe
