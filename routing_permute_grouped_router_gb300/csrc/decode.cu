// The whole layer for a few tokens in one kernel: host side, and the kernel
// for fp32 weights.
//
//   y[t] = residual[t] + sum over kept picks j of
//          g_tj * (silu(x_t W1_e) * (x_t W3_e)) W2_e,   e = ids[t, j]
//
// With few tokens the layer is bound by reading the picked experts' weights
// once from HBM, and everything else has to stay out of the way.  One
// cooperative launch, one CTA an SM, in three steps:
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
// Nothing is summed in an order that depends on timing.
#include "decode.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int SM_NT = 512, SM_WARPS = SM_NT / 32;
constexpr int SM_KR = 32;    // rows of a unit
constexpr int SM_KC = 1024;  // rows staged at a time
constexpr int SM_TOK = 8;    // tokens at a time

struct SimtSmem {
  Routing R;
  float yacc[DEC_T][DEC_N];
  union {
    ScoreScratch score;
    struct {
      float in[SM_KC][SM_TOK];
      float red[SM_WARPS][SM_TOK][DEC_N];
    };
  };
};

// out[m][c] = sum over rows k0..k1 of in(m, k) * W[k][c] for up to SM_TOK
// inputs and the 128 columns at c0 (`width` columns wide); the warps take
// rows in turn and add up through shared memory.  out(m, c, value) is called
// once for each of the n x 128 sums.
template <typename In, typename Out>
__device__ __forceinline__ void thin_product(SimtSmem& S, const float* W, int width, int c0, int k0, int k1, int n, In in,
                                             Out out) {
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, c = c0 + lane * 4;
  float acc[SM_TOK][4];
#pragma unroll
  for (int m = 0; m < SM_TOK; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[m][j] = 0.f;
  for (int kc = k0; kc < k1; kc += SM_KC) {
    const int nk = k1 - kc < SM_KC ? k1 - kc : SM_KC;
    __syncthreads();
    for (int i = threadIdx.x; i < nk * SM_TOK; i += SM_NT) {
      const int m = i / nk, r = i % nk;
      S.in[r][m] = m < n ? in(m, kc + r) : 0.f;
    }
    __syncthreads();
    if (c < width) {
#pragma unroll 4
      for (int r = warp; r < nk; r += SM_WARPS) {
        float w[4];
        unpack(ldg16(W + (int64_t)(kc + r) * width + c), w);
#pragma unroll
        for (int m = 0; m < SM_TOK; ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[m][j] = fmaf(S.in[r][m], w[j], acc[m][j]);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < SM_TOK; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j) S.red[warp][m][lane * 4 + j] = acc[m][j];
  __syncthreads();
  for (int i = threadIdx.x; i < n * DEC_N; i += SM_NT) {
    const int m = i / DEC_N, col = i % DEC_N;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < SM_WARPS; ++w) v += S.red[w][m][col];
    if (c0 + col < width) out(m, col, v);
  }
}

__global__ void __launch_bounds__(SM_NT, 1) decode_kernel(const __grid_constant__ DecodeArgs a) {
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
  const Split up(R.nact * FT * KU, G);
  // h of the sums i0..i1 of a tile (row, column) from the parts of its `segs` CTAs
  auto finish_up = [&](int tile, int first, int segs, int i0, int i1) {
    const int f0 = tile % FT * DEC_N, base = R.base[R.act[tile / FT]];
    for (int i = i0 + tid; i < i1; i += SM_NT) {
      const int m = i / DEC_N, col = i % DEC_N;
      float va = 0.f, vb = 0.f;
      for (int s = 0; s < segs; ++s) {
        const float* p = a.up_part + ((int64_t)(first + s) * 2 + (s > 0 ? 0 : 1)) * pslot + (int64_t)m * 2 * DEC_N + col;
        va += __ldcg(p);
        vb += __ldcg(p + DEC_N);
      }
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
      const float* W[2] = {static_cast<const float*>(a.io.W1) + (int64_t)e * a.d * a.f,
                       static_cast<const float*>(a.io.W3) + (int64_t)e * a.d * a.f};
      for (int m0 = 0; m0 < n; m0 += SM_TOK)
        for (int q = 0; q < 2; ++q)
          thin_product(S, W[q], a.f, f0, k0, k1, n - m0 < SM_TOK ? n - m0 : SM_TOK,
                       [&](int m, int k) { return x[(int64_t)R.tok[base + m0 + m] * a.d + k]; },
                       [&](int m, int col, float v) { part[(int64_t)(m0 + m) * 2 * DEC_N + q * DEC_N + col] = v; });
      if (kb0 > 0 || kb1 < KU) {  // shared: tell the others of the tile
        __threadfence();
        __syncthreads();
        if (tid == 0) red_release(a.ctr + up.owner(tile * KU));
      } else {
        __syncthreads();
        finish_up(tile, c, 1, 0, n * DEC_N);
      }
      u += kb1 - kb0;
    }
    // a share of each tile that other CTAs have a part of
    for (int u = u0; u < u1;) {
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
  cg::this_grid().sync();

  // ---- down product ----
  const int64_t dslot = (int64_t)a.T * DEC_N;
  const int per = R.nact * KD;  // units of a column tile: all experts' rows of W2
  const Split down(per * DT, G);
  const float* res = static_cast<const float*>(a.io.residual);
  float* y = static_cast<float*>(a.io.y);
  if (R.nact == 0) {  // every assignment was dropped
    for (int64_t i = (int64_t)c * SM_NT + tid; i < (int64_t)a.T * a.d; i += (int64_t)G * SM_NT)
      y[i] = res ? res[i] : 0.f;
    return;
  }
  auto finish_down = [&](int dt, int first, int segs, int i0, int i1) {
    for (int i = i0 + tid; i < i1; i += SM_NT) {
      const int t = i / DEC_N, col = dt * DEC_N + i % DEC_N;
      float v = 0.f;
      for (int s = 0; s < segs; ++s) v += __ldcg(a.down_part + (int64_t)(first + s + dt) * dslot + i);
      if (col < a.d) {
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
      for (int m0 = 0; m0 < n; m0 += SM_TOK)
        thin_product(S, static_cast<const float*>(a.io.W2) + (int64_t)e * a.f * a.d, a.d, d0, k0, k1,
                     n - m0 < SM_TOK ? n - m0 : SM_TOK,
                     [&](int m, int k) { return __ldcg(h + (int64_t)(base + m0 + m) * a.f + k); },
                     [&](int m, int col, float v) { S.yacc[R.tok[base + m0 + m]][col] += v; });
      u += kb1 - kb0;
    }
    __syncthreads();
    for (int i = tid; i < a.T * DEC_N; i += SM_NT) part[i] = (&S.yacc[0][0])[i];
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (tid == 0) red_release(a.ctr + G + down.owner(dt * per));
    } else {
      __syncthreads();
      finish_down(dt, c, 1, 0, a.T * DEC_N);
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
inline size_t up256(size_t x) { return (x + 255) / 256 * 256; }

struct DecodeWs {
  size_t score, ids, gates, ctr, h, up, whole, down, total;
};
DecodeWs decode_ws(const Shape& s) {
  const size_t G = sm_count(), T = s.T, DT = (s.d + DEC_N - 1) / DEC_N;
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
  const int G = sm_count();
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
