// The whole layer for a few tokens in one kernel, bf16 weights on the tensor
// cores.  The steps and the split of the weights over the CTAs are those of
// decode.cu.
//
// The weights are the M side of the products: a tile of 128 columns of W1 and
// W3 (or W2) is the A operand, stored with its columns contiguous (MN-major),
// and the tokens are the N side, 16 to 64 columns of the accumulator.  The MMAs
// of a 16 KB weight tile take a tenth of the time that HBM needs to deliver it
// to an SM, so the kernel is a stream of TMA loads with everything else behind:
//   warp 0, one lane: TMA producer.  A stage of the up product is 64 rows of d
//     of a W1 and a W3 tile and the same columns of all tokens; one of the down
//     product 64 rows of f of a W2 tile and those columns of the expert's rows
//     of h.  It fills the ring with the first W2 tiles before it waits for the
//     other CTAs' h, so HBM is busy across the grid barrier.
//   warp 1, one lane: MMAs.  Two accumulators in turn, so the next segment's
//     products run under a segment's epilogue.
//   warps 4-7: epilogue, one weight column a thread.
// h is split into two bf16 parts, hi + lo, whose products go to the same
// accumulator: 16 significant bits where one bf16 would round h to 8 and
// double the error of y.  The second product is free here.
#include <cudaTypedefs.h>

#include "decode.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int TC_NT = 256;
constexpr int TC_KB = 64;                 // rows of a unit: 128 bytes of a token's row
constexpr int TC_TILE = DEC_N * TC_KB * 2;  // 16 KB: two boxes of 64 columns x 64 rows
constexpr int TC_MAX_ST = 8;
constexpr int TC_SMEM_MAX = 232448;       // 227 KB a CTA
constexpr uint32_t TC_COLS = 256;         // TMEM: two accumulators of a and b, 64 tokens each
constexpr uint32_t TC_BUF = 128, TC_B = 64;

struct alignas(16) TcCtrl {
  uint64_t full[TC_MAX_ST], empty[TC_MAX_ST], tfull[2], tempty[2], drain;
  uint32_t tmem;
  int abort;
  int8_t row_of[4][DEC_T];  // a warp's map from token to the row of the segment's expert
};

struct TcMapsD {
  CUtensorMap x, W1, W3, W2, h;
};

__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// The epilogue warps agree whether to go on, so that a wait that gave up in one
// of them ends all of them at the same place.
__device__ __forceinline__ bool epi_all(bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void fence_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }
__host__ __device__ constexpr uint32_t dec_idesc(int n) {  // fp32 D, bf16 A (MN-major) and B (K-major), M = 128, N = n
  return (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(DEC_N >> 4) << 24);
}

// A CTA's consecutive units of one weight tile.
struct Seg {
  int e, n, base;  // expert, its rows, the first of them
  int c0;          // first weight column
  int kb0, kb1;    // units
  int64_t tile;    // up: the weight tile; down: the column tile of y
};
__device__ __forceinline__ Seg up_seg(const Routing& R, int64_t u, int64_t u1, int FT, int KU) {
  Seg s;
  s.tile = u / KU;
  s.kb0 = (int)(u - s.tile * KU);
  s.kb1 = (int)(u1 - s.tile * KU < KU ? u1 - s.tile * KU : KU);
  s.e = R.act[s.tile / FT];
  s.c0 = (int)(s.tile % FT) * DEC_N;
  s.n = R.cnt[s.e];
  s.base = R.base[s.e];
  return s;
}
__device__ __forceinline__ Seg down_seg(const Routing& R, int64_t u, int64_t u1, int64_t per, int KD) {
  Seg s;
  s.tile = u / per;
  const int64_t q = u - s.tile * per;
  const int ai = (int)(q / KD);
  s.kb0 = (int)(q - (int64_t)ai * KD);
  s.kb1 = u1 - u < KD - s.kb0 ? s.kb0 + (int)(u1 - u) : KD;
  s.e = R.act[ai];
  s.c0 = (int)s.tile * DEC_N;
  s.n = R.cnt[s.e];
  s.base = R.base[s.e];
  return s;
}
__device__ __forceinline__ int pad16(int n) { return (n + 15) & ~15; }

__device__ __forceinline__ void put_h(__nv_bfloat16* h, int64_t row, int f, int col, float v) {
  const __nv_bfloat16 hi = __float2bfloat16_rn(v);
  const float r = v - __bfloat162float(hi);
  h[row * 2 * f + col] = hi;
  h[row * 2 * f + f + col] = __float2bfloat16_rn(isfinite(r) ? r : 0.f);  // hi of an infinite v carries it alone
}

__global__ void __launch_bounds__(TC_NT, 1) decode_tc_kernel(const __grid_constant__ TcMapsD maps,
                                                             const __grid_constant__ DecodeArgs a, int nst, int slot) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Routing& R = *reinterpret_cast<Routing*>(smem + nst * slot);
  TcCtrl& C = *reinterpret_cast<TcCtrl*>(smem + nst * slot + sizeof(Routing));
  float* yacc = reinterpret_cast<float*>(smem + nst * slot + sizeof(Routing) + sizeof(TcCtrl));  // [T][DEC_N]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int* abort_flag = &C.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < nst; ++i) {
      mbar_init(smem_addr(&C.full[i]), 1);
      mbar_init(smem_addr(&C.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&C.tfull[i]), 1);
      mbar_init(smem_addr(&C.tempty[i]), 4);
    }
    mbar_init(smem_addr(&C.drain), 1);
    C.abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_map(&maps.x);
    prefetch_map(&maps.W1);
    prefetch_map(&maps.W3);
    prefetch_map(&maps.W2);
    prefetch_map(&maps.h);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(&C.tmem), TC_COLS);
    tmem_relinquish();
  }
  route<__nv_bfloat16, TC_NT>(a, *reinterpret_cast<ScoreScratch*>(smem), R);
  fence_async_smem();  // the ring held the scores: the TMA writes it from here on
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = C.tmem, ring = smem_addr(smem);

  const int G = gridDim.x, c = blockIdx.x;
  const int FT = a.f / DEC_N, DT = a.d / DEC_N, KU = a.d / TC_KB, KD = a.f / TC_KB;
  const int NT = pad16(a.T);
  const Split up((int64_t)R.nact * FT * KU, G);
  const int64_t per = (int64_t)R.nact * KD;
  const Split down(per * DT, G);
  const int64_t u0 = R.nact ? up.begin(c) : 0, u1 = R.nact ? up.begin(c + 1) : 0;
  const int64_t v0 = R.nact ? down.begin(c) : 0, v1 = R.nact ? down.begin(c + 1) : 0;

  if (warp == 0) {
    if (lane == 0) {
      int st = 0, issued = 0;
      uint32_t phase = 0;
      bool alive = true;
      auto acquire = [&]() {
        if (!mbar_wait(smem_addr(&C.empty[st]), phase ^ 1u, abort_flag, a.err, 710)) alive = false;
        return alive;
      };
      auto next = [&]() {
        ++issued;
        if (++st == nst) {
          st = 0;
          phase ^= 1u;
        }
      };
      for (int64_t u = u0; u < u1 && alive;) {
        const Seg s = up_seg(R, u, u1, FT, KU);
        for (int kb = s.kb0; kb < s.kb1 && acquire(); ++kb) {
          const uint32_t fb = smem_addr(&C.full[st]), sA = ring + st * slot;
          mbar_expect_tx(fb, 2 * TC_TILE + NT * 128);
          const int row = s.e * a.d + kb * TC_KB;
          tma_load_2d(sA, &maps.W1, fb, s.c0, row);
          tma_load_2d(sA + TC_TILE / 2, &maps.W1, fb, s.c0 + 64, row);
          tma_load_2d(sA + TC_TILE, &maps.W3, fb, s.c0, row);
          tma_load_2d(sA + TC_TILE + TC_TILE / 2, &maps.W3, fb, s.c0 + 64, row);
          tma_load_2d(sA + 2 * TC_TILE, &maps.x, fb, kb * TC_KB, 0);
          next();
        }
        u += s.kb1 - s.kb0;
      }
      auto load_w2 = [&](const Seg& s, int kb) {
        const uint32_t fb = smem_addr(&C.full[st]), sA = ring + st * slot;
        mbar_expect_tx(fb, TC_TILE + 2 * pad16(s.n) * 128);
        const int row = s.e * a.f + kb * TC_KB;
        tma_load_2d(sA, &maps.W2, fb, s.c0, row);
        tma_load_2d(sA + TC_TILE / 2, &maps.W2, fb, s.c0 + 64, row);
      };
      auto load_h = [&](const Seg& s, int kb, int stage) {
        const uint32_t fb = smem_addr(&C.full[stage]), sB = ring + stage * slot + TC_TILE;
        const int n16 = pad16(s.n);
        for (int r = 0; r < n16; r += 16) {
          tma_load_2d(sB + r * 128, &maps.h, fb, kb * TC_KB, s.base + r);
          tma_load_2d(sB + (n16 + r) * 128, &maps.h, fb, a.f + kb * TC_KB, s.base + r);
        }
      };
      // the ring full of W2 tiles, then the wait for every CTA's h, then their h tiles
      const int first = st;
      int ahead = 0;
      int64_t v = v0;
      for (; v < v1 && ahead < nst && alive; ++v, ++ahead) {
        if (!acquire()) break;
        const Seg s = down_seg(R, v, v1, per, KD);
        load_w2(s, s.kb0);
        next();
      }
      if (v0 < v1) {
        if (alive && !wait_count(a.ctr + 2 * G, G, a.err, 711)) {
          *abort_flag = 1;
          alive = false;
        }
        fence_async_all();
        int stage = first;
        for (int i = 0; i < ahead; ++i) {  // after a timeout too: every stage begun is completed
          const Seg s = down_seg(R, v0 + i, v1, per, KD);
          load_h(s, s.kb0, stage);
          if (++stage == nst) stage = 0;
        }
      }
      while (v < v1 && alive) {
        const Seg s = down_seg(R, v, v1, per, KD);
        for (int kb = s.kb0; kb < s.kb1 && acquire(); ++kb) {
          load_w2(s, kb);
          load_h(s, kb, st);
          next();
        }
        v += s.kb1 - s.kb0;
      }
      if (!alive) {  // wait for the copies in flight
        const int n = issued < nst ? issued : nst;
        int s = st;
        uint32_t ph = phase;
        for (int i = 0; i < n; ++i) {
          if (--s < 0) {
            s = nst - 1;
            ph ^= 1u;
          }
          for (uint32_t it = 0; it < (1u << 20) && !mbar_try_wait(smem_addr(&C.full[s]), ph); ++it) {
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int st = 0, seg = 0;
      uint32_t phase = 0;
      bool alive = true;
      auto advance = [&]() {
        umma_commit(smem_addr(&C.empty[st]));
        if (++st == nst) {
          st = 0;
          phase ^= 1u;
        }
      };
      auto open = [&]() {  // the segment's accumulator is free
        const uint32_t par = ((seg >> 1) & 1) ^ 1;
        if (!mbar_wait(smem_addr(&C.tempty[seg & 1]), par, abort_flag, a.err, 720)) alive = false;
        tc_fence_after();
        return alive;
      };
      auto filled = [&]() {
        if (!mbar_wait(smem_addr(&C.full[st]), phase, abort_flag, a.err, 721)) alive = false;
        tc_fence_after();
        return alive;
      };
      for (int64_t u = u0; u < u1 && open();) {
        const Seg s = up_seg(R, u, u1, FT, KU);
        const uint32_t acc = tmem + (seg & 1) * TC_BUF, id = dec_idesc(NT);
        for (int kb = s.kb0; kb < s.kb1 && filled(); ++kb) {
          const uint32_t sA = ring + st * slot, sB = sA + 2 * TC_TILE;
#pragma unroll
          for (int q = 0; q < TC_KB / 16; ++q) {
            const uint64_t bd = sdesc(sB + q * 32, 16, 1024);
            const uint32_t on = kb != s.kb0 || q != 0;
            umma_bf16(acc, sdesc(sA + q * 2048, 8192, 1024), bd, id, on);
            umma_bf16(acc + TC_B, sdesc(sA + TC_TILE + q * 2048, 8192, 1024), bd, id, on);
          }
          advance();
        }
        if (!alive) break;
        umma_commit(smem_addr(&C.tfull[seg & 1]));
        ++seg;
        u += s.kb1 - s.kb0;
      }
      for (int64_t v = v0; v < v1 && alive && open();) {
        const Seg s = down_seg(R, v, v1, per, KD);
        const int n16 = pad16(s.n);
        const uint32_t acc = tmem + (seg & 1) * TC_BUF, id = dec_idesc(n16);
        for (int kb = s.kb0; kb < s.kb1 && filled(); ++kb) {
          const uint32_t sA = ring + st * slot, sB = sA + TC_TILE;
#pragma unroll
          for (int q = 0; q < TC_KB / 16; ++q) {
            const uint64_t ad = sdesc(sA + q * 2048, 8192, 1024);
            umma_bf16(acc, ad, sdesc(sB + q * 32, 16, 1024), id, kb != s.kb0 || q != 0);
            umma_bf16(acc, ad, sdesc(sB + n16 * 128 + q * 32, 16, 1024), id, 1);
          }
          advance();
        }
        if (!alive) break;
        umma_commit(smem_addr(&C.tfull[seg & 1]));
        ++seg;
        v += s.kb1 - s.kb0;
      }
      umma_commit(smem_addr(&C.drain));
      for (uint32_t it = 0; it < (1u << 26) && !mbar_try_wait(smem_addr(&C.drain), 0); ++it) {
      }
    }
  } else if (warp >= 4) {
    const int q = warp - 4, tid = threadIdx.x - 128, col = tid;  // TMEM lanes q * 32 ..: the thread's weight column
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    int seg = 0;
    bool alive = true;
    auto ready = [&]() {
      alive = epi_all(mbar_wait(smem_addr(&C.tfull[seg & 1]), (seg >> 1) & 1, abort_flag, a.err, 730));
      tc_fence_after();
      return alive;
    };
    auto release = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_addr(&C.tempty[seg & 1]));
      ++seg;
    };
    auto signal = [&](uint32_t* ctr) {  // this CTA's part is written
      __threadfence();
      epi_sync();
      if (tid == 0) red_release(ctr);
    };
    auto wait_all = [&](const uint32_t* ctr, int want, uint32_t where) {
      const bool ok = tid != 0 || wait_count(ctr, want, a.err, where);
      if (!ok) *abort_flag = 1;
      alive = epi_all(ok);
      return alive;
    };

    // ---- up product ----
    __nv_bfloat16* h = static_cast<__nv_bfloat16*>(a.h);
    const int64_t pslot = (int64_t)a.T * 2 * DEC_N;
    int8_t* row_of = C.row_of[q];
    for (int64_t u = u0; u < u1 && ready();) {
      const Seg s = up_seg(R, u, u1, FT, KU);
      const bool whole = s.kb0 == 0 && s.kb1 == KU;
      float* part = a.up_part + ((int64_t)c * 2 + (s.kb0 > 0 ? 0 : 1)) * pslot + col;
      for (int t = lane; t < DEC_T; t += 32) row_of[t] = -1;
      __syncwarp();
      for (int m = lane; m < s.n; m += 32) row_of[R.tok[s.base + m]] = (int8_t)m;
      __syncwarp();
      for (int t0 = 0; t0 < NT; t0 += 16) {
        uint32_t ra[16], rb[16];
        const uint32_t at = tmem + lanes + (seg & 1) * TC_BUF + t0;
        tmem_ld16(at, ra);
        tmem_ld16(at + TC_B, rb);
        tmem_ld_wait16(ra);
        tmem_reg_fence16(rb);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int m = row_of[t0 + i];
          if (m < 0) continue;
          const float va = __uint_as_float(ra[i]), vb = __uint_as_float(rb[i]);
          if (whole) {
            put_h(h, s.base + m, a.f, s.c0 + col, R.gate[s.base + m] * dec_silu(va) * vb);
          } else {
            part[m * 2 * DEC_N] = va;
            part[m * 2 * DEC_N + DEC_N] = vb;
          }
        }
      }
      release();
      if (!whole) signal(a.ctr + up.owner(s.tile * KU));
      u += s.kb1 - s.kb0;
    }
    // a share of each tile that other CTAs have a part of
    for (int64_t u = u0; u < u1 && alive;) {
      const int64_t tile = u / KU, end = (tile + 1) * KU;
      const int first = up.owner(tile * KU), segs = up.owner(end - 1) - first + 1;
      if (segs > 1 && wait_all(a.ctr + first, segs, 731)) {
        const int e = R.act[tile / FT], c0 = (int)(tile % FT) * DEC_N, N = R.cnt[e] * DEC_N;
        const int i1 = (int)((int64_t)(c - first + 1) * N / segs);
        for (int i = (int)((int64_t)(c - first) * N / segs) + tid; i < i1; i += 128) {
          const int m = i / DEC_N, cc = i % DEC_N, row = R.base[e] + m;
          float va = 0.f, vb = 0.f;
#pragma unroll 4
          for (int g = 0; g < segs; ++g) {
            const float* p = a.up_part + ((int64_t)(first + g) * 2 + (g > 0 ? 0 : 1)) * pslot + m * 2 * DEC_N + cc;
            va += __ldcg(p);
            vb += __ldcg(p + DEC_N);
          }
          put_h(h, row, a.f, c0 + cc, R.gate[row] * dec_silu(va) * vb);
        }
      }
      u = end < u1 ? end : u1;
    }
    fence_async_all();  // h is read by the TMA
    if (alive) signal(a.ctr + 2 * G);

    // ---- down product ----
    const int64_t dslot = (int64_t)a.T * DEC_N;
    const __nv_bfloat16* res = static_cast<const __nv_bfloat16*>(a.io.residual);
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.io.y);
    auto put_y = [&](int t, int column, float v) {
      const int64_t o = (int64_t)t * a.d + column;
      y[o] = __float2bfloat16_rn(res ? v + __bfloat162float(res[o]) : v);
    };
    if (R.nact == 0) {  // every assignment was dropped
      for (int64_t i = (int64_t)c * 128 + tid; i < (int64_t)a.T * a.d; i += (int64_t)G * 128)
        put_y((int)(i / a.d), (int)(i % a.d), 0.f);
    }
    for (int t = 0; t < a.T; ++t) yacc[t * DEC_N + col] = 0.f;
    for (int64_t v = v0; v < v1 && alive && ready();) {
      const Seg s = down_seg(R, v, v1, per, KD);
      for (int m0 = 0; m0 < s.n; m0 += 16) {
        uint32_t r[16];
        tmem_ld16(tmem + lanes + (seg & 1) * TC_BUF + m0, r);
        tmem_ld_wait16(r);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (m0 + i < s.n) yacc[R.tok[s.base + m0 + i] * DEC_N + col] += __uint_as_float(r[i]);
      }
      release();
      v += s.kb1 - s.kb0;
      if (v == v1 || v == (s.tile + 1) * per) {  // the last of this column tile here
        const bool head = v0 > s.tile * per, whole = !head && v == (s.tile + 1) * per;
        float* part = a.down_part + ((int64_t)c * 2 + (head ? 0 : 1)) * dslot + col;
        for (int t = 0; t < a.T; ++t) {
          const float w = yacc[t * DEC_N + col];
          yacc[t * DEC_N + col] = 0.f;
          if (whole) put_y(t, s.c0 + col, w);
          else part[t * DEC_N] = w;
        }
        if (!whole) signal(a.ctr + G + down.owner(s.tile * per));
      }
    }
    for (int64_t v = v0; v < v1 && alive;) {
      const int64_t tile = v / per, end = (tile + 1) * per;
      const int first = down.owner(tile * per), segs = down.owner(end - 1) - first + 1;
      if (segs > 1 && wait_all(a.ctr + G + first, segs, 732)) {
        const int N = a.T * DEC_N, i1 = (int)((int64_t)(c - first + 1) * N / segs);
        for (int i = (int)((int64_t)(c - first) * N / segs) + tid; i < i1; i += 128) {
          float w = 0.f;
#pragma unroll 4
          for (int g = 0; g < segs; ++g)
            w += __ldcg(a.down_part + ((int64_t)(first + g) * 2 + (g > 0 ? 0 : 1)) * dslot + i);
          put_y(i / DEC_N, (int)tile * DEC_N + i % DEC_N, w);
        }
      }
      v = end < v1 ? end : v1;
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, TC_COLS);
}

PFN_cuTensorMapEncodeTiled_v12000 dec_encode = nullptr;

bool dec_encode_ready() {
  static bool tried = false;
  if (!tried) {
    tried = true;
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      dec_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  return dec_encode != nullptr;
}

// 2-D bf16 tensor map of dense rows, boxes of 64 columns, 128-byte swizzle.
bool dec_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return dec_encode(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_decode_tc(const Shape& s, const DecodeArgs& args, int G, cudaStream_t st) {
  if (!dec_encode_ready()) return cudaErrorNotSupported;
  DecodeArgs a = args;
  const uint32_t NT = (uint32_t)(s.T + 15) / 16 * 16;
  int slot = 2 * TC_TILE + (int)NT * 128;
  const int fixed = 1024 + (int)sizeof(Routing) + (int)sizeof(TcCtrl) + s.T * DEC_N * 4;
  int nst = (TC_SMEM_MAX - fixed) / slot;
  if (nst > TC_MAX_ST) nst = TC_MAX_ST;
  TcMapsD m;
  if (!dec_map(&m.x, a.io.x, s.T, s.d, NT) || !dec_map(&m.W1, a.io.W1, (uint64_t)s.E * s.d, s.f, 64) ||
      !dec_map(&m.W3, a.io.W3, (uint64_t)s.E * s.d, s.f, 64) || !dec_map(&m.W2, a.io.W2, (uint64_t)s.E * s.f, s.d, 64) ||
      !dec_map(&m.h, a.h, (uint64_t)s.T * s.k, 2 * (uint64_t)s.f, 16))
    return cudaErrorInvalidValue;
  static bool attr_done[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  if (!attr_done[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(decode_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, TC_SMEM_MAX);
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  void* params[] = {&m, &a, &nst, &slot};
  LaunchScope ls(KK_DECODE, st);
  return cudaLaunchCooperativeKernel((const void*)decode_tc_kernel, dim3(G), dim3(TC_NT), params,
                                     (size_t)(fixed + nst * slot), st);
}

}  // namespace moe
