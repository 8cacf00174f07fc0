// The whole layer for a few tokens in one kernel, bf16 weights on the tensor
// cores.  The steps and the split of the weights over the CTAs are those of
// decode.cu.
//
// The weights are the M side of the products: a tile of 128 columns of W1 and
// W3 (or W2) is the A operand, stored with its columns contiguous (MN-major),
// and the tokens are the N side, 16 to 64 columns of the accumulator (up to 128
// with both parts of h).  The MMAs of a 16 KB weight tile take a fifth of the
// time that HBM needs to deliver it to an SM, so the kernel is a stream of TMA
// loads with everything else behind:
//   warp 0, one lane: weights.  A stage of the up product is 64 rows of d of a
//     W1 and a W3 tile, one of the down product 64 or 128 rows of f of a W2
//     tile.
//   warp 2, one lane: the tokens' side of the same stages, the columns of all
//     tokens of x, then those of the expert's rows of h.  Where rows are few
//     (few_rows) warps 2, 3, 8 and 9 make the rows of h themselves, from the
//     partial sums of the up product.
//   warp 1: MMAs.  Two accumulators in turn, so the next segment's products run
//     under a segment's epilogue.
//   warps 4-7: epilogue, one weight column a thread.
// Both products are done in two halves of f, in the order up 0, up 1, down 0,
// down 1: the exchange of the partial sums of one half and the grid barrier
// behind its h (5 to 10 us: fences and atomics queue behind the stream) run
// under the stream of the next part's weights.
// h is split into two bf16 parts, hi + lo, side by side in the N dimension: 16
// significant bits where one bf16 would round h to 8 and double the square of
// y's error.  The second product is free here: an MMA of this shape is bound by
// reading its 4 KB of A.
// The weights are loaded with an evict-first policy, so that code, tokens and
// partial sums stay in L2 (64 tokens of the dropless layer below: 147 us, and
// 151.5 without).
// Measured, inputs from HBM: one token of a layer with d 4096, f 1536, 32
// experts, top-4 (151 MB of weights) 39 us, 64 tokens of it (680 to 780 MB) 143
// to 155; the stream itself runs at 6 to 7 TB/s, and 17 us are routing, launch
// and the ends of the two products.
#include <cudaTypedefs.h>

#include "decode.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

constexpr int TC_NT = 320;
constexpr int TC_KB = 64;                 // rows of a unit: 128 bytes of a token's row
constexpr int TC_TILE = DEC_N * TC_KB * 2;  // 16 KB: two boxes of 64 columns x 64 rows
constexpr int TC_MAX_ST = 8;
constexpr int TC_SLOT = 2 * TC_TILE + 8192;  // and 64 tokens of x, or two units' hi and lo of 16 rows of h
constexpr int TC_QUEUE = 6;  // units of weights on their way to an SM, 96 KB
constexpr int TC_SMEM_MAX = 232448;       // 227 KB a CTA
constexpr uint32_t TC_COLS = 256;         // TMEM: two accumulators of a and b, 64 tokens each
constexpr uint32_t TC_BUF = 128, TC_B = 64;

struct alignas(16) TcCtrl {
  uint64_t wfull[TC_MAX_ST], bfull[TC_MAX_ST], empty[TC_MAX_ST], tfull[2], tempty[2], drain;
  uint32_t tmem;
  int abort;
};

struct TcMapsD {
  CUtensorMap x, W1, W3, W2;
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
  int ai, e, n, base, block;  // place in the list, expert, its rows, the first of them, its first block of rows of h
  int c0;          // first weight column
  int kb0, kb1;    // units
  int tile;        // up: the weight tile; down: the column tile of y
};
// half: 0 or 1, FT and KD are those of a half
__device__ __forceinline__ Seg up_seg(const Routing& R, int u, int u1, int half, int FT, int KU) {
  Seg s;
  s.tile = u / KU;
  s.kb0 = u - s.tile * KU;
  s.kb1 = u1 - s.tile * KU < KU ? u1 - s.tile * KU : KU;
  const int ai = s.tile / FT;
  s.ai = ai;
  s.e = R.act[ai];
  s.c0 = (half * FT + s.tile - ai * FT) * DEC_N;
  s.n = R.cnt[s.e];
  s.base = R.base[s.e];
  s.block = R.block[s.e];
  return s;
}
__device__ __forceinline__ Seg down_seg(const Routing& R, int u, int u1, int half, int per, int KD) {
  Seg s;
  s.tile = u / per;
  const int q = u - s.tile * per, ai = q / KD;
  s.kb0 = q - ai * KD;
  s.kb1 = u1 - u < KD - s.kb0 ? s.kb0 + u1 - u : KD;
  s.kb0 += half * KD;
  s.kb1 += half * KD;
  s.ai = ai;
  s.e = R.act[ai];
  s.c0 = s.tile * DEC_N;
  s.n = R.cnt[s.e];
  s.base = R.base[s.e];
  s.block = R.block[s.e];
  return s;
}
// A 128-column weight tile: two boxes of 64 columns.
__device__ __forceinline__ void load_weights(uint32_t dst, const CUtensorMap* map, uint32_t bar, int row, int chunk,
                                             uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(row), "r"(chunk), "l"(policy)
      : "memory");
}
// bytes, a multiple of 16, between 16-byte boundaries
__device__ __forceinline__ void load_bytes(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
// tcgen05.mma and its commit by one lane of a converged warp
__device__ __forceinline__ void umma_elected(uint32_t d, uint64_t ad, uint64_t bd, uint32_t id, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(id), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit_elected(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "elect.sync _|q, 0xffffffff;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
      : "memory");
}
// wait, the call only where the phase is not complete yet
__device__ __forceinline__ bool ring_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t* err,
                                          uint32_t where) {
  return mbar_try_wait(smem_addr(bar), parity) || mbar_wait(smem_addr(bar), parity, abort_flag, err, where);
}
__device__ __forceinline__ int pad16(int n) { return (n + 15) & ~15; }
// units of a stage of the down product: two where the rows are few enough for both to fit
__device__ __forceinline__ int down_units(const Seg& s, int kb) { return s.n <= 16 && kb + 1 < s.kb1 ? 2 : 1; }

// a and b of one token, four consecutive rows of y
__device__ __forceinline__ float2 tmem_ld_ab(uint32_t at) {
  float2 v;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%2];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%1}, [%3];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&f"(v.x), "=&f"(v.y)
      : "r"(at), "r"(at + TC_B)
      : "memory");
  return v;
}
// four columns and the four `lo` columns behind them, added
__device__ __forceinline__ float4 tmem_ld4_sum(uint32_t at, int lo) {
  float4 v, w;
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%8];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x4.b32 {%4, %5, %6, %7}, [%9];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=&f"(v.x), "=&f"(v.y), "=&f"(v.z), "=&f"(v.w), "=&f"(w.x), "=&f"(w.y), "=&f"(w.z), "=&f"(w.w)
      : "r"(at), "r"(at + lo)
      : "memory");
  return make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
}
__device__ __forceinline__ void add4(float4& v, const float4& w) {
  v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
}
__device__ __forceinline__ void xor4(float4& v, int o) {
  add4(v, make_float4(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o),
                      __shfl_xor_sync(0xffffffffu, v.z, o), __shfl_xor_sync(0xffffffffu, v.w, o)));
}
// The fast divide and exponential, whose documented errors, 2 ulp and 2 + |1.173 z|,
// are about 2^-20 of the result at z = -5 and 2^-17 at z = -64: h is held in 16 bits, and
// where the error comes near those silu(z) is below 2^-80.
__device__ __forceinline__ float silu_bf16(float z) { return __fdividef(z, 1.f + __expf(-z)); }
// h is kept as the down product reads it: for every 64 columns an expert's
// blocks of 16 rows, [hi rows | lo rows] of 128 bytes in the 128-byte swizzle
// of the MMA operand, so one plain copy brings a unit's rows.
__device__ __forceinline__ char* h_at(const DecodeArgs& a, int blocks, const Seg& s, int m, int col) {
  const int64_t tile = (int64_t)(col / 64) * blocks + s.block;
  return static_cast<char*>(a.h) + tile * 4096 + m * 128 + ((((col % 64) / 8) ^ (m & 7)) << 4) + (col % 8) * 2;
}
__device__ __forceinline__ float lo_part(float v, float hi) {
  const float r = v - hi;
  return isfinite(r) ? r : 0.f;  // the hi of an infinite v carries it alone
}
__device__ __forceinline__ void put_h(char* p, int n16, float v) {
  const __nv_bfloat16 hi = __float2bfloat16_rn(v);
  *reinterpret_cast<__nv_bfloat16*>(p) = hi;
  *reinterpret_cast<__nv_bfloat16*>(p + n16 * 128) = __float2bfloat16_rn(lo_part(v, __bfloat162float(hi)));
}
__device__ __forceinline__ void split4(const float4& v, __nv_bfloat162 (&hi)[2], __nv_bfloat162 (&lo)[2]) {
  hi[0] = __floats2bfloat162_rn(v.x, v.y);
  hi[1] = __floats2bfloat162_rn(v.z, v.w);
  const float2 p = __bfloat1622float2(hi[0]), q = __bfloat1622float2(hi[1]);
  lo[0] = __floats2bfloat162_rn(lo_part(v.x, p.x), lo_part(v.y, p.y));
  lo[1] = __floats2bfloat162_rn(lo_part(v.z, q.x), lo_part(v.w, q.y));
}
__device__ __forceinline__ void put_h4(char* p, int n16, const float4& v) {
  __nv_bfloat162 hi[2], lo[2];
  split4(v, hi, lo);
  *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(hi);
  *reinterpret_cast<uint2*>(p + n16 * 128) = *reinterpret_cast<const uint2*>(lo);
}

__device__ __forceinline__ float4 swiglu4(float gate, const float4& a, const float4& b) {
  return make_float4(gate * silu_bf16(a.x) * b.x, gate * silu_bf16(a.y) * b.y, gate * silu_bf16(a.z) * b.z,
                     gate * silu_bf16(a.w) * b.w);
}
// The parts of a split tile: the first CTA's is its second, the others' are
// their first, counted from the first CTA's second.
__device__ __forceinline__ int part_at(int g) { return g == 0 ? 0 : g * 2 - 1; }
// item j of a tile: four columns of a row
__device__ __forceinline__ int item_at(int j) { return j / (DEC_N / 4) * 2 * DEC_N + j % (DEC_N / 4) * 4; }
__device__ __forceinline__ void load_ab(const float* p, float4& a, float4& b) {
  a = __ldcg(reinterpret_cast<const float4*>(p));
  b = __ldcg(reinterpret_cast<const float4*>(p + DEC_N));
}
// a and b of row `row` and columns c0.. (a whole tile's)
__device__ __forceinline__ float* up_whole(const DecodeArgs& a, int row, int c0) {
  return a.up_whole + (int64_t)row * a.f * 2 + c0 * 2;
}

// After a wait that gave up: the copies in flight land within this time.
__device__ __noinline__ void settle() {
  const uint64_t t0 = dec_now();
  while (dec_now() - t0 < 5000000ull) {
  }
}

__global__ void __launch_bounds__(TC_NT, 1) decode_tc_kernel(const __grid_constant__ TcMapsD maps,
                                                             const __grid_constant__ DecodeArgs a, int nst, int blocks) {
  constexpr int slot = TC_SLOT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Routing& R = *reinterpret_cast<Routing*>(smem + nst * slot);
  TcCtrl& C = *reinterpret_cast<TcCtrl*>(smem + nst * slot + sizeof(Routing));
  float* yacc = reinterpret_cast<float*>(smem + nst * slot + sizeof(Routing) + sizeof(TcCtrl));  // [T][DEC_N]
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile int* abort_flag = &C.abort;

  if (threadIdx.x == 0) {
    for (int i = 0; i < nst; ++i) {
      mbar_init(smem_addr(&C.wfull[i]), 1);
      mbar_init(smem_addr(&C.bfull[i]), 1);
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
  const int FT = a.f / DEC_N / 2, DT = a.d / DEC_N, KU = a.d / TC_KB, KD = a.f / TC_KB / 2;  // FT, KD: of a half of f
  const int NT = pad16(a.T);
  const int per = R.nact * KD;  // units of a column tile of y: all experts' rows of W2
  const Split up(R.nact * FT * KU, G), down(per * DT, G);
  const int u0 = up.begin(c), u1 = up.begin(c + 1), v0 = down.begin(c), v1 = down.begin(c + 1);
  uint32_t* bar = a.ctr + 2 * G;  // h of half 0, of half 1, the partial sums of y
  const int64_t dslot = (int64_t)a.T * DEC_N, pslot = (int64_t)a.T * 2 * DEC_N;
  const bool direct = few_rows(a, R);

  if (warp == 0) {
    // ---- weights ----
    if (lane == 0) {
      const uint64_t once = l2_evict_first_policy();
      int st = 0, oldest = 0, stages = 0, queued = 0;
      uint32_t phase = 0, oldest_phase = 0, sizes = 0;  // sizes: units of the stages on their way, 4 bits each
      bool alive = true;
      // At most TC_QUEUE units of weights are on their way: more only lengthen
      // HBM's queue, and with it the latency of every fence and atomic.
      auto arrived = [&]() {
        queued -= sizes & 15;
        sizes >>= 4;
        --stages;
        if (++oldest == nst) {
          oldest = 0;
          oldest_phase ^= 1u;
        }
      };
      auto open = [&](int units) {
        while (stages > 0 && queued + units > TC_QUEUE) {
          if (!ring_wait(&C.wfull[oldest], oldest_phase, abort_flag, a.err, 712)) return alive = false;
          arrived();
        }
        if (!ring_wait(&C.empty[st], phase ^ 1u, abort_flag, a.err, 710)) return alive = false;
        if (stages == nst) arrived();  // this slot's last, which has been read
        mbar_expect_tx(smem_addr(&C.wfull[st]), units * TC_TILE);
        sizes |= (uint32_t)units << (4 * stages++);
        queued += units;
        return true;
      };
      auto next = [&]() {
        if (++st == nst) {
          st = 0;
          phase ^= 1u;
        }
      };
#pragma unroll 1
      for (int half = 0; half < 2; ++half)
        for (int u = u0; u < u1 && alive;) {
          const Seg s = up_seg(R, u, u1, half, FT, KU);
          int row = s.e * a.d + s.kb0 * TC_KB;
#pragma unroll 1
          for (int kb = s.kb0; kb < s.kb1 && open(2); ++kb, row += TC_KB) {
            const uint32_t fb = smem_addr(&C.wfull[st]), sA = ring + st * slot;
            load_weights(sA, &maps.W1, fb, row, s.c0 / 64, once);
            load_weights(sA + TC_TILE, &maps.W3, fb, row, s.c0 / 64, once);
            next();
          }
          u += s.kb1 - s.kb0;
        }
#pragma unroll 1
      for (int half = 0; half < 2; ++half)
        for (int v = v0; v < v1 && alive;) {
          const Seg s = down_seg(R, v, v1, half, per, KD);
          int row = s.e * a.f + s.kb0 * TC_KB;
#pragma unroll 1
          for (int kb = s.kb0; kb < s.kb1;) {
            const int nk = down_units(s, kb);
            if (!open(nk)) break;
            const uint32_t fb = smem_addr(&C.wfull[st]), sA = ring + st * slot;
            load_weights(sA, &maps.W2, fb, row, s.c0 / 64, once);
            if (nk == 2) load_weights(sA + TC_TILE, &maps.W2, fb, row + TC_KB, s.c0 / 64, once);
            next();
            kb += nk;
            row += nk * TC_KB;
          }
          v += s.kb1 - s.kb0;
        }
      if (!alive) settle();
    }
  } else if (warp == 2 && !direct) {
    // ---- tokens: x, then h ----
    if (lane == 0) {
      int st = 0;
      uint32_t phase = 0;
      bool alive = true;
      auto open = [&](int bytes) {
        if (!ring_wait(&C.empty[st], phase ^ 1u, abort_flag, a.err, 713)) return alive = false;
        mbar_expect_tx(smem_addr(&C.bfull[st]), bytes);
        return true;
      };
      auto next = [&]() {
        if (++st == nst) {
          st = 0;
          phase ^= 1u;
        }
      };
#pragma unroll 1
      for (int half = 0; half < 2; ++half)
        for (int u = u0; u < u1 && alive;) {
          const Seg s = up_seg(R, u, u1, half, FT, KU);
#pragma unroll 1
          for (int kb = s.kb0; kb < s.kb1 && open(NT * 128); ++kb) {
            tma_load_2d(ring + st * slot + 2 * TC_TILE, &maps.x, smem_addr(&C.bfull[st]), kb * TC_KB, 0);
            next();
          }
          u += s.kb1 - s.kb0;
        }
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        if (v0 < v1 && alive && !wait_count(bar + half, G, a.err, 711)) {
          *abort_flag = 1;
          alive = false;
        }
        fence_async_all();  // the other CTAs' h is read by copies
        for (int v = v0; v < v1 && alive;) {
          const Seg s = down_seg(R, v, v1, half, per, KD);
          const uint32_t bytes = pad16(s.n) * 256;
          const char* src = static_cast<const char*>(a.h) + ((int64_t)s.kb0 * blocks + s.block) * 4096;
#pragma unroll 1
          for (int kb = s.kb0; kb < s.kb1;) {
            const int nk = down_units(s, kb);
            if (!open(nk * bytes)) break;
            const uint32_t fb = smem_addr(&C.bfull[st]), sB = ring + st * slot + nk * TC_TILE;
            load_bytes(sB, src, bytes, fb);
            if (nk == 2) load_bytes(sB + bytes, src + (int64_t)blocks * 4096, bytes, fb);
            next();
            kb += nk;
            src += (int64_t)nk * blocks * 4096;
          }
          v += s.kb1 - s.kb0;
        }
      }
      if (!alive) settle();
    }
  } else if (direct && (warp == 2 || warp == 3 || warp >= 8)) {
    // ---- tokens of few rows: x as above, then h from the partial sums; the four warps take stages in turn ----
    int st = 0, turn = (warp & 1) + (warp >= 8 ? 2 : 0);  // 0: this warp's
    uint32_t phase = 0;
    bool alive = true;
    auto next = [&]() {
      turn = (turn + 1) & 3;
      if (++st == nst) {
        st = 0;
        phase ^= 1u;
      }
    };
    auto open = [&]() {
      const bool ok = ring_wait(&C.empty[st], phase ^ 1u, abort_flag, a.err, 714);
      return alive = __all_sync(0xffffffffu, ok);
    };
#pragma unroll 1
    for (int half = 0; half < 2; ++half)
      for (int u = u0; u < u1 && alive;) {
        const Seg s = up_seg(R, u, u1, half, FT, KU);
#pragma unroll 1
        for (int kb = s.kb0; kb < s.kb1; ++kb) {
          if (turn == 0) {
            if (!open()) break;
            if (lane == 0) {
              mbar_expect_tx(smem_addr(&C.bfull[st]), NT * 128);
              tma_load_2d(ring + st * slot + 2 * TC_TILE, &maps.x, smem_addr(&C.bfull[st]), kb * TC_KB, 0);
            }
          }
          next();
        }
        u += s.kb1 - s.kb0;
      }
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      const float* parts = a.up_part + (int64_t)half * G * 2 * pslot;
      if (v0 < v1 && alive) {
        const bool ok = lane != 0 || wait_count(bar + half, G, a.err, 715);
        alive = __all_sync(0xffffffffu, ok);
        __syncwarp();  // a vote orders no memory: lane 0 has acquired the other CTAs' sums, all lanes read them
        if (!alive) *abort_flag = 1;
      }
      for (int v = v0; v < v1 && alive;) {
        const Seg s = down_seg(R, v, v1, half, per, KD);
        const int n16 = pad16(s.n);
#pragma unroll 1
        for (int kb = s.kb0; kb < s.kb1;) {
          const int nk = down_units(s, kb);
          if (turn == 0) {
            if (!open()) break;
            char* sB = reinterpret_cast<char*>(smem + st * slot + nk * TC_TILE);
#pragma unroll 1
            for (int i = lane; i < nk * s.n * (TC_KB / 4); i += 32) {
              const int r = i / (TC_KB / 4), m = r % s.n, q = r / s.n;  // row m of unit q, four columns
              const int at = i % (TC_KB / 4) * 4, col = (kb + q) * TC_KB + at;
              const int tile = s.ai * FT + col / DEC_N - half * FT;
              const int first = up.owner(tile * KU), segs = up.owner(tile * KU + KU - 1) - first + 1;
              const float* p = segs == 1 ? up_whole(a, s.base + m, col / DEC_N * DEC_N) + col % DEC_N
                                         : parts + ((int64_t)first * 2 + 1) * pslot + m * 2 * DEC_N + col % DEC_N;
              float4 va = make_float4(0.f, 0.f, 0.f, 0.f), vb = va;
#pragma unroll 1
              for (int g0 = 0; g0 < segs; g0 += 8) {
                float4 x[8], z[8];
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                  x[g] = z[g] = make_float4(0.f, 0.f, 0.f, 0.f);
                  if (g0 + g < segs) load_ab(p + part_at(g0 + g) * pslot, x[g], z[g]);
                }
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                  add4(va, x[g]);
                  add4(vb, z[g]);
                }
              }
              put_h4(sB + q * n16 * 256 + m * 128 + (((at / 8) ^ (m & 7)) << 4) + at % 8 * 2, n16,
                     swiglu4(R.gate[s.base + m], va, vb));
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&C.bfull[st]));
          }
          next();
          kb += nk;
        }
        v += s.kb1 - s.kb0;
      }
    }
    if (!alive) settle();
  } else if (warp == 1) {
    // ---- MMAs: the whole warp walks the stages, so descriptors stay in uniform registers; one lane issues ----
    int st = 0, seg = 0;
    uint32_t phase = 0;
    bool alive = true;
    auto wait = [&](uint64_t* b, uint32_t parity, uint32_t where) {
      return __all_sync(0xffffffffu, ring_wait(b, parity, abort_flag, a.err, where));
    };
    auto advance = [&]() {
      commit_elected(smem_addr(&C.empty[st]));
      if (++st == nst) {
        st = 0;
        phase ^= 1u;
      }
    };
    auto open = [&]() {  // the segment's accumulator is free
      alive = wait(&C.tempty[seg & 1], ((seg >> 1) & 1) ^ 1, 720);
      tc_fence_after();
      return alive;
    };
    auto filled = [&]() {
      alive = wait(&C.wfull[st], phase, 721) && wait(&C.bfull[st], phase, 722);
      tc_fence_after();
      return alive;
    };
#pragma unroll 1
    for (int half = 0; half < 2; ++half)
      for (int u = u0; u < u1 && alive && open();) {
        const Seg s = up_seg(R, u, u1, half, FT, KU);
        const uint32_t acc = tmem + (seg & 1) * TC_BUF, id = dec_idesc(NT);
#pragma unroll 1
        for (int kb = s.kb0; kb < s.kb1 && filled(); ++kb) {
          // descriptors of the following K steps differ in the address alone (in 16-byte units)
          const uint64_t ad = sdesc(ring + st * slot, 8192, 1024), bd = sdesc(ring + st * slot + 2 * TC_TILE, 16, 1024);
#pragma unroll
          for (int q = 0; q < TC_KB / 16; ++q) {
            const uint32_t on = q != 0 || kb != s.kb0;
            umma_elected(acc, ad + q * (2048 / 16), bd + q * (32 / 16), id, on);
            umma_elected(acc + TC_B, ad + TC_TILE / 16 + q * (2048 / 16), bd + q * (32 / 16), id, on);
          }
          advance();
        }
        if (!alive) break;
        commit_elected(smem_addr(&C.tfull[seg & 1]));
        ++seg;
        u += s.kb1 - s.kb0;
      }
#pragma unroll 1
    for (int half = 0; half < 2; ++half)
      for (int v = v0; v < v1 && alive && open();) {
        const Seg s = down_seg(R, v, v1, half, per, KD);
        const int n16 = pad16(s.n);
        const uint32_t acc = tmem + (seg & 1) * TC_BUF, id = dec_idesc(2 * n16);
#pragma unroll 1
        for (int kb = s.kb0; kb < s.kb1 && filled();) {
          const int nk = down_units(s, kb);
          uint64_t ad = sdesc(ring + st * slot, 8192, 1024), bd = sdesc(ring + st * slot + nk * TC_TILE, 16, 1024);
#pragma unroll 1
          for (int i = 0; i < nk; ++i, ad += TC_TILE / 16, bd += 2 * n16 * 128 / 16) {
#pragma unroll
            for (int q = 0; q < TC_KB / 16; ++q)
              umma_elected(acc, ad + q * (2048 / 16), bd + q * (32 / 16), id, q != 0 || i != 0 || kb != s.kb0);
          }
          advance();
          kb += nk;
        }
        if (!alive) break;
        commit_elected(smem_addr(&C.tfull[seg & 1]));
        ++seg;
        v += s.kb1 - s.kb0;
      }
    commit_elected(smem_addr(&C.drain));
    for (uint32_t it = 0; it < (1u << 26) && !mbar_try_wait(smem_addr(&C.drain), 0); ++it) {
    }
  } else if (warp >= 4 && warp < 8) {
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
    for (int half = 0; half < 2 && alive; ++half) {
      float* parts = a.up_part + (int64_t)half * G * 2 * pslot;
      uint32_t* ctr = a.ctr + half * G;
      for (int u = u0; u < u1 && ready();) {
        const Seg s = up_seg(R, u, u1, half, FT, KU);
        const bool whole = s.kb0 == 0 && s.kb1 == KU;
        float* part = whole ? up_whole(a, s.base, s.c0) : parts + ((int64_t)c * 2 + (s.kb0 > 0 ? 0 : 1)) * pslot;
        const int64_t step = whole ? (int64_t)a.f * 2 : 2 * DEC_N;
#pragma unroll 1
        for (int m = 0; m < s.n; ++m) {  // the row's token is its column
          const int row = s.base + m;
          const float2 v = tmem_ld_ab(tmem + lanes + (seg & 1) * TC_BUF + R.tok[row]);
          if (whole && !direct) {
            put_h(h_at(a, blocks, s, m, s.c0 + col), pad16(s.n), R.gate[row] * silu_bf16(v.x) * v.y);
          } else {
            part[m * step + col] = v.x;
            part[m * step + col + DEC_N] = v.y;
          }
        }
        release();
        if (!whole && !direct) signal(ctr + up.owner(s.tile * KU));
        u += s.kb1 - s.kb0;
      }
      // a share of each tile that other CTAs have a part of
      for (int u = u0; u < u1 && alive && !direct;) {
        const int tile = u / KU, end = (tile + 1) * KU;
        const int first = up.owner(tile * KU), segs = up.owner(end - 1) - first + 1;
        if (segs > 1 && wait_all(ctr + first, segs, 731)) {
          const Seg s = up_seg(R, tile * KU, end, half, FT, KU);
          const float* p0 = parts + ((int64_t)first * 2 + 1) * pslot;
          const int N4 = s.n * (DEC_N / 4), j0 = (c - first) * N4 / segs, j1 = (c - first + 1) * N4 / segs;
          // four columns to `L` threads, each some of the parts; two such items at once
          int L = 8;
          while (L > 1 && (j1 - j0) * L > 128) L /= 2;
          const int sub = tid % L;
#pragma unroll 1
          for (int jb = j0 + tid / L; jb - tid / L < j1; jb += 256 / L) {
            float4 va[2], vb[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) va[i] = vb[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int g0 = sub; g0 < segs; g0 += 2 * L) {
              float4 x[4], z[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int g = g0 + (i & 1) * L, j = jb + (i >> 1) * (128 / L);
                x[i] = z[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (g < segs && j < j1) load_ab(p0 + part_at(g) * pslot + item_at(j), x[i], z[i]);
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                add4(va[i >> 1], x[i]);
                add4(vb[i >> 1], z[i]);
              }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll 1
              for (int o = 1; o < L; o *= 2) {
                xor4(va[i], o);
                xor4(vb[i], o);
              }
              const int j = jb + i * (128 / L), m = j / (DEC_N / 4), cc = j % (DEC_N / 4) * 4;
              if (sub == 0 && j < j1) put_h4(h_at(a, blocks, s, m, s.c0 + cc), pad16(s.n), swiglu4(R.gate[s.base + m], va[i], vb[i]));
            }
          }
        }
        u = end < u1 ? end : u1;
      }
      fence_async_all();  // h is read by the TMA
      if (alive) signal(bar + half);
    }

    // ---- down product ----
    for (int t = 0; t < a.T; ++t) yacc[t * DEC_N + col] = 0.f;
    for (int half = 0; half < 2; ++half)
      for (int v = v0; v < v1 && alive && ready();) {
        const Seg s = down_seg(R, v, v1, half, per, KD);
#pragma unroll 1
        for (int m0 = 0; m0 < s.n; m0 += 4) {
          const float4 r = tmem_ld4_sum(tmem + lanes + (seg & 1) * TC_BUF + m0, pad16(s.n));
          const uint8_t* tok = R.tok + s.base + m0;
          yacc[tok[0] * DEC_N + col] += r.x;
          if (m0 + 1 < s.n) yacc[tok[1] * DEC_N + col] += r.y;
          if (m0 + 2 < s.n) yacc[tok[2] * DEC_N + col] += r.z;
          if (m0 + 3 < s.n) yacc[tok[3] * DEC_N + col] += r.w;
        }
        release();
        v += s.kb1 - s.kb0;
        if (v == v1 || v == (s.tile + 1) * per) {  // the last of this column tile here
          float* part = a.down_part + ((int64_t)half * (G + DT) + c + s.tile) * dslot + col;
#pragma unroll 4
          for (int t = 0; t < a.T; ++t) {
            part[t * DEC_N] = yacc[t * DEC_N + col];
            yacc[t * DEC_N + col] = 0.f;
          }
        }
      }
    if (alive) signal(bar + 2);
    if (alive) wait_all(bar + 2, G, 732);
    if (!alive) *abort_flag = 1;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, TC_COLS);
  if (*abort_flag) return;

  // ---- y: the sums of a column tile's CTAs, half 0 and then half 1; `L` threads
  // take every L-th of them for four columns ----
  const __nv_bfloat16* res = static_cast<const __nv_bfloat16*>(a.io.residual);
  __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.io.y);
  const int64_t items = (int64_t)a.T * a.d / 4;
  const int i0 = (int)(c * items / G), i1 = (int)((c + 1) * items / G);
  const int L = i1 - i0 <= TC_NT / 8 ? 8 : 1, sub = threadIdx.x % L;
#pragma unroll 1
  for (int ib = i0; ib < i1; ib += TC_NT / L) {
    const int i = ib + threadIdx.x / L;
    const bool on = i < i1;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    const int t = i / (a.d / 4), col = (i - t * (a.d / 4)) * 4;
    const int64_t o = (int64_t)t * a.d + col;
    uint2 u = make_uint2(0, 0);
    if (on && sub == 0 && res) u = *reinterpret_cast<const uint2*>(res + o);
    if (on && R.nact > 0) {
      const int dt = col / DEC_N, first = down.owner(dt * per), n = down.owner((dt + 1) * per - 1) - first + 1;
      const float* p = a.down_part + (int64_t)(first + dt) * dslot + t * DEC_N + col % DEC_N;
#pragma unroll 1
      for (int g0 = sub; g0 < 2 * n; g0 += 8 * L) {
        float4 w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int g = g0 + j * L;
          w[j] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (g < 2 * n) w[j] = __ldcg(reinterpret_cast<const float4*>(p + (int64_t)(g < n ? g : G + DT + g - n) * dslot));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) add4(v, w[j]);
      }
    }
#pragma unroll 1
    for (int o = 1; o < L; o *= 2) xor4(v, o);
    if (on && sub == 0) {
      if (res) {
        const float2 r0 = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(u.x));
        const float2 r1 = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(u.y));
        v = make_float4(v.x + r0.x, v.y + r0.y, v.z + r1.x, v.w + r1.y);
      }
      __nv_bfloat162 w[2] = {__floats2bfloat162_rn(v.x, v.y), __floats2bfloat162_rn(v.z, v.w)};
      *reinterpret_cast<uint2*>(y + o) = *reinterpret_cast<const uint2*>(w);
    }
  }
}

// Looked up once; a thread that comes meanwhile waits for it.
PFN_cuTensorMapEncodeTiled_v12000 dec_encode() {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q{};
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) ==
                        cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ok ? fn : nullptr);
  }();
  return encode;
}

// bf16 rows in boxes of 64 columns, 128-byte swizzle: x as [rows][cols], weights
// as [cols / 64][rows][64] with two neighbouring chunks of columns to a box.
bool dec_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows, bool weights) {
  cuuint64_t dims[3] = {weights ? 64 : cols, rows, cols / 64};
  cuuint64_t strides[2] = {cols * 2, 128};
  cuuint32_t box[3] = {64, box_rows, 2};
  cuuint32_t estr[3] = {1, 1, 1};
  return dec_encode()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, weights ? 3 : 2, const_cast<void*>(base), dims, strides, box,
                    estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Most blocks of 16 rows of h: every expert with rows begins one.
int h_blocks(const Shape& s) {
  const int Tk = s.T * s.k, experts = s.E < Tk ? s.E : Tk;
  return (Tk + 15 * experts) / 16;
}

}  // namespace

size_t decode_tc_whole_bytes(const Shape& s) {
  return s.T * s.k <= DEC_DIRECT ? (size_t)s.T * s.k * s.f * 8 : 0;
}
size_t decode_tc_h_bytes(const Shape& s) { return (size_t)(s.f / 64) * h_blocks(s) * 4096; }

cudaError_t launch_decode_tc(const Shape& s, const DecodeArgs& args, int G, cudaStream_t st) {
  if (dec_encode() == nullptr) return cudaErrorNotSupported;
  DecodeArgs a = args;
  const uint32_t NT = (uint32_t)(s.T + 15) / 16 * 16;
  const int fixed = 1024 + (int)sizeof(Routing) + (int)sizeof(TcCtrl) + s.T * DEC_N * 4;
  int nst = (TC_SMEM_MAX - fixed) / TC_SLOT, blocks = h_blocks(s);
  if (nst > TC_MAX_ST) nst = TC_MAX_ST;
  TcMapsD m;
  if (!dec_map(&m.x, a.io.x, s.T, s.d, NT, false) || !dec_map(&m.W1, a.io.W1, (uint64_t)s.E * s.d, s.f, 64, true) ||
      !dec_map(&m.W3, a.io.W3, (uint64_t)s.E * s.d, s.f, 64, true) ||
      !dec_map(&m.W2, a.io.W2, (uint64_t)s.E * s.f, s.d, 64, true))
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
  void* params[] = {&m, &a, &nst, &blocks};
  LaunchScope ls(KK_DECODE, st);
  return cudaLaunchCooperativeKernel((const void*)decode_tc_kernel, dim3(G), dim3(TC_NT), params,
                                     (size_t)(fixed + nst * TC_SLOT), st);
}

}  // namespace moe
