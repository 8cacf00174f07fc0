// The vocabulary loss of at most 64 bf16 or 48 float32 tokens, as a serving step scores them.
//
// The weights are read once and bound it.  They are the M side of the MMAs (128
// words), the tokens the 16, 32 or 64 columns, so few tokens cost few MMA cycles:
// with tokens as rows of 256 the zeros around them take as long as the weights
// (one token, 128000 x 4096: 196 us; this form 169, 6.2 TB/s).  Each CTA takes an equal,
// contiguous range of words, in tiles of 128 and a last one of what is left, 32
// words a copy.  A thread has one word of a tile and keeps each token's maximum
// and sum of exponentials over its words in registers; the CTA's threads join
// theirs at the end, and a second kernel the CTAs'.
//
// Sums over K of 256 at a time are added up in TMEM, where they are cut off, and
// then, rounded, in registers.  Longer ones lean to 0: the loss of one token that has
// learned its label, 4096 x 128000, is 8e-8 off (root mean square, 6e-8 of products
// in fp32), 1.4e-7 with K of 512, 2.8e-7 with the 1024 of many tokens' products;
// shorter ones cost more than they give (K of 128: 6e-8, 177 us for 173, 190 for 182
// at 64 tokens; K of 1024: 171 and 180).
//
// Few float32 tokens take no tensor core: W's parts would have to be written and
// read again, 12 bytes for each 4.  Groups of 8 tokens, or of fewer where more do
// not fit in shared memory, have an equal share of the CTAs each; a warp brings
// four words' weights from memory to its registers once and multiplies them with
// each token's elements from shared memory.  CTAs of different groups that have
// the same words run side by side, so that the weights come from HBM once and
// otherwise from L2.  128000 x 4096 at 1 and 8 tokens 295 and 326 us (7.1 and 6.4
// TB/s), at 16, 32 and 48 464, 864 and 1290: there the multiplications, the reads
// of shared memory and those of L2 add up.  The form for many takes 1837 for any
// of them (256 columns: 45, and 44 here at 48 tokens), so six groups of 8 are the
// most; of fewer, longer ones, twelve (12 of 32768 x 16384 1482, 13 of the other
// form 1983).  Two multiplications an instruction and 12 warps with the next
// columns on their way instead of 16 without: 16 tokens 513 to 464.  16 tokens a
// group, 64 sums a lane, is slower (2048 x 50257: 140 us, not 105).
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "tc_ptx.cuh"
#include "vocab_loss.h"

namespace moe {
namespace {

constexpr int MW = 128, KB = 64, KS = 2 * KB;   // words of a tile, columns of a box, K of a stage
constexpr int W_BYTES = MW * KS * 2;
constexpr int NST = 4;
constexpr int STAGE = W_BYTES + LOSS_FEW * KS * 2;  // for the most tokens
constexpr int BUFS = 4;                         // accumulators
constexpr int CHAIN = 2;                        // stages added up in TMEM
constexpr int TAIL = 32;                        // words a copy of the last tile
constexpr int THREADS = 192, EPI = 128;
constexpr int CTRL_OFF = NST * STAGE;
constexpr int SMEM = CTRL_OFF + 1024 + 1024;    // control block, alignment
static_assert(SMEM <= 232448, "shared memory budget");

struct FewMaps {
  CUtensorMap w, tail, x;
};
struct FewArgs {
  const int32_t* labels;
  float2* partial;  // [T][CTAs]
  float* picked;    // [LOSS_FEW]
  int T, d, V, words;
  uint32_t* err;
};

__device__ __forceinline__ float exp_of(float x) {  // of a difference, <= 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.44269504088896340736f));
  return y;
}
// One more logit: a token's maximum and the sum of exp of the distances to it.
__device__ __forceinline__ void add_logit(float& top, float& sum, float z) {
  const float best = fmaxf(top, z);
  const float e = exp_of(fminf(top, z) - base_of(best));  // 0 for a first one, and of -inf; NaN stays
  sum = z > top ? fmaf(sum, e, 1.f) : sum + (z == z ? e : z);
  top = best;
}

__device__ __forceinline__ uint4 ldg16_once(const float* p) {  // not to be read again
  uint4 u;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(p));
  return u;
}

template <int N>
__global__ void __launch_bounds__(THREADS, 1) loss_few_kernel(const __grid_constant__ FewMaps maps, const FewArgs a) {
  constexpr uint32_t IDESC = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(MW >> 4) << 24);
  constexpr uint32_t X_BYTES = N * KS * 2, COLS = BUFS * N;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + CTRL_OFF);
  uint64_t* empty_bar = full_bar + NST;
  uint64_t* tfull_bar = empty_bar + NST;    // [BUFS]
  uint64_t* tempty_bar = tfull_bar + BUFS;  // [BUFS]
  uint64_t* drain_bar = tempty_bar + BUFS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_label = reinterpret_cast<int*>(tmem_slot + 2);  // [N]

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(smem_addr(&full_bar[i]), 1);
      mbar_init(smem_addr(&empty_bar[i]), 1);
    }
    for (int i = 0; i < BUFS; ++i) {
      mbar_init(smem_addr(&tfull_bar[i]), 1);
      mbar_init(smem_addr(&tempty_bar[i]), EPI / 32);
    }
    mbar_init(smem_addr(drain_bar), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_enter();  // no global memory or TMEM access above this line
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), COLS);
    tmem_relinquish();
  }
  for (int i = threadIdx.x; i < N; i += THREADS) s_label[i] = i < a.T ? a.labels[i] : -1;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot, smem_base = smem_addr(smem);
  const int w0 = blockIdx.x * a.words, w1 = min(w0 + a.words, a.V);
  const int tiles = (w1 - w0 + MW - 1) / MW, stages = (a.d + KS - 1) / KS;

  if (warp == 0) {
    if (lane == 0) {
      prefetch_map(&maps.w);
      prefetch_map(&maps.tail);
      prefetch_map(&maps.x);
      int st = 0, issued = 0;
      uint32_t phase = 0;
      bool alive = true;
      for (int t = 0; t < tiles && alive; ++t) {
        const int word = w0 + t * MW, left = w1 - word, copies = left >= MW ? 0 : (left + TAIL - 1) / TAIL;
        for (int k = 0; k < stages; ++k) {
          if (!mbar_wait(smem_addr(&empty_bar[st]), phase ^ 1u, abort_flag, a.err, 970)) {
            alive = false;
            break;
          }
          const uint32_t fb = smem_addr(&full_bar[st]), sW = smem_base + st * STAGE, sX = sW + W_BYTES;
          mbar_expect_tx(fb, (copies == 0 ? W_BYTES : copies * TAIL * KS * 2) + X_BYTES);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int col = k * KS + b * KB;
            if (copies == 0) tma_load_2d(sW + b * (MW * 128), &maps.w, fb, col, word);
            for (int c = 0; c < copies; ++c)
              tma_load_2d(sW + b * (MW * 128) + c * (TAIL * 128), &maps.tail, fb, col, word + c * TAIL);
            tma_load_2d(sX + b * (N * 128), &maps.x, fb, col, 0);
          }
          ++issued;
          if (++st == NST) {
            st = 0;
            phase ^= 1u;
          }
        }
      }
      if (!alive) {  // the copies in flight end before the CTA may exit
        const int n = issued < NST ? issued : NST;
        for (int i = 0; i < n; ++i) {
          if (--st < 0) {
            st = NST - 1;
            phase ^= 1u;
          }
          for (uint32_t it = 0; it < (1u << 24) && !mbar_try_wait(smem_addr(&full_bar[st]), phase); ++it) {
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      int st = 0;
      uint32_t phase = 0, uses = 0;
      bool alive = true;
      for (int t = 0; t < tiles && alive; ++t)
        for (int k0 = 0; k0 < stages && alive; k0 += CHAIN, ++uses) {
          const uint32_t buf = uses % BUFS;
          if (!mbar_wait(smem_addr(&tempty_bar[buf]), ((uses / BUFS) & 1u) ^ 1u, abort_flag, a.err, 971)) {
            alive = false;
            break;
          }
          tc_fence_after();
          for (int k = k0; k < stages && k < k0 + CHAIN; ++k) {
            if (!mbar_wait(smem_addr(&full_bar[st]), phase, abort_flag, a.err, 972)) {
              alive = false;
              break;
            }
            tc_fence_after();
            const uint32_t sW = smem_base + st * STAGE, sX = sW + W_BYTES;
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
              for (int q = 0; q < KB / 16; ++q)
                umma_bf16(tmem_base + buf * N, sdesc(sW + b * (MW * 128) + q * 32, 16, 1024),
                          sdesc(sX + b * (N * 128) + q * 32, 16, 1024), IDESC, ((k - k0) | b | q) != 0 ? 1u : 0u);
            umma_commit(smem_addr(&empty_bar[st]));
            if (++st == NST) {
              st = 0;
              phase ^= 1u;
            }
          }
          if (alive) umma_commit(smem_addr(&tfull_bar[buf]));
        }
      umma_commit(smem_addr(drain_bar));
      for (uint32_t it = 0; it < (1u << 26) && !mbar_try_wait(smem_addr(drain_bar), 0); ++it) {
      }
    }
  } else {
    // ---- four warps, a word a thread ----
    const int q = warp & 3, row = q * 32 + lane;
    float top[N], sum[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      top[i] = -INFINITY;
      sum[i] = 0.f;
    }
    uint32_t uses = 0;
    bool alive = true;
    for (int t = 0; t < tiles && alive; ++t) {
      float v[N];
      for (int k0 = 0; k0 < stages; k0 += CHAIN, ++uses) {
        const uint32_t buf = uses % BUFS;
        if (!mbar_wait(smem_addr(&tfull_bar[buf]), (uses / BUFS) & 1u, abort_flag, a.err, 973)) {
          alive = false;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < N; c += 16) {
          uint32_t r[16];
          tmem_ld16(tmem_base + ((uint32_t)(q * 32) << 16) + buf * N + c, r);
          tmem_ld_wait16(r);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[c + i] = k0 == 0 ? __uint_as_float(r[i]) : v[c + i] + __uint_as_float(r[i]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_addr(&tempty_bar[buf]));
      }
      const int word = w0 + t * MW + row;
      if (alive && word < w1) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          add_logit(top[i], sum[i], v[i]);
          if (s_label[i] == word) a.picked[i] = v[i];
        }
      }
      __syncwarp();
    }
    // every copy has been used: the ring's memory holds the threads' sums [N][EPI + 1],
    // then the warps' [4][N]; a lane takes a token, the maximum first
    asm volatile("bar.sync 1, %0;" ::"n"(EPI) : "memory");
    float2* all = reinterpret_cast<float2*>(smem);
    float2* four = all + N * (EPI + 1);
    if (alive) {
#pragma unroll
      for (int i = 0; i < N; ++i) all[i * (EPI + 1) + row] = make_float2(top[i], sum[i]);
    }
    asm volatile("bar.sync 1, %0;" ::"n"(EPI) : "memory");
    auto join = [&](const float2* p, int n) {
      float best = -INFINITY, s = 0.f;
#pragma unroll 8
      for (int k = 0; k < n; ++k) best = fmaxf(best, p[k].x);
      const float at = base_of(best);
#pragma unroll 8
      for (int k = 0; k < n; ++k) s += p[k].y * exp_of(p[k].x - at);
      return make_float2(best, s);
    };
    for (int i = lane; i < N; i += 32) four[i * 5 + q] = join(all + i * (EPI + 1) + q * 32, 32);
    asm volatile("bar.sync 1, %0;" ::"n"(EPI) : "memory");
    if (row < N && row < a.T) a.partial[row * gridDim.x + blockIdx.x] = join(four + row * 5, 4);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, COLS);
}

// ---- float32 ----
constexpr int F32_NT = 384, F32_WARPS = F32_NT / 32, R = 4;  // words of a warp
constexpr int F32_SMEM = 208 * 1024;                         // of the tokens' rows
constexpr int F32_GROUPS = 6, F32_GROUPS_LONG = 12;          // of 8 tokens, of fewer

__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t x, float lo, float hi) {
  uint64_t w;
  asm("mov.b64 %0, {%1, %2};" : "=l"(w) : "f"(lo), "f"(hi));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(x), "l"(w));
}
// acc[n * R + r] = the lane's part of token n with word r; rows past the last word read it again.
// U * 128 columns at a time, with AHEAD those behind them on their way; a sum is
// that of the even and that of the odd columns, two multiplications an
// instruction.  CAP: infinities count as the largest bf16, as in the products of parts.
template <int N, int U, bool AHEAD, bool CAP>
__device__ __forceinline__ void dot_words(float (&acc)[N * R], const float* W, const float* xs, int d, int word, int V, int lane) {
  uint64_t two_sums[N * R];
#pragma unroll
  for (int i = 0; i < N * R; ++i) two_sums[i] = 0;
  const float* src[R];
#pragma unroll
  for (int r = 0; r < R; ++r) src[r] = W + (int64_t)min(word + r, V - 1) * d;
  auto load = [&](uint4 (&u)[U][R], int c0) {
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int r = 0; r < R; ++r) u[j][r] = c0 + j * 128 < d ? ldg16_once(src[r] + c0 + j * 128) : make_uint4(0, 0, 0, 0);
  };
  auto multiply = [&](const uint4 (&u)[U][R], int c0) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      if (c0 + j * 128 >= d) break;
      float w[R][4];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        unpack(u[j][r], w[r]);
        if constexpr (CAP) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (isinf(w[r][i])) w[r][i] = copysignf(0x1.fep127f, w[r][i]);
        }
      }
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(xs + n * d + c0 + j * 128);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          fma2(two_sums[n * R + r], x.x, w[r][0], w[r][1]);
          fma2(two_sums[n * R + r], x.y, w[r][2], w[r][3]);
        }
      }
    }
  };
  uint4 one[U][R];
  if constexpr (AHEAD) {
    uint4 two[U][R];
    load(one, lane * 4);
    for (int c0 = lane * 4; c0 < d; c0 += U * 256) {
      load(two, c0 + U * 128);
      multiply(one, c0);
      if (c0 + U * 128 >= d) break;
      load(one, c0 + U * 256);
      multiply(two, c0 + U * 128);
    }
  } else {
    for (int c0 = lane * 4; c0 < d; c0 += U * 128) {
      load(one, c0);
      multiply(one, c0);
    }
  }
#pragma unroll
  for (int i = 0; i < N * R; ++i)
    acc[i] = __uint_as_float((uint32_t)two_sums[i]) + __uint_as_float((uint32_t)(two_sums[i] >> 32));
}
// Sums over the lanes, halving what a lane has: it ends with those from lane * C / 32 on.
template <int C, int O>
__device__ __forceinline__ void add_lanes(float* v, int lane) {
  if constexpr (O > 0) {
    if constexpr (C > 1) {
      const bool upper = lane & O;
#pragma unroll
      for (int i = 0; i < C / 2; ++i) {
        const float keep = upper ? v[i + C / 2] : v[i], give = upper ? v[i] : v[i + C / 2];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, O);
      }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], O);
    }
    add_lanes<(C > 1 ? C / 2 : 1), O / 2>(v, lane);
  }
}

template <int N, int U, bool AHEAD>
__global__ void __launch_bounds__(F32_NT, 1) loss_few_f32_kernel(const FewArgs a, const float* x, const float* W, int groups) {
  extern __shared__ uint8_t smem_raw[];
  float* xs = reinterpret_cast<float*>(smem_raw);  // [N][d], 0 for tokens that are ignored
  __shared__ float2 s_sum[F32_WARPS][N];
  pdl_enter();
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, vecs = a.d / 4;
  const int t0 = blockIdx.x % groups * N, place = blockIdx.x / groups, places = gridDim.x / groups;
  for (int n = 0; n < N; ++n) {
    const int label = t0 + n < a.T ? a.labels[t0 + n] : -1;
    const bool valid = label >= 0 && label < a.V;
    for (int i = threadIdx.x; i < vecs; i += F32_NT)
      *reinterpret_cast<uint4*>(xs + n * a.d + i * 4) = valid ? ldg16(x + (int64_t)(t0 + n) * a.d + i * 4) : make_uint4(0, 0, 0, 0);
  }
  __syncthreads();
  constexpr int C = N * R, COPIES = 32 / C;  // lanes of a sum
  const int n = lane / (32 / N), at = lane / COPIES % R;
  const int label = t0 + n < a.T ? a.labels[t0 + n] : -1;
  float top = -INFINITY, sum = 0.f;
  for (int word = (place * F32_WARPS + warp) * R; word < a.V; word += places * F32_WARPS * R) {
    float acc[C];
    dot_words<N, U, AHEAD, false>(acc, W, xs, a.d, word, a.V, lane);
    add_lanes<C, 16>(acc, lane);
    if (!__all_sync(0xffffffffu, isfinite(acc[0]))) {
      dot_words<N, 1, false, true>(acc, W, xs, a.d, word, a.V, lane);
      add_lanes<C, 16>(acc, lane);
    }
    const int v = word + at;
    if (lane % COPIES == 0 && v < a.V) {
      add_logit(top, sum, acc[0]);
      if (v == label) a.picked[t0 + n] = acc[0];
    }
  }
  auto join = [](float& t, float& s, float t2, float s2) {
    const float best = fmaxf(t, t2), from = base_of(best);
    s = s * exp_of(t - from) + s2 * exp_of(t2 - from);
    t = best;
  };
#pragma unroll
  for (int o = 16 / N; o > 0; o /= 2) {
    const float t2 = __shfl_xor_sync(0xffffffffu, top, o), s2 = __shfl_xor_sync(0xffffffffu, sum, o);
    join(top, sum, t2, s2);
  }
  if (lane % (32 / N) == 0) s_sum[warp][n] = make_float2(top, sum);
  __syncthreads();
  if (threadIdx.x >= N || t0 + threadIdx.x >= a.T) return;
  float2 p = s_sum[0][threadIdx.x];
  for (int k = 1; k < F32_WARPS; ++k) join(p.x, p.y, s_sum[k][threadIdx.x].x, s_sum[k][threadIdx.x].y);
  a.partial[(t0 + threadIdx.x) * places + place] = p;
}

// A warp a token: the CTAs' sums, the loss; then the sum of the losses in token order.
__global__ void __launch_bounds__(1024) loss_few_join_kernel(const FewArgs a, int ctas, float* loss, float* lse, float* total) {
  pdl_enter();
  __shared__ float s_loss[LOSS_FEW];
  __shared__ int s_valid[LOSS_FEW];
  const int lane = threadIdx.x % 32;
  for (int t = threadIdx.x / 32; t < a.T; t += 32) {
    const int label = a.labels[t];
    const bool valid = label >= 0 && label < a.V;
    float best = -INFINITY, sum = 0.f;
#pragma unroll 4
    for (int c = lane; c < ctas; c += 32) best = fmaxf(best, a.partial[t * ctas + c].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
    const float at = base_of(best);
#pragma unroll 4
    for (int c = lane; c < ctas; c += 32) {
      const float2 p = a.partial[t * ctas + c];
      sum += p.y * expf(p.x - at);
    }
    sum = warp_sum(sum);
    if (lane == 0) {
      if (label >= a.V) report_error(a.err, DEV_BAD_LABEL, (uint32_t)t);
      const float l = valid ? (best - a.picked[t]) + logf(sum) : 0.f;
      loss[t] = s_loss[t] = l;
      lse[t] = valid ? best + logf(sum) : 0.f;
      s_valid[t] = valid;
    }
  }
  if (total == nullptr) return;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    int n = 0;
    for (int t = 0; t < a.T; ++t) {
      s += s_loss[t];
      n += s_valid[t];
    }
    total[0] = (float)s;
    total[1] = (float)n;
  }
}

// ------------------------------ host side ---------------------------------- //
// Words of a CTA: an equal share each, whole copies of the last tile's where they are few.
int words_of(int V) { return std::max(TAIL, ((V + sm_count() - 1) / sm_count() + 15) / 16 * 16); }

template <int N>
cudaError_t launch(const FewMaps& maps, const FewArgs& a, int ctas, cudaStream_t st) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  if (!done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(loss_few_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  LaunchScope ls(KK_LOSS_LOGITS, st);
  return launch_pdl(loss_few_kernel<N>, dim3(ctas), dim3(THREADS), SMEM, st, maps, a);
}

// float32 tokens of a group: 8, or fewer where they are few or long.
int f32_tokens(int T, int d) {
  int n = 1;
  while (n < 8 && n < T && (int64_t)2 * n * d * 4 <= F32_SMEM) n *= 2;
  return n;
}

template <int N, int U, bool AHEAD>
cudaError_t launch_f32(const LossArgs& l, const FewArgs& a, int groups, int places, cudaStream_t st) {
  static std::atomic<bool> done[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  if (!done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(loss_few_f32_kernel<N, U, AHEAD>, cudaFuncAttributeMaxDynamicSharedMemorySize, F32_SMEM);
    if (e != cudaSuccess) return e;
    done[dev] = true;
  }
  LaunchScope ls(KK_LOSS_LOGITS, st);
  return launch_pdl(loss_few_f32_kernel<N, U, AHEAD>, dim3(groups * places), dim3(F32_NT), (size_t)N * l.d * 4, st, a,
                    static_cast<const float*>(l.x), static_cast<const float*>(l.W), groups);
}

}  // namespace

bool loss_is_few(int T, int d, bool bf16) {
  if (bf16) return T <= LOSS_FEW;
  const int n = f32_tokens(T, d);
  return (int64_t)n * d * 4 <= F32_SMEM && T <= n * (n == 8 ? F32_GROUPS : F32_GROUPS_LONG);
}

size_t loss_few_bytes() { return ((size_t)sm_count() * sizeof(float2) + sizeof(float)) * LOSS_FEW; }

cudaError_t launch_loss_few(const LossArgs& l, uint32_t* err, cudaStream_t st) {
  FewArgs a{l.labels, static_cast<float2*>(l.ws), nullptr, l.T, l.d, l.V, words_of(l.V), err};
  a.picked = reinterpret_cast<float*>(a.partial + (size_t)sm_count() * LOSS_FEW);
  int ctas = (l.V + a.words - 1) / a.words;
  cudaError_t e;
  if (l.bf16) {
    if (!maps_ready()) return cudaErrorNotSupported;
    const int n = l.T <= 16 ? 16 : l.T <= 32 ? 32 : 64;
    FewMaps maps{};
    if (!make_map(&maps.w, l.W, l.V, l.d, KB, MW) || !make_map(&maps.tail, l.W, l.V, l.d, KB, TAIL) ||
        !make_map(&maps.x, l.x, l.T, l.d, KB, n))
      return cudaErrorInvalidValue;
    e = n == 16 ? launch<16>(maps, a, ctas, st) : n == 32 ? launch<32>(maps, a, ctas, st) : launch<64>(maps, a, ctas, st);
  } else {
    const int n = f32_tokens(l.T, l.d), groups = (l.T + n - 1) / n;
    ctas = std::min(sm_count() / groups, (l.V + F32_WARPS * R - 1) / (F32_WARPS * R));
    e = n == 1       ? launch_f32<1, 4, false>(l, a, groups, ctas, st)
        : n == 2     ? launch_f32<2, 4, false>(l, a, groups, ctas, st)
        : n == 4     ? launch_f32<4, 4, false>(l, a, groups, ctas, st)
        : l.d <= 512 ? launch_f32<8, 2, false>(l, a, groups, ctas, st)  // 48 x 32000 x 256: 44 us, 50 ahead
                     : launch_f32<8, 2, true>(l, a, groups, ctas, st);
  }
  if (e != cudaSuccess) return e;
  LaunchScope ls(KK_LOSS_COMBINE, st);
  return launch_pdl(loss_few_join_kernel, dim3(1), dim3(1024), 0, st, a, ctas, l.loss, l.lse, l.total);
}

}  // namespace moe
