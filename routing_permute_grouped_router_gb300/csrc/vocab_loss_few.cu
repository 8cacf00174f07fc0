// The vocabulary loss of at most 64 bf16 tokens, as a serving step scores them.
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
// Sums over K of 1024 at a time are added up in TMEM and then, rounded, in
// registers, as in the products of many tokens.
#include <cuda.h>
#include <cudaTypedefs.h>

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
constexpr int CHAIN = 8;                        // stages added up in TMEM
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
  if (best == -INFINITY && z == z) return;  // nothing but -inf so far
  const float e = exp_of(fminf(top, z) - best);  // 0 for a first one; NaN stays
  sum = z > top ? fmaf(sum, e, 1.f) : sum + (z == z ? e : z);
  top = best;
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
      const float at = best == -INFINITY ? 0.f : best;
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
    const float at = best == -INFINITY ? 0.f : best;
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
// Looked up once; a thread that comes meanwhile waits for it.
PFN_cuTensorMapEncodeTiled_v12000 encoder() {
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
bool make_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_rows) {
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {KB, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
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

}  // namespace

size_t loss_few_bytes() { return ((size_t)sm_count() * sizeof(float2) + sizeof(float)) * LOSS_FEW; }

cudaError_t launch_loss_few(const LossArgs& l, uint32_t* err, cudaStream_t st) {
  if (encoder() == nullptr) return cudaErrorNotSupported;
  const int n = l.T <= 16 ? 16 : l.T <= 32 ? 32 : 64;
  FewArgs a{l.labels, static_cast<float2*>(l.ws), nullptr, l.T, l.d, l.V, words_of(l.V), err};
  a.picked = reinterpret_cast<float*>(a.partial + (size_t)sm_count() * LOSS_FEW);
  FewMaps maps{};
  if (!make_map(&maps.w, l.W, l.V, l.d, MW) || !make_map(&maps.tail, l.W, l.V, l.d, TAIL) || !make_map(&maps.x, l.x, l.T, l.d, n))
    return cudaErrorInvalidValue;
  const int ctas = (l.V + a.words - 1) / a.words;
  const cudaError_t e = n == 16 ? launch<16>(maps, a, ctas, st) : n == 32 ? launch<32>(maps, a, ctas, st) : launch<64>(maps, a, ctas, st);
  if (e != cudaSuccess) return e;
  LaunchScope ls(KK_LOSS_COMBINE, st);
  return launch_pdl(loss_few_join_kernel, dim3(1), dim3(1024), 0, st, a, ctas, l.loss, l.lse, l.total);
}

}  // namespace moe
