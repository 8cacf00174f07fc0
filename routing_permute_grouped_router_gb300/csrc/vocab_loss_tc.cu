// The products of the vocabulary loss on the 5th-generation tensor cores.
//
//   LOGITS   z = x W^T -> each tile's maximum and sum of exponentials, the label's logit   A, B K-major
//   DLOGITS  z again -> dz = g (exp(z - lse) - [label]) in bf16 parts                      A, B K-major
//   GRADS    acc (+)= dz W (A K-major, B MN-major) and dW (+)= dz^T x (A, B MN-major)
//
// CTA pairs (clusters of two, one CTA an SM, 320 threads each) compute tiles of
// 256 x 256 with the 2-SM tcgen05 MMA, as the grouped GEMMs of the layer do:
// warp 0 loads by TMA (three 64 KB stages of two 64-wide k-blocks), warp 1
// issues the MMAs into one of two TMEM accumulators, warps 2 to 9 of both CTAs
// take the finished one, a row and 128 columns a thread.  Logits leave the SM as
// two floats a row and 128 columns.
//
// The tensor core cuts a sum off to fp32 after each MMA (it does not round), so
// a sum over K shrinks by some 2e-8 a step of 16: 1.6e-4 over a vocabulary of
// 130000.  Eight stages (K of 1024) at a time are therefore added up in TMEM, four
// of float32 operands, and their sums in the epilogue's registers, rounded; the two
// accumulators alternate, so the MMAs do not wait.  (float32 gradients are 1.2e-6 off
// with eight and 6.6e-7 with four, products in fp32 5e-7 to 3e-6; 777 x 1000 x 10007
// forward 121 and 124 us, backward 307 and 326.  Two cost 20 %.)
//
// float32 operands come as three bf16 parts of 8 bits each, whose sum they are
// exactly.  A product then runs over six pairs of parts, the smallest first (so
// the sums that are rounded often are small); the pairs left out are 2^-23 of
// the product in the mean, 2^-21 at most.  dz likewise has one part for a result in
// bf16, two (16 bits) for a float32 dW of bf16 inputs, three in float32.
//
// Every mbarrier wait is bounded (2 s); on expiry the kernel records
// DEV_TIMEOUT, drains its copies and MMAs, frees TMEM and exits.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "tc_ptx.cuh"
#include "vocab_loss.h"

namespace moe {
namespace {

constexpr int BM = 128, BN = 256, BK = 64;  // rows of a CTA (a pair has twice that), columns of a tile, a k-block
constexpr int BNH = BN / 2;
constexpr int KB = 2;                       // k-blocks of a stage
constexpr int BLOCK_BYTES = BM * BK * 2;    // a loaded box
constexpr int A_BYTES = KB * BLOCK_BYTES, STAGE = 2 * A_BYTES;
static_assert(BM == BNH && KB == 2, "boxes of A and B are alike");
constexpr int CHAIN = 8, CHAIN_F32 = 4;      // stages added up in TMEM
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int HALF = BN / 2;                // columns of a row that an epilogue thread holds
constexpr int BOX_BYTES = 4096;             // a warp's staged output box: 32 rows x 128 bytes
static_assert(HALF == LOSS_PART, "columns of a partial sum");
// A tile of long K wants three stages, which leaves a box a warp; one of short K
// waits for its epilogue, and has two boxes a warp and two stages.  (4096 x 512 x
// 32000 dz: 169 us with two boxes, 194 with three stages; at d 1024 248 and 221.
// A float32 dW of 64 and of 300 tokens, 4096 x 128000: 895 and 980, 1217 and 993.)
template <bool SHORT>
struct Shape {
  static constexpr int NST = SHORT ? 2 : 3, BOXES = SHORT ? 2 : 1;
  static constexpr int EPI_OFF = NST * STAGE, CTRL_OFF = EPI_OFF + EPI_WARPS * BOXES * BOX_BYTES;
  static constexpr int SMEM = CTRL_OFF + 512 + 1024;  // control block, alignment
  static_assert(SMEM <= 232448, "shared memory budget");
};
constexpr uint32_t TMEM_COLS = 512;         // two accumulators of 256 columns
constexpr int MAX_SEG = 6;
constexpr int GROUP_M = 16;                 // row tiles that share the columns' panels through L2
constexpr int SHORT_K = 4;                  // stages: K of 512
constexpr float LOG2E = 1.44269504088896340736f;

enum Kind { LOGITS = 0, DLOGITS = 1, GRADS = 2 };

// Tensor maps: LOGITS and DLOGITS 0 x, 1 W, 2 dz (store); GRADS 0 dz (A of acc), 1 W, 2 dz (A of dW), 3 x, 4 acc, 5 dW
struct Maps {
  CUtensorMap m[6];
};
// The pairs of parts of a product, as offsets of A and B in their maps.
struct Segs {
  int n;
  int a[MAX_SEG], b[MAX_SEG];
};
struct TcArgs {
  LossWork w;
  Segs seg[2];  // of the logits or of acc; of dW
  int with_dx, with_dw, dw_bf16, add_acc, add_dw;
  int chain;    // stages added up in TMEM
};

__host__ __device__ constexpr uint32_t idesc(bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((uint32_t)(BN >> 3) << 17) | ((uint32_t)((2 * BM) >> 4) << 24);
}

// 16-byte chunk j of row `lane` of a box, in the 128-byte swizzle of its tensor map
__device__ __forceinline__ uint32_t box_chunk(uint32_t box, int lane, int j) {
  return box + lane * 128 + (((uint32_t)j ^ (uint32_t)(lane & 7)) << 4);
}
// exp of a difference, which is formed first: it is exact where it matters, next to the maximum
__device__ __forceinline__ float exp_from(float z, float from) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"((z - from) * LOG2E));
  return y;
}

// ------------------------------ tiles -------------------------------------- //
struct Tile {
  int what;    // GRADS: 0 acc, 1 dW
  int m0, n0;  // the pair's first row, the first column
  int slice;   // of K: acc has a sum of its own for each
  int b0;      // the first stage
  int blocks;  // stages of one pair of parts
};
// How the tiles are dealt to the pairs.  LOGITS, DLOGITS: one after the other.
// GRADS: those of the longer kind first, in turn; the pairs that got one less
// then take `early` tiles of the other kind before all take theirs in turn.
struct Deal {
  int count[2];  // tiles of acc and of dW
  int len[2];    // their stages
  int first;     // the kind that comes first
  int extra, early;
  int nm, nn;    // row and column tiles of the logits; of acc
};

__device__ __forceinline__ int cdiv(int a, int b) { return (a + b - 1) / b; }

template <int KIND>
__device__ __forceinline__ Deal deal_of(const TcArgs& a, int n, int npairs) {
  Deal d{};
  const int rows = cdiv(n, 2 * BM);
  if (KIND != GRADS) {
    d.nm = rows;
    d.nn = KIND == LOGITS ? cdiv(a.w.V, BN) : a.w.piece / BN;
    d.count[0] = d.nm * d.nn;
    d.len[0] = cdiv(a.w.d, BK * KB);
    return d;
  }
  const int cols = cdiv(a.w.d, BN);
  d.nm = rows;
  d.nn = cols;
  d.count[0] = a.with_dx ? rows * cols * a.w.slices : 0;
  d.len[0] = cdiv(a.w.piece / (BK * KB), a.w.slices);
  d.count[1] = a.with_dw ? a.w.piece / BN * cols : 0;
  d.len[1] = cdiv(n, BK * KB);
  const int c0 = d.len[0] * a.seg[0].n, c1 = d.len[1] * a.seg[1].n;
  d.first = c1 > c0;
  const int longer = d.first ? c1 : c0, shorter = d.first ? c0 : c1;
  d.extra = d.count[d.first] % npairs;
  if (d.extra > 0 && shorter > 0) {
    d.early = (longer + shorter / 2) / shorter;
    const int most = d.count[d.first ^ 1] / (npairs - d.extra);
    d.early = d.early < most ? d.early : most;
  }
  return d;
}

// The j-th tile of a pair; false past the last.  `stages` are the piece's.
template <int KIND>
__device__ __forceinline__ bool tile_of(const Deal& d, int pair, int npairs, int stages, int j, Tile* t) {
  t->what = t->slice = t->b0 = 0;
  if (KIND != GRADS) {
    const int i = pair + j * npairs;
    if (i >= d.count[0]) return false;
    const int per = GROUP_M * d.nn, g = i / per, gm = d.nm - g * GROUP_M < GROUP_M ? d.nm - g * GROUP_M : GROUP_M;
    const int l = i - g * per;
    t->m0 = (g * GROUP_M + l % gm) * 2 * BM;
    t->n0 = l / gm * BN;
    t->blocks = d.len[0];
    return true;
  }
  int kind = d.first, i = pair + j * npairs;
  if (i >= d.count[kind]) {
    j -= d.count[kind] / npairs + (pair < d.extra ? 1 : 0);
    kind ^= 1;
    const int ahead = d.early * (npairs - d.extra);
    if (pair >= d.extra && j < d.early) i = j * (npairs - d.extra) + pair - d.extra;
    else i = ahead + (j - (pair >= d.extra ? d.early : 0)) * npairs + pair;
    if (i >= d.count[kind]) return false;
  }
  t->what = kind;
  t->n0 = i % d.nn * BN;
  int m = i / d.nn;
  t->blocks = d.len[kind];
  if (kind == 0) {
    t->slice = m / d.nm;
    m -= t->slice * d.nm;
    t->b0 = t->slice * d.len[0];
    const int left = stages - t->b0;  // fewer in the last slice; perhaps none
    t->blocks = left < t->blocks ? (left > 0 ? left : 0) : t->blocks;
  }
  t->m0 = m * 2 * BM;
  return true;
}

// This CTA's half of one stage: its 128 rows of A and its 128 columns of B over a K
// of 128, in boxes of 16 KB.  K-major operands: a box a k-block.  MN-major ones:
// a box 64 rows (columns) for all of the stage's K; boxes of one k-block each,
// twice as many, bound the products with W and x (TMA issue: 1.45 and 1.27
// PFLOP/s against the logits' 1.93).
template <int KIND>
__device__ __forceinline__ void load_stage(const Maps& maps, const TcArgs& a, const Tile& t, int seg, int b, uint32_t sA,
                                           uint32_t bar, uint32_t rank) {
  auto ld = [&](uint32_t dst, const CUtensorMap* m, int c0, int c1) {
    if (rank == 0) tma_load_2d(dst, m, bar, c0, c1);
    else tma_load_2d_pair(dst, m, bar, c0, c1);
  };
  const uint32_t sB = sA + A_BYTES;
  const int m0 = t.m0 + (int)rank * BM, n0 = t.n0 + (int)rank * BNH, k0 = b * (BK * KB);
  const Segs& s = a.seg[KIND == GRADS ? t.what : 0];
#pragma unroll
  for (int i = 0; i < KB; ++i) {
    const uint32_t dA = sA + i * BLOCK_BYTES, dB = sB + i * BLOCK_BYTES;
    if (KIND != GRADS) {
      ld(dA, &maps.m[0], s.a[seg] + k0 + i * BK, m0);
      ld(dB, &maps.m[1], s.b[seg] + k0 + i * BK, (KIND == DLOGITS ? a.w.v0 : 0) + n0);
    } else if (t.what == 0) {
      ld(dA, &maps.m[0], k0 + i * BK, s.a[seg] + m0);
      ld(dB, &maps.m[1], s.b[seg] + n0 + i * 64, a.w.v0 + k0);
    } else {
      ld(dA, &maps.m[2], m0 + i * 64, s.a[seg] + k0);
      ld(dB, &maps.m[3], s.b[seg] + n0 + i * 64, k0);
    }
  }
}

// ------------------------------ epilogues ---------------------------------- //
// A thread has 128 columns of one row, in registers; TMEM is free again.
template <int BOXES>
struct Epi {
  uint32_t box;          // the one that is filled next
  uint32_t uses[BOXES];  // completed waits on the boxes' input barriers
  bool pending[BOXES];   // an input load is in flight
  __device__ __forceinline__ void next() {
    if (BOXES == 2) box ^= 1u;
  }
};

// Columns past the vocabulary are left out; `left` is how many of the thread's are not.
__device__ __forceinline__ void mask_tail(float (&v)[HALF], int left) {
  if (left < HALF) {
#pragma unroll
    for (int i = 0; i < HALF; ++i)
      if (i >= left) v[i] = -INFINITY;
  }
}

// What an epilogue wants of a row, loaded while the MMAs run (rows up to Tp are there).
struct RowData {
  int label;
  float g, lse;
};

// The row's maximum over the columns, and the sum of exp of the distances to it.
__device__ __forceinline__ void logits_epilogue(const LossWork& w, int row, int col, const RowData& rd, float (&v)[HALF]) {
  const int at = rd.label - col;
  if (at >= 0 && at < HALF) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < HALF; ++i) z = at == i ? v[i] : z;
    w.picked[row] = z;
  }
  mask_tail(v, w.V - col);
  float top[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
  for (int i = 4; i < HALF; ++i) top[i & 3] = fmaxf(top[i & 3], v[i]);
  const float best = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  const float from = base_of(best);
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < HALF; ++i) s[i & 3] += exp_from(v[i], from);
  w.partial[(int64_t)(col / HALF) * w.Tp + row] = make_float2(best, (s[0] + s[1]) + (s[2] + s[3]));
}

// The warp's next box may be written again.  (Boxes of half the width, one filled
// while the other leaves, and plain stores of whole lines from the box are both
// slower: a tile of a float32 dW with one token's K 11 and 14 us, these 6.)
template <int BOXES>
__device__ __forceinline__ void wait_box(int lane) {
  if (lane == 0) {
    if (BOXES == 2) bulk_wait_read1();
    else bulk_wait_read0();
  }
  __syncwarp();
}
__device__ __forceinline__ void store_box(const CUtensorMap* map, uint32_t buf, int c0, int c1, int lane) {
  fence_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(map, buf, c0, c1);
    bulk_commit();
  }
}

// dz of the row over the columns, 64 of them a box, a box a part
template <int BOXES>
__device__ __forceinline__ void dlogits_epilogue(const Maps& maps, const LossWork& w, int row, int col, int lane,
                                                 uint32_t buf, Epi<BOXES>& es, const RowData& rd, float (&v)[HALF]) {
  const int at = rd.label - w.v0 - col;
  mask_tail(v, w.V - w.v0 - col);
#pragma unroll
  for (int i = 0; i < HALF; ++i) v[i] = exp_from(v[i], rd.lse);
  if (rd.label >= 0 && at >= 0 && at < HALF) {
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < HALF; ++i) {
      v[i] -= at == i ? 1.f : 0.f;
      z = at == i ? v[i] : z;
    }
    z *= rd.g;
    w.off[row] = z - __bfloat162float(__float2bfloat16_rn(z));  // of the first part
  }
#pragma unroll
  for (int i = 0; i < HALF; ++i) v[i] = rd.label >= 0 ? v[i] * rd.g : 0.f;  // 0 on padding, whatever W holds
#pragma unroll
  for (int c = 0; c < HALF; c += 64) {
#pragma unroll 1
    for (int p = 0; p < w.dzp; ++p) {
      const uint32_t box = buf + es.box * BOX_BYTES;
      wait_box<BOXES>(lane);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = v[c + 8 * q + i];
        const uint4 u = pack(x);
        sts128(box_chunk(box, lane, q), u);
        unpack(u, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c + 8 * q + i] -= x[i];  // what the part leaves
      }
      store_box(&maps.m[2], box, col + c, p * w.Tp + row - lane, lane);
      es.next();
    }
  }
}

// The old values of the box that is filled `ahead` from now, on their way while
// the MMAs run or the box before leaves.
template <int BOXES>
__device__ __forceinline__ void fetch_box(const CUtensorMap* map, uint32_t buf, uint32_t bar, int c0, int c1, int lane,
                                          uint32_t ahead, Epi<BOXES>& es) {
  const uint32_t h = BOXES == 2 ? es.box ^ ahead : 0;
  if (lane == 0) {
    bulk_wait_read0();
    mbar_expect_tx(bar + 8 * h, BOX_BYTES);
    tma_load_2d(buf + h * BOX_BYTES, map, bar + 8 * h, c0, c1);
  }
  es.pending[h] = true;
  __syncwarp();
}
// 128 columns of a row of acc or dW, stored or added to what is there, a box of 128 bytes a row at a time.
template <bool BF16, int BOXES>
__device__ __forceinline__ bool grads_epilogue(const CUtensorMap* map, int row0, int col, int d, bool add, int lane,
                                               uint32_t buf, uint32_t bar, Epi<BOXES>& es, float (&v)[HALF], float scale,
                                               uint32_t* err, volatile int* abort_flag) {
  constexpr int W = BF16 ? 64 : 32;  // columns of a box
#pragma unroll
  for (int c = 0; c < HALF; c += W) {
    if (col + c >= d) break;
    const uint32_t h = es.box, box = buf + h * BOX_BYTES;
    if (add) {
      if (!es.pending[h]) fetch_box<BOXES>(map, buf, bar, col + c, row0, lane, 0, es);
      if (BOXES == 2 && c + W < HALF && col + c + W < d) fetch_box<BOXES>(map, buf, bar, col + c + W, row0, lane, 1, es);
      if (!mbar_wait(bar + 8 * h, es.uses[h] & 1u, abort_flag, err, 962)) return false;
      ++es.uses[h];
      es.pending[h] = false;
    } else {
      wait_box<BOXES>(lane);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      constexpr int N = BF16 ? 8 : 4;
      float x[N], o[N];
      const uint32_t at = box_chunk(box, lane, j);
      if (add) unpack(lds128(at), o);
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = add ? fmaf(v[c + N * j + i], scale, o[i]) : v[c + N * j + i] * scale;
      sts128(at, pack(x));
    }
    store_box(map, box, col + c, row0, lane);
    es.next();
  }
  return true;
}

// ------------------------------ the kernel --------------------------------- //
// 168 registers a thread are all that ten warps can have (three share a quarter of
// the SM's): next to its 128 columns an epilogue thread spills 600 bytes in GRADS, 100
// to 140 in DLOGITS, 56 in LOGITS.
template <int KIND, bool SHORT>
__global__ void __launch_bounds__(THREADS, 1) loss_tc_kernel(const __grid_constant__ Maps maps,
                                                             const __grid_constant__ TcArgs a) {
  constexpr int NST = Shape<SHORT>::NST, BOXES = Shape<SHORT>::BOXES;
  extern __shared__ uint8_t smem_raw[];
  // the same offsets in both CTAs of the pair: the MMA reads both at these addresses
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(smem + Shape<SHORT>::CTRL_OFF);  // [NST] (used in the first CTA)
  uint64_t* empty_bar = full_bar + NST;                               // [NST]
  uint64_t* tfull_bar = empty_bar + NST;                              // [2]
  uint64_t* tempty_bar = tfull_bar + 2;                               // [2] (used in the first CTA)
  uint64_t* drain_bar = tempty_bar + 2;
  uint64_t* load_bar = drain_bar + 1;                                 // [EPI_WARPS][BOXES]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(load_bar + BOXES * EPI_WARPS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_ok = reinterpret_cast<int*>(tmem_slot + 2);

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x / 2, npairs = gridDim.x / 2;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(smem_addr(&full_bar[i]), 1);
      mbar_init(smem_addr(&empty_bar[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_addr(&tfull_bar[i]), 1);
      mbar_init(smem_addr(&tempty_bar[i]), 2 * EPI_WARPS);
    }
    mbar_init(smem_addr(drain_bar), 1);
    for (int i = 0; i < BOXES * EPI_WARPS; ++i) mbar_init(smem_addr(&load_bar[i]), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  pdl_enter();  // no global memory or TMEM access above this line
  cluster_sync();  // the peer's barriers exist before any arrival crosses the pair
  if (warp == 1) {
    tmem_alloc_pair(smem_addr(tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both TMEM bases written
  tc_fence_after();
  if (threadIdx.x == 0) {
    // both CTAs must see one TMEM base: the MMA writes the same columns in both
    const bool same = ld_shared_cluster_u32(mapa_shared(smem_addr(tmem_slot), rank ^ 1u)) == *tmem_slot;
    const int n = *a.w.count;
    const bool ok = same && n >= 0 && n <= a.w.T;
    if (!ok) report_error(a.w.err, DEV_BAD_COUNT, 900 + KIND);
    *s_ok = ok ? n : -1;
  }
  __syncthreads();
  // a CTA that found something wrong deals no tiles, and its peer has found the same
  const int n = *s_ok;
  Deal deal{};
  if (n >= 0) deal = deal_of<KIND>(a, n, npairs);
  const bool any = deal.count[0] + deal.count[1] > 0;
  const int stages = KIND == GRADS ? a.w.piece / (BK * KB) : 0;
  const uint32_t tmem_base = *tmem_slot, smem_base = smem_addr(smem);

  if (warp == 0) {
    if (lane == 0 && any) {
      // ---------------- TMA producer (both CTAs) ----------------
      for (int i = 0; i < (KIND == GRADS ? 4 : 2); ++i) prefetch_map(&maps.m[i]);
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool alive = true;
      Tile t;
      for (int j = 0; alive && tile_of<KIND>(deal, pair, npairs, stages, j, &t); ++j) {
        const int nseg = a.seg[KIND == GRADS ? t.what : 0].n;
        for (int s = 0; s < nseg && alive; ++s)
          for (int b = 0; b < t.blocks; ++b) {
            if (!mbar_wait(smem_addr(&empty_bar[stage]), phase ^ 1u, abort_flag, a.w.err, 910 + KIND)) {
              alive = false;
              break;
            }
            const uint32_t fb_local = smem_addr(&full_bar[stage]);
            if (rank == 0) mbar_expect_tx(fb_local, 2 * STAGE);
            const uint32_t fb = rank == 0 ? fb_local : mapa_shared(fb_local, 0);
            load_stage<KIND>(maps, a, t, s, t.b0 + b, smem_base + stage * STAGE, fb, rank);
            ++issued;
            if (++stage == NST) {
              stage = 0;
              phase ^= 1u;
            }
          }
      }
      if (!alive) {
        // drain the copies in flight before the CTA may exit: the first CTA watches its full
        // barriers; the second, whose copies complete on the first's, gives them a bounded 20 ms
        if (rank == 0) {
          const int k = issued < NST ? issued : NST;
          int s = stage;
          uint32_t ph = phase;
          for (int i = 0; i < k; ++i) {
            if (--s < 0) {
              s = NST - 1;
              ph ^= 1u;
            }
            for (uint32_t it = 0; it < (1u << 24) && !mbar_try_wait(smem_addr(&full_bar[s]), ph); ++it) {
            }
          }
        } else if (issued > 0) {
          const uint64_t t0 = globaltimer();
          while (globaltimer() - t0 < 20000000ull) {
          }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0 && any) {
      // ---------------- MMA issuer (first CTA of the pair) ----------------
      int stage = 0;
      uint32_t phase = 0, uses = 0;
      bool alive = true;
      Tile t;
      for (int j = 0; alive && tile_of<KIND>(deal, pair, npairs, stages, j, &t); ++j) {
        const bool a_mn = KIND == GRADS && t.what == 1, b_mn = KIND == GRADS;
        const uint32_t id = a_mn ? idesc(true, true) : b_mn ? idesc(false, true) : idesc(false, false);
        const int total = t.blocks * a.seg[KIND == GRADS ? t.what : 0].n;
        for (int b0 = 0; b0 < total && alive; b0 += a.chain) {
          const uint32_t acc = uses & 1u;
          if (!mbar_wait(smem_addr(&tempty_bar[acc]), ((uses >> 1) & 1u) ^ 1u, abort_flag, a.w.err, 920 + KIND)) {
            alive = false;
            break;
          }
          ++uses;
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + acc * BN;
          const int b1 = b0 + a.chain < total ? b0 + a.chain : total;
          for (int b = b0; b < b1; ++b) {
            if (!mbar_wait(smem_addr(&full_bar[stage]), phase, abort_flag, a.w.err, 930 + KIND)) {
              alive = false;
              break;
            }
            tc_fence_after();
            const uint32_t sA = smem_base + stage * STAGE, sB = sA + A_BYTES;
#pragma unroll
            for (int k16 = 0; k16 < KB * BK / 16; ++k16) {
              const uint32_t at = k16 / 4 * BLOCK_BYTES + k16 % 4 * 32;  // K-major
              const uint64_t ad = a_mn ? sdesc(sA + k16 * 2048, BLOCK_BYTES, 1024) : sdesc(sA + at, 16, 1024);
              const uint64_t bd = b_mn ? sdesc(sB + k16 * 2048, BLOCK_BYTES, 1024) : sdesc(sB + at, 16, 1024);
              umma_bf16_pair(d_tmem, ad, bd, id, ((b - b0) | k16) != 0 ? 1u : 0u);
            }
            umma_commit_pair(smem_addr(&empty_bar[stage]), 0x3);
            if (++stage == NST) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (alive) umma_commit_pair(smem_addr(&tfull_bar[acc]), 0x3);
        }
      }
      // all MMAs of the pair complete (in both CTAs' TMEM) before TMEM is released
      umma_commit_pair(smem_addr(drain_bar), 0x3);
    }
    if (lane == 0 && any) {
      for (uint32_t it = 0; it < (1u << 26) && !mbar_try_wait(smem_addr(drain_bar), 0); ++it) {
      }
    }
  } else if (any) {
    // ---------------- epilogue warps 2..9 (both CTAs) ----------------
    const int q = warp & 3;                   // TMEM lane quarter this warp may access
    const int side = (warp - 2) / 4 * HALF;   // and its columns
    const int ew = warp - 2;
    const uint32_t buf = smem_base + Shape<SHORT>::EPI_OFF + ew * BOXES * BOX_BYTES;
    const uint32_t lbar = smem_addr(&load_bar[BOXES * ew]);
    Epi<BOXES> es{};
    uint32_t uses = 0;  // accumulators taken so far
    Tile t;
    for (int j = 0; tile_of<KIND>(deal, pair, npairs, stages, j, &t); ++j) {
      const int row0 = t.m0 + (int)rank * BM + q * 32, col = t.n0 + side;
      const CUtensorMap* map = &maps.m[4 + t.what];
      const int orow = row0 + (KIND != GRADS ? 0 : t.what == 1 ? a.w.v0 : t.slice * a.w.Tp);
      const bool add = KIND == GRADS && (t.what == 0 ? a.add_acc : a.add_dw);
      const bool wanted = KIND != GRADS || ((t.what == 0 || orow < a.w.V) && col < a.w.d);
      const int total = t.blocks * a.seg[KIND == GRADS ? t.what : 0].n;
      if (add && wanted && total > 0) fetch_box<BOXES>(map, buf, lbar, col, orow, lane, 0, es);
      RowData rd{};
      if (KIND != GRADS) rd.label = a.w.label[row0 + lane];
      if (KIND == DLOGITS) {
        rd.g = a.w.grad[row0 + lane];
        rd.lse = a.w.lse[row0 + lane];
      }
      float v[HALF];
      if (total == 0) {
#pragma unroll
        for (int i = 0; i < HALF; ++i) v[i] = 0.f;
      }
      bool ok = true;
      for (int b = 0; b < total; b += a.chain) {
        const uint32_t acc = uses & 1u;
        if (!mbar_wait(smem_addr(&tfull_bar[acc]), (uses >> 1) & 1u, abort_flag, a.w.err, 940 + KIND)) {
          ok = false;
          break;
        }
        ++uses;
        tc_fence_after();
        const uint32_t tacc = tmem_base + ((uint32_t)(q * 32) << 16) + acc * BN + side;
#pragma unroll
        for (int c = 0; c < HALF; c += 32) {
          uint32_t r[32];
          tmem_ld32(tacc + c, r);
          tmem_ld_wait(r);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[c + i] = b == 0 ? __uint_as_float(r[i]) : v[c + i] + __uint_as_float(r[i]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          const uint32_t te = smem_addr(&tempty_bar[acc]);
          if (rank == 0) mbar_arrive(te);
          else mbar_arrive_cluster(mapa_shared(te, 0));
        }
      }
      if (!ok) break;
      if (KIND == LOGITS) {
        logits_epilogue(a.w, row0 + lane, col, rd, v);
      } else if (KIND == DLOGITS) {
        dlogits_epilogue<BOXES>(maps, a.w, row0 + lane, col, lane, buf, es, rd, v);
      } else if (wanted && (total > 0 || !add)) {  // no labelled tokens: dW is 0, or as it was
        const float scale = t.what == 1 && a.w.mean && n > 0 ? 1.f / (float)n : 1.f;
        if (t.what == 1 && a.dw_bf16)
          ok = grads_epilogue<true, BOXES>(map, orow, col, a.w.d, add, lane, buf, lbar, es, v, scale, a.w.err,
                                    abort_flag);
        else
          ok = grads_epilogue<false, BOXES>(map, orow, col, a.w.d, add, lane, buf, lbar, es, v, scale, a.w.err, abort_flag);
        if (!ok) break;
      }
    }
    // input loads still in flight (only after an abort), then every store
    for (int h = 0; h < BOXES; ++h)
      if (es.pending[h])
        for (uint32_t it = 0; it < (1u << 24) && !mbar_try_wait(lbar + 8 * h, es.uses[h] & 1u); ++it) {
        }
    if (lane == 0) bulk_wait_all();
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still touch its barriers, operands or TMEM
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, TMEM_COLS);
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
// The pairs of parts, smallest products first; la and lb are the parts' distances in the maps.
Segs segs(int pa, int pb, int la, int lb) {
  Segs s{};
  for (int sum = (pa > pb ? pa : pb) - 1; sum >= 0; --sum)
    for (int i = 0; i <= sum; ++i)
      if (i < pa && sum - i < pb) {
        s.a[s.n] = i * la;
        s.b[s.n] = (sum - i) * lb;
        ++s.n;
      }
  return s;
}

template <int KIND, bool SHORT>
cudaError_t launch(const Maps& maps, const TcArgs& args, int64_t tiles, int kind, cudaStream_t st) {
  static std::atomic<int> pairs_of[64];  // pairs that are resident at once, 0 where it has not been asked
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = Shape<SHORT>::SMEM;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(2);
  int pairs = pairs_of[dev].load(std::memory_order_acquire);
  if (pairs == 0) {
    const cudaError_t e = cudaFuncSetAttribute(loss_tc_kernel<KIND, SHORT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Shape<SHORT>::SMEM);
    if (e != cudaSuccess) return e;
    if (cudaOccupancyMaxActiveClusters(&pairs, loss_tc_kernel<KIND, SHORT>, &cfg) != cudaSuccess || pairs <= 0) {
      cudaGetLastError();
      pairs = sm_count() / 2;
    }
    pairs_of[dev].store(pairs, std::memory_order_release);
  }
  if (tiles <= 0) return cudaSuccess;
  cfg.gridDim = dim3((unsigned)(2 * std::min<int64_t>(tiles, pairs)));
  cfg.numAttrs = 2;
  LaunchScope ls(kind, st);
  return cudaLaunchKernelEx(&cfg, loss_tc_kernel<KIND, SHORT>, maps, args);
}

template <int KIND>
cudaError_t logits(const LossWork& w, cudaStream_t st) {
  if (!maps_ready()) return cudaErrorNotSupported;
  Maps maps{};
  TcArgs a{};
  a.w = w;
  a.chain = w.parts == 1 ? CHAIN : CHAIN_F32;
  a.seg[0] = segs(w.parts, w.parts, w.ldx, w.ldw);
  bool ok = make_map(&maps.m[0], w.xp, w.Tp, (uint64_t)w.parts * w.ldx, BK, BM) &&
            make_map(&maps.m[1], w.wp, w.V, (uint64_t)w.parts * w.ldw, BK, BNH);
  if (KIND == DLOGITS) ok = ok && make_map(&maps.m[2], w.dz, (uint64_t)w.dzp * w.Tp, w.piece, 64, 32);
  if (!ok) return cudaErrorInvalidValue;
  const int64_t cols = KIND == LOGITS ? (w.V + BN - 1) / BN : w.piece / BN;
  const int64_t tiles = (int64_t)(w.Tp / (2 * BM)) * cols;
  if constexpr (KIND == LOGITS)
    return launch<KIND, false>(maps, a, tiles, KK_LOSS_LOGITS, st);
  else
    return (w.d + 127) / 128 * a.seg[0].n <= SHORT_K ? launch<KIND, true>(maps, a, tiles, KK_LOSS_DLOGITS, st)
                                                    : launch<KIND, false>(maps, a, tiles, KK_LOSS_DLOGITS, st);
}

}  // namespace

bool maps_ready() { return encoder() != nullptr; }
bool make_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols, uint32_t box_cols, uint32_t box_rows,
              bool fp32) {
  const uint64_t es = fp32 ? 4 : 2;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * es};
  cuuint32_t box[2] = {box_cols, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return encoder()(m, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
                   const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t tc_loss_logits(const LossWork& w, cudaStream_t st) { return logits<LOGITS>(w, st); }
cudaError_t tc_loss_dlogits(const LossWork& w, cudaStream_t st) { return logits<DLOGITS>(w, st); }

cudaError_t tc_loss_grads(const LossWork& w, bool dx, void* dW, bool dw_bf16, bool accumulate, cudaStream_t st) {
  if (!maps_ready()) return cudaErrorNotSupported;
  Maps maps{};
  TcArgs a{};
  a.w = w;
  a.chain = w.parts == 1 ? CHAIN : CHAIN_F32;
  a.with_dx = dx;
  a.with_dw = dW != nullptr;
  a.dw_bf16 = dw_bf16;
  a.add_acc = w.v0 > 0;
  a.add_dw = accumulate;
  // dx in bf16 needs the first part of dz alone
  a.seg[0] = segs(w.parts == 1 ? 1 : w.dzp, w.parts, w.Tp, w.ldw);
  a.seg[1] = segs(w.dzp, w.parts, w.Tp, w.ldx);
  const uint64_t planes = (uint64_t)w.dzp * w.Tp;
  bool ok = make_map(&maps.m[0], w.dz, planes, w.piece, BK, BM) && make_map(&maps.m[2], w.dz, planes, w.piece, 64, KB * BK) &&
            make_map(&maps.m[1], w.wp, w.V, (uint64_t)w.parts * w.ldw, 64, KB * BK) &&
            make_map(&maps.m[3], w.xp, w.Tp, (uint64_t)w.parts * w.ldx, 64, KB * BK);
  if (dx) ok = ok && make_map(&maps.m[4], w.acc, (uint64_t)w.slices * w.Tp, w.d, 32, 32, true);
  if (dW) ok = ok && make_map(&maps.m[5], dW, w.V, w.d, dw_bf16 ? 64 : 32, 32, !dw_bf16);
  if (!ok) return cudaErrorInvalidValue;
  const int64_t cols = (w.d + BN - 1) / BN;
  const int64_t tiles = ((dx ? (int64_t)w.Tp / (2 * BM) * w.slices : 0) + (dW ? w.piece / BN : 0)) * cols;
  return dW && w.Tp / 128 * a.seg[1].n <= SHORT_K ? launch<GRADS, true>(maps, a, tiles, KK_LOSS_GRADS, st)
                                                 : launch<GRADS, false>(maps, a, tiles, KK_LOSS_GRADS, st);
}

}  // namespace moe
