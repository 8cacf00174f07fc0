// Layer norm of the rows in front of the layer, forward and backward.
//
//   forward   mean = sum(x) / d,  rstd = 1 / sqrt(sum((x - mean)^2) / d + eps)
//             y = (x - mean) * rstd * gamma + beta
//   backward  n = (x - mean) * rstd,  v = dy * gamma
//             dx = rstd * (v - sum(v) / d - n * sum(v n) / d)  [+ dres]
//             dgamma = sum over rows of dy * n,  dbeta = sum over rows of dy
//
// Both passes are bound by HBM: the forward reads and writes a row once, the
// backward reads x, dy (and dres) and writes dx.  `tpr` threads share a row (a
// CTA, or a warp of one where 32 are enough), 16 elements each: 24 rows of up to
// 512 elements, three of 4096, one of 8192 are in the registers of an SM in the
// forward (16, two and one in the backward) while plain copies bring the next
// ones into a ring in shared memory, up to four rows deep, so the loads' latency is out of
// the way of the two reductions of a row.  (32768 x 4096 bf16: 87 us forward,
// 6.2 TB/s, and 168 us backward, 6.4 TB/s; with the loads in registers and no
// ring 155 and 367.)  The variance is of distances from a point near the mean,
// so a large mean neither cancels nor loses the last bits of x - mean, and needs
// no second read.  Threads keep their columns' gamma, beta and, in the
// backward, dgamma and dbeta sums in registers over all rows of the CTA; the
// sums of the CTAs are added in CTA order by a second kernel, so results do
// not depend on timing.  All statistics and sums are fp32.
//
// A copy has to begin and end on 16 bytes.  Rows of another length are copied
// with up to 15 bytes more on either side and read from shared memory element
// by element; what that would read past the tensor's end is loaded directly.
// Rows of more than 8192 elements are walked in a loop (the wide kernels),
// again from cache for each pass, and the backward reads x and dy once more for
// dgamma and dbeta.
#include "block.h"
#include "common.cuh"

namespace moe {
namespace {

constexpr int MAX_TPR = 512;   // most threads that share a row held in registers
constexpr int EPT = 16;        // elements of a row a thread holds
constexpr int FWD_REGS = 80;   // a thread's in the forward: three CTAs of 256 fit an SM
constexpr int BWD_NT = 512;    // threads of the backward's CTAs, one an SM (few partial sums)
constexpr int MAX_GROUPS = BWD_NT / 32;
constexpr int SMEM_SM = 220 * 1024;             // shared memory of an SM that the rings may take
constexpr int RING = 4;        // most rows on their way to a group of threads
constexpr int WIDE_NT = 512;   // threads a CTA of the wide kernels
constexpr int RED_COLS = 32, RED_STRIPS = 32;

// Element c (of EPT) of thread r of tpr, in whole vectors of VN or one by one.
template <int VN>
__device__ __forceinline__ int column(int r, int tpr, int c) {
  return (r + c / VN * tpr) * VN + c % VN;
}
// whether it is one of the row's d (d is a multiple of VN)
template <int VN>
__device__ __forceinline__ bool in_row(int r, int tpr, int c, int d) {
  return (r + c / VN * tpr) * VN < d;
}

// Two fp32 operations in one instruction; each half rounds as the scalar one does.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "add.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 z, x, y;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// A group of threads: `warps` warps that share a row, the g-th of its CTA.
// (SEVERAL: the CTA may have several groups of more than a warp.)
template <bool SEVERAL>
struct Group {
  int g, r, tpr, warps;
  __device__ __forceinline__ explicit Group(int tpr_) : g(threadIdx.x / tpr_), r(threadIdx.x % tpr_), tpr(tpr_), warps(tpr_ / 32) {}
  __device__ __forceinline__ void sync() const {
    if (warps == 1) __syncwarp();
    else if (SEVERAL) asm volatile("bar.sync %0, %1;" ::"r"(g + 1), "r"(tpr) : "memory");
    else __syncthreads();
  }
  // Every warp gives one float4; after sync() each thread gets that of warp
  // lane % warps, so xor shuffles over the warps (a power of two) finish a
  // sum.  scratch has two rows of 16, used in turn.
  __device__ __forceinline__ void give(float4 v, float4* scratch, int turn) const {
    if (threadIdx.x % 32 == 0) scratch[turn * 16 + threadIdx.x / 32] = v;
  }
  __device__ __forceinline__ float4 get(const float4* scratch, int turn) const {
    return scratch[turn * 16 + g * warps + (threadIdx.x & (warps - 1))];
  }
};
// Two sums over a warp: of a in the lower half of its lanes, of b in the upper half.
__device__ __forceinline__ float half_sums(float a, float b, bool upper) {
  float v = upper ? b : a;
  v += __shfl_xor_sync(0xffffffffu, upper ? a : b, 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float sum_over(float v, int n) {  // n a power of two up to 16
#pragma unroll
  for (int o = 1; o <= 8; o *= 2)
    if (o < n) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---- the ring ----
__device__ __forceinline__ uint32_t sm_addr(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy_row(uint32_t dst, const char* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ bool ring_ready(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits for the barrier's phase, two seconds at most.
__device__ __noinline__ void ring_wait(uint32_t bar, uint32_t parity, uint32_t* err) {
  uint64_t t0 = 0;
  for (uint32_t i = 0; i < (1u << 30); ++i) {
    if (ring_ready(bar, parity)) return;
    if ((i & 255u) == 255u) {
      uint64_t t;
      asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
      if (t0 == 0) t0 = t;
      if (t - t0 > 2000000000ull) break;
    }
  }
  report_error(err, DEV_TIMEOUT, 760);
}

// Where a row's copy begins and how long it is: the row itself, or the 16-byte
// units that hold it, cut off at the end of the tensor.
struct Span {
  int64_t at;       // byte offset of the copy in the tensor
  int skip, bytes;  // bytes before the row's first element; bytes of the copy
  bool whole;       // it has all of the row
};
template <typename T, bool WHOLE>
__device__ __forceinline__ Span row_span(int64_t row, int64_t rows, int d) {
  const int64_t b0 = row * d * (int64_t)sizeof(T), b1 = b0 + d * (int64_t)sizeof(T);
  if (WHOLE) return {b0, 0, (int)(b1 - b0), true};
  const int64_t total = rows * d * (int64_t)sizeof(T), a0 = b0 & ~(int64_t)15;
  int64_t a1 = (b1 + 15) & ~(int64_t)15;
  if (a1 > total) a1 = total & ~(int64_t)15;
  return {a0, (int)(b0 - a0), a1 > a0 ? (int)(a1 - a0) : 0, a1 >= b1};
}

// A thread's elements come in chunks, pairs of fp32: a vector of the row, or
// eight single elements where rows are not whole vectors.
template <typename T, bool WHOLE>
struct Chunk {
  static constexpr int N = WHOLE ? Vec<T>::N : 8;
};

// Chunk i of a row, from the ring.  Past the row's end come zeros, or `fill`
// where rows are not whole vectors.
template <typename T, bool WHOLE>
__device__ __forceinline__ void take(const char* stage, const Span& sp, const T* tensor, int r, int tpr, int d, int i,
                                     float2 (&v)[Chunk<T, WHOLE>::N / 2], float fill = 0.f) {
  if constexpr (WHOLE) {
    const int q = r + i * tpr;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (q * Vec<T>::N < d) u = *reinterpret_cast<const uint4*>(stage + q * 16);
    float w[Vec<T>::N];
    unpack(u, w);
#pragma unroll
    for (int j = 0; j < Vec<T>::N; j += 2) v[j / 2] = make_float2(w[j], w[j + 1]);
  } else {
    const int step = tpr * (int)sizeof(T), left = ((d - r + tpr - 1) >> (31 - __clz(tpr))) - i * 8;  // the thread's elements from here on
    int at = sp.skip + (r + i * 8 * tpr) * (int)sizeof(T);
    if (sp.whole) {
      const char* p = stage + at;
#pragma unroll
      for (int j = 0; j < 8; ++j, p += step) {
        const float w = j < left ? to_f32(*reinterpret_cast<const T*>(p)) : fill;
        (j & 1 ? v[j / 2].y : v[j / 2].x) = w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j, at += step) {
        float w = fill;
        if (j < left)
          w = to_f32(at < sp.bytes ? *reinterpret_cast<const T*>(stage + at) : tensor[(sp.at + at) / (int64_t)sizeof(T)]);
        (j & 1 ? v[j / 2].y : v[j / 2].x) = w;
      }
    }
  }
}
template <typename T, bool WHOLE>
__device__ __forceinline__ void put(T* row, int r, int tpr, int d, int i, const float2 (&v)[Chunk<T, WHOLE>::N / 2]) {
  if constexpr (WHOLE) {
    const int q = r + i * tpr;
    float w[Vec<T>::N];
#pragma unroll
    for (int j = 0; j < Vec<T>::N; j += 2) {
      w[j] = v[j / 2].x;
      w[j + 1] = v[j / 2].y;
    }
    if (q * Vec<T>::N < d) stg16(row + (size_t)q * Vec<T>::N, pack(w));
  } else {
    const int left = ((d - r + tpr - 1) >> (31 - __clz(tpr))) - i * 8;
    T* p = row + r + i * 8 * tpr;
#pragma unroll
    for (int j = 0; j < 8; ++j, p += tpr)
      if (j < left) *p = from_f32<T>(j & 1 ? v[j / 2].y : v[j / 2].x);
  }
}

struct NormArgs {
  const void* x;
  const void* dy;
  const void* dres;
  const float* gamma;
  const float* beta;
  const float* mean_in;
  const float* rstd_in;
  void* out;  // y or dx
  float* mean;
  float* rstd;
  float* partial;  // [CTAs][2][d]: dgamma, dbeta
  float* dgamma;
  float* dbeta;
  int64_t rows;
  int d, tpr, parts, accumulate;
  int slot, ring;  // bytes of a row's place in the ring, places
  float eps;
  uint32_t* err;
};

// A group of tpr threads, its rows (first, first + step, ...) and its ring.
// The group's first thread starts the copies; a place is filled again once the
// group has read its row for the last time.
template <typename T, bool WHOLE, int NBUF>
struct Rows {
  const char* src[NBUF];
  char* base;
  uint64_t* bars;
  int64_t first, step, rows;
  int d, slot, ring;
  int at = 0;           // the place of the row in work
  uint32_t phase = 0;   // and its barrier's phase
  __device__ __forceinline__ void start(int64_t row, int p) const {
    if (row >= rows) return;
    const Span sp = row_span<T, WHOLE>(row, rows, d);
    const uint32_t bar = sm_addr(bars + p);
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(sp.bytes * NBUF) : "memory");
    if (sp.bytes > 0) {
#pragma unroll
      for (int b = 0; b < NBUF; ++b) copy_row(sm_addr(base + (p * NBUF + b) * slot), src[b] + sp.at, sp.bytes, bar);
    }
  }
  __device__ __forceinline__ void wait(uint32_t* err) const {
    if (!ring_ready(sm_addr(bars + at), phase)) ring_wait(sm_addr(bars + at), phase, err);
  }
  __device__ __forceinline__ const char* place_at(int p, int b) const { return base + (p * NBUF + b) * slot; }
  __device__ __forceinline__ const char* place(int b) const { return place_at(at, b); }
  __device__ __forceinline__ void next() {
    if (++at == ring) {
      at = 0;
      phase ^= 1u;
    }
  }
  // The row in work has been taken: its place gets the row `ring` turns on.
  __device__ __forceinline__ void taken(int64_t row, bool leader) {
    if (leader) start(row + ring * step, at);
    next();
  }
};

extern __shared__ __align__(128) char norm_smem[];

template <typename T, bool WHOLE, int NBUF>
__device__ __forceinline__ Rows<T, WHOLE, NBUF> begin_rows(const NormArgs& a, uint64_t* bars, int r) {
  const int groups = blockDim.x / a.tpr, g = threadIdx.x / a.tpr;  // rows go to all CTAs before a second group of any
  Rows<T, WHOLE, NBUF> R;
  R.src[0] = static_cast<const char*>(a.x);
  if (NBUF > 1) R.src[1] = static_cast<const char*>(a.dy);
  if (NBUF > 2) R.src[2] = static_cast<const char*>(a.dres);
  R.base = norm_smem + (size_t)g * a.ring * NBUF * a.slot;
  R.bars = bars + g * RING;
  R.first = (int64_t)g * gridDim.x + blockIdx.x;
  R.step = (int64_t)gridDim.x * groups;
  R.rows = a.rows;
  R.d = a.d;
  R.slot = a.slot;
  R.ring = a.ring;
  if (threadIdx.x == 0) {
    for (int i = 0; i < groups * RING; ++i)
      asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(sm_addr(bars + i)) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_enter();  // see pdl_wait: no global access before this
  if (r == 0)
    for (int i = 0; i < a.ring; ++i) R.start(R.first + i * R.step, i);
  return R;
}

// The columns' weights, in pairs (0 past the row's end).
template <int VN>
__device__ __forceinline__ void take_weights(const float* w, int r, int tpr, int d, float2 (&v)[EPT / 2]) {
#pragma unroll
  for (int c = 0; c < EPT; ++c) {
    const float u = in_row<VN>(r, tpr, c, d) ? __ldg(w + column<VN>(r, tpr, c)) : 0.f;
    (c & 1 ? v[c / 2].y : v[c / 2].x) = u;
  }
}

// Distances are taken from the mean of a sample of the row, 32 elements spread
// over it (fewer of a short row), and their sum and the sum of their squares
// then give the mean and the variance in one reduction:
//   mean = near + s1 / d,  variance = s2 / d - (s1 / d)^2
// The sample's mean is about a sixth of a deviation off, so hardly anything
// cancels; at worst, where the sample alone holds what is large, the terms are
// d / 32 times their difference (a channel of 1000 in the sample, d 8192: rstd to
// 1e-6, not 2e-7).  The sample's size is a power of two, so the mean of a row of
// one value is that value and x - mean is 0, for any d and value: the rounded
// sum of a row times a rounded 1 / d can be ulps away, which eps 1e-5 makes 0.02
// gamma of y at the value 1000.  (Two-pass sums over the warps, corrected by the
// sum of the distances: 107 us at 32768 x 4096 bf16, this form 87.)
template <typename T, bool WHOLE>
__global__ void __maxnreg__(FWD_REGS) norm_fwd_kernel(const NormArgs a) {
  constexpr int VN = WHOLE ? Vec<T>::N : 1, CN = Chunk<T, WHOLE>::N / 2;
  __shared__ float scratch[2][2][16];
  __shared__ uint64_t bars[MAX_GROUPS * RING];
  int turn = 0;
  const Group<false> grp(a.tpr);
  const int r = grp.r, nw = grp.warps;
  Rows<T, WHOLE, 1> R = begin_rows<T, WHOLE, 1>(a, bars, r);
  T* y = static_cast<T*>(a.out);
  const float inv = 1.f / (float)a.d;
  float2 ga[EPT / 2], be[EPT / 2];
  take_weights<VN>(a.gamma, r, a.tpr, a.d, ga);
  take_weights<VN>(a.beta, r, a.tpr, a.d, be);
  // The lane's element of the sample: the first one that it holds where a warp
  // has the row (of `size` lanes that hold any), else one of its own 4-byte bank
  // of shared memory, 33 banks at least ahead of the row's end.
  const int lane = threadIdx.x % 32, full = __popc(__ballot_sync(0xffffffffu, in_row<VN>(lane, a.tpr, 0, a.d)));
  const int size = 1 << (31 - __clz(full | 1));
  const float each = lane < size ? 1.f / (float)size : 0.f;
  const int from_at = nw > 1 ? (lane * (a.d * (int)sizeof(T) / 4 - 64) / 32 / 32 * 32 + lane) * 4
                             : (lane < size ? lane * VN * (int)sizeof(T) : 0);
  const bool upper = lane >= 16;
  const float eps = upper ? a.eps : 0.f;
#pragma unroll 1
  for (int64_t row = R.first; row < a.rows; row += R.step) {
    const Span sp = row_span<T, WHOLE>(row, a.rows, a.d);
    R.wait(a.err);
    const int sat = sp.skip + from_at;
    float near = to_f32(WHOLE || sp.whole || sat < sp.bytes ? *reinterpret_cast<const T*>(R.place(0) + sat)
                                                            : static_cast<const T*>(a.x)[(sp.at + sat) / (int64_t)sizeof(T)]);
    near = warp_sum(each != 0.f ? near * each : 0.f);
    float2 v[EPT / 2 / CN][CN];
#pragma unroll
    for (int i = 0; i < EPT / 2 / CN; ++i)
      take<T, WHOLE>(R.place(0), sp, static_cast<const T*>(a.x), r, a.tpr, a.d, i, v[i], near);
    float2 s1 = both(0.f), s2 = both(0.f);
#pragma unroll
    for (int i = 0; i < EPT / 2 / CN; ++i)
#pragma unroll
      for (int c = 0; c < CN; ++c) {
        // past the row's end the distance is 0
        v[i][c] = add2(v[i][c], both(!WHOLE || in_row<VN>(r, a.tpr, 2 * (i * CN + c), a.d) ? -near : 0.f));
        s1 = add2(s1, v[i][c]);
        s2 = fma2(v[i][c], v[i][c], s2);
      }
    // s1 in the lower half of the lanes, s2 in the upper half, over the warp and then over the warps
    float m = half_sums(s1.x + s1.y, s2.x + s2.y, upper);
    if (nw > 1) {
      if ((lane & 15) == 0) scratch[turn][upper][threadIdx.x / 32] = m;
      grp.sync();
      m = sum_over(scratch[turn][upper][lane & (nw - 1)], nw);
      turn ^= 1;
    }
    __syncwarp();
    R.taken(row, r == 0);
    m = fmaf(m, inv, eps);
    const float left = __shfl_sync(0xffffffffu, m, 0), rstd = rsqrtf(fmaf(-left, left, __shfl_sync(0xffffffffu, m, 16)));
    const float2 by = both(rstd), shift = both(-left * rstd);
#pragma unroll
    for (int i = 0; i < EPT / 2 / CN; ++i) {
#pragma unroll
      for (int c = 0; c < CN; ++c) v[i][c] = fma2(fma2(v[i][c], by, shift), ga[i * CN + c], be[i * CN + c]);
      put<T, WHOLE>(y + row * a.d, r, a.tpr, a.d, i, v[i]);
    }
    if (r == 0) {
      if (a.mean) a.mean[row] = near + left;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// A row is read from the ring twice, for the sums and for dx, and the sums of
// the next row are formed before dx of this one: the reduction's shuffles and
// barrier run under arithmetic that does not wait for them.  (32768 x 4096 bf16:
// 168 us; one row after the other 197.  The forward, bound by instruction issue,
// lost by it when it had two reductions a row: 104 us, not 92.5.)
template <typename T, bool WHOLE, bool RES>
__global__ void __launch_bounds__(BWD_NT, 1) norm_bwd_kernel(const NormArgs a) {
  constexpr int VN = WHOLE ? Vec<T>::N : 1, CN = Chunk<T, WHOLE>::N / 2, NBUF = RES ? 3 : 2;
  __shared__ float4 scratch[2 * 16];
  __shared__ uint64_t bars[MAX_GROUPS * RING];
  const Group<true> grp(a.tpr);
  const int r = grp.r;
  Rows<T, WHOLE, NBUF> R = begin_rows<T, WHOLE, NBUF>(a, bars, r);
  T* dx = static_cast<T*>(a.out);
  const float inv = 1.f / (float)a.d;
  float2 ga[EPT / 2], dg[EPT / 2], db[EPT / 2];
  take_weights<VN>(a.gamma, r, a.tpr, a.d, ga);
#pragma unroll
  for (int c = 0; c < EPT / 2; ++c) dg[c] = db[c] = both(0.f);
  const T *x = static_cast<const T*>(a.x), *dy = static_cast<const T*>(a.dy), *res = static_cast<const T*>(a.dres);

  // the warp's sums of row `row`, and its part of dgamma and dbeta
  auto sums = [&](int64_t row, float2 stat) {
    const Span sp = row_span<T, WHOLE>(row, a.rows, a.d);
    const float2 by = both(stat.y), from = both(-stat.x);
    R.wait(a.err);
    float2 sv = both(0.f), sn = both(0.f);
#pragma unroll
    for (int i = 0; i < EPT / 2 / CN; ++i) {
      float2 n[CN], v[CN];
      take<T, WHOLE>(R.place(0), sp, x, r, a.tpr, a.d, i, n);
      take<T, WHOLE>(R.place(1), sp, dy, r, a.tpr, a.d, i, v);
#pragma unroll
      for (int c = 0; c < CN; ++c) {  // past the row's end dy and gamma are 0
        const int at = i * CN + c;
        n[c] = mul2(add2(n[c], from), by);
        dg[at] = fma2(v[c], n[c], dg[at]);
        db[at] = add2(db[at], v[c]);
        v[c] = mul2(v[c], ga[at]);
        sv = add2(sv, v[c]);
        sn = fma2(v[c], n[c], sn);
      }
    }
    return make_float2(warp_sum(sv.x + sv.y), warp_sum(sn.x + sn.y));
  };

  // mean and rstd of a row, loaded two rows ahead of their use
  auto stats = [&](int64_t row) {
    return row < a.rows ? make_float2(__ldg(a.mean_in + row), __ldg(a.rstd_in + row)) : make_float2(0.f, 0.f);
  };
  float2 stat = stats(R.first), stat1 = stats(R.first + R.step);
  int turn = 0, before = 0;  // before: the place of the row whose dx comes next
  float2 own = make_float2(0.f, 0.f);
  if (R.first < a.rows) {
    own = sums(R.first, stat);
    grp.give(make_float4(own.x, own.y, 0.f, 0.f), scratch, 0);
  }
#pragma unroll 1
  for (int64_t row = R.first; row < a.rows; row += R.step, turn ^= 1) {
    const float2 stat2 = stats(row + 2 * R.step);
    grp.sync();  // the row's sums are there, and everyone is done with the row before it
    if (r == 0 && row != R.first) R.start(row + (R.ring - 1) * R.step, before == 0 ? R.ring - 1 : before - 1);
    float4 w = grp.get(scratch, turn);
    const bool alone = grp.warps == 1;
    const float m1 = alone ? own.x : sum_over(w.x, grp.warps), m2 = alone ? own.y : sum_over(w.y, grp.warps);
    R.next();
    if (row + R.step < a.rows) {
      own = sums(row + R.step, stat1);
      grp.give(make_float4(own.x, own.y, 0.f, 0.f), scratch, turn ^ 1);
    }
    const Span sp = row_span<T, WHOLE>(row, a.rows, a.d);
    const float2 by = both(stat.y), from = both(-stat.x);
    const float2 k1 = both(-m1 * inv), k2 = both(-m2 * inv);
#pragma unroll
    for (int i = 0; i < EPT / 2 / CN; ++i) {
      float2 n[CN], v[CN], o[CN];
      take<T, WHOLE>(R.place_at(before, 0), sp, x, r, a.tpr, a.d, i, n);
      take<T, WHOLE>(R.place_at(before, 1), sp, dy, r, a.tpr, a.d, i, v);
      if (RES) take<T, WHOLE>(R.place_at(before, 2), sp, res, r, a.tpr, a.d, i, o);
#pragma unroll
      for (int c = 0; c < CN; ++c) {
        n[c] = mul2(add2(n[c], from), by);
        const float2 t = fma2(n[c], k2, fma2(v[c], ga[i * CN + c], k1));
        o[c] = RES ? fma2(t, by, o[c]) : mul2(t, by);
      }
      put<T, WHOLE>(dx + row * a.d, r, a.tpr, a.d, i, o);
    }
    before = R.at;
    stat = stat1;
    stat1 = stat2;
  }
  __syncthreads();
  // the CTA's sums, over its groups in order, are one row pair of the partials
  const int groups = blockDim.x / a.tpr;
  float* out = a.partial + (size_t)blockIdx.x * 2 * a.d;
  float* mine = groups == 1 ? out : reinterpret_cast<float*>(norm_smem) + (size_t)grp.g * 2 * a.d;
#pragma unroll
  for (int c = 0; c < EPT; ++c) {
    const int col = column<VN>(r, a.tpr, c);
    if (in_row<VN>(r, a.tpr, c, a.d)) {
      mine[col] = c & 1 ? dg[c / 2].y : dg[c / 2].x;
      mine[a.d + col] = c & 1 ? db[c / 2].y : db[c / 2].x;
    }
  }
  if (groups == 1) return;
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(norm_smem);
  for (int i = threadIdx.x; i < 2 * a.d; i += blockDim.x) {
    float u = 0.f;
#pragma unroll 4
    for (int g = 0; g < groups; ++g) u += all[(size_t)g * 2 * a.d + i];
    out[i] = u;
  }
}

// dgamma and dbeta from the partials [parts][2][d], added in part order within
// RED_STRIPS interleaved strips and then over the strips.
__global__ void __launch_bounds__(RED_COLS * RED_STRIPS) norm_bwd_reduce_kernel(const NormArgs a) {
  pdl_enter();
  __shared__ float tile[RED_STRIPS][RED_COLS + 1];
  const int c = threadIdx.x % RED_COLS, strip = threadIdx.x / RED_COLS;
  const int col = blockIdx.x * RED_COLS + c;  // of the 2 d columns
  float s = 0.f;
  if (col < 2 * a.d) {
#pragma unroll 1
    for (int p = strip; p < a.parts; p += 8 * RED_STRIPS) {  // eight loads at once
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = p + j * RED_STRIPS < a.parts ? a.partial[(size_t)(p + j * RED_STRIPS) * 2 * a.d + col] : 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s += v[j];
    }
  }
  tile[strip][c] = s;
  __syncthreads();
  if (strip == 0 && col < 2 * a.d) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < RED_STRIPS; ++i) s += tile[i][c];
    float* dst = col < a.d ? a.dgamma + col : a.dbeta + (col - a.d);
    *dst = a.accumulate ? *dst + s : s;
  }
}

// ---- rows of more than MAX_TPR * EPT elements: one CTA a row, walked in a
// loop, again from cache for each pass; dgamma and dbeta in a pass of their own.
// The forward takes distances from the rounded mean and what is left of their
// sum off again. ----
__device__ __forceinline__ float2 cta_sum(float2 s, float4* scratch, int& turn) {
  const Group<false> all(WIDE_NT);
  all.give(make_float4(warp_sum(s.x), warp_sum(s.y), 0.f, 0.f), scratch, turn);
  all.sync();
  const float4 w = all.get(scratch, turn);
  turn ^= 1;
  return make_float2(sum_over(w.x, WIDE_NT / 32), sum_over(w.y, WIDE_NT / 32));
}

// VN elements: a 16-byte vector, or one
template <typename T, int VN>
__device__ __forceinline__ void ld_n(const T* p, float (&v)[VN]) {
  if constexpr (VN == 1) v[0] = to_f32(*p);
  else unpack(*reinterpret_cast<const uint4*>(p), v);
}
template <int VN>
__device__ __forceinline__ void ld_w(const float* p, float (&v)[VN]) {  // of the weights
  if constexpr (VN == 1) {
    v[0] = __ldg(p);
  } else {
#pragma unroll
    for (int j = 0; j < VN; j += 4) {
      const float4 w = __ldg(reinterpret_cast<const float4*>(p + j));
      v[j] = w.x;
      v[j + 1] = w.y;
      v[j + 2] = w.z;
      v[j + 3] = w.w;
    }
  }
}
template <typename T, int VN>
__device__ __forceinline__ void st_n(T* p, const float (&v)[VN]) {
  if constexpr (VN == 1) *p = from_f32<T>(v[0]);
  else stg16(p, pack(v));
}

template <typename T, int VN>
__global__ void __launch_bounds__(WIDE_NT) norm_fwd_wide_kernel(const NormArgs a) {
  pdl_enter();
  __shared__ float4 scratch[2 * WIDE_NT / 32];
  int turn = 0;
  const float inv = 1.f / (float)a.d;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* xr = static_cast<const T*>(a.x) + row * a.d;
    T* yr = static_cast<T*>(a.out) + row * a.d;
    float s = 0.f;
#pragma unroll 4
    for (int i = threadIdx.x * VN; i < a.d; i += WIDE_NT * VN) {
      float v[VN];
      ld_n<T, VN>(xr + i, v);
#pragma unroll
      for (int j = 0; j < VN; ++j) s += v[j];
    }
    const float near = cta_sum(make_float2(s, 0.f), scratch, turn).x * inv;
    float2 q = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int i = threadIdx.x * VN; i < a.d; i += WIDE_NT * VN) {
      float v[VN];
      ld_n<T, VN>(xr + i, v);
#pragma unroll
      for (int j = 0; j < VN; ++j) {
        q.x += v[j] - near;
        q.y = fmaf(v[j] - near, v[j] - near, q.y);
      }
    }
    q = cta_sum(q, scratch, turn);
    const float left = q.x * inv, rstd = rsqrtf(fmaf(q.y, inv, a.eps) - left * left), mean = near + left;
#pragma unroll 2
    for (int i = threadIdx.x * VN; i < a.d; i += WIDE_NT * VN) {
      float v[VN], g[VN], b[VN];
      ld_n<T, VN>(xr + i, v);
      ld_w<VN>(a.gamma + i, g);
      ld_w<VN>(a.beta + i, b);
#pragma unroll
      for (int j = 0; j < VN; ++j) v[j] = fmaf(((v[j] - near) - left) * rstd, g[j], b[j]);
      st_n<T, VN>(yr + i, v);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

template <typename T, int VN>
__global__ void __launch_bounds__(WIDE_NT) norm_bwd_wide_kernel(const NormArgs a) {
  pdl_enter();
  __shared__ float4 scratch[2 * WIDE_NT / 32];
  int turn = 0;
  const float inv = 1.f / (float)a.d;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float mean = a.mean_in[row], rstd = a.rstd_in[row];
    const T* x = static_cast<const T*>(a.x) + row * a.d;
    const T* dy = static_cast<const T*>(a.dy) + row * a.d;
    const T* res = static_cast<const T*>(a.dres) + (a.dres ? row * a.d : 0);
    T* dx = static_cast<T*>(a.out) + row * a.d;
    float2 s = make_float2(0.f, 0.f);
#pragma unroll 2
    for (int i = threadIdx.x * VN; i < a.d; i += WIDE_NT * VN) {
      float n[VN], v[VN], g[VN];
      ld_n<T, VN>(x + i, n);
      ld_n<T, VN>(dy + i, v);
      ld_w<VN>(a.gamma + i, g);
#pragma unroll
      for (int j = 0; j < VN; ++j) {
        v[j] *= g[j];
        s.x += v[j];
        s.y = fmaf(v[j], (n[j] - mean) * rstd, s.y);
      }
    }
    s = cta_sum(s, scratch, turn);
    const float m1 = s.x * inv, m2 = s.y * inv;
#pragma unroll 2
    for (int i = threadIdx.x * VN; i < a.d; i += WIDE_NT * VN) {
      float n[VN], v[VN], o[VN], g[VN];
      ld_n<T, VN>(x + i, n);
      ld_n<T, VN>(dy + i, v);
      ld_w<VN>(a.gamma + i, g);
      if (a.dres) ld_n<T, VN>(res + i, o);
#pragma unroll
      for (int j = 0; j < VN; ++j) {
        const float t = (fmaf(v[j], g[j], -m1) - (n[j] - mean) * rstd * m2) * rstd;
        o[j] = a.dres ? o[j] + t : t;
      }
      st_n<T, VN>(dx + i, o);
    }
  }
}

// dgamma and dbeta of VN columns a thread over the rows blockIdx.y, + gridDim.y,
// ...; it runs before dx is written, which may be x or dy
constexpr int COL_NT = 128;
template <typename T, int VN>
__global__ void __launch_bounds__(COL_NT) norm_bwd_columns_kernel(const NormArgs a) {
  pdl_enter();
  const int i = (blockIdx.x * COL_NT + threadIdx.x) * VN;
  if (i >= a.d) return;
  float g[VN], b[VN];
#pragma unroll
  for (int j = 0; j < VN; ++j) g[j] = b[j] = 0.f;
#pragma unroll 4
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float mean = __ldg(a.mean_in + row), rstd = __ldg(a.rstd_in + row);
    float n[VN], v[VN];
    ld_n<T, VN>(static_cast<const T*>(a.x) + row * a.d + i, n);
    ld_n<T, VN>(static_cast<const T*>(a.dy) + row * a.d + i, v);
#pragma unroll
    for (int j = 0; j < VN; ++j) {
      g[j] = fmaf(v[j], (n[j] - mean) * rstd, g[j]);
      b[j] += v[j];
    }
  }
  float* out = a.partial + (size_t)blockIdx.y * 2 * a.d;
#pragma unroll
  for (int j = 0; j < VN; ++j) {
    out[i + j] = g[j];
    out[a.d + i + j] = b[j];
  }
}

bool wide(int d) { return d > MAX_TPR * EPT; }

// Threads that share a row: as few as hold it, a warp at least.
int threads_per_row(int d) {
  int tpr = 32;
  while (tpr * EPT < d) tpr *= 2;
  return tpr;
}
// Sizes of a launch whose kernel reads `bufs` tensors.  Forward: CTAs of one
// group of threads, or of four warps with rows of their own, as many as the
// registers allow.  Backward: one CTA an SM.  The rings take what shared memory
// that leaves, up to RING rows.
struct Grid {
  int threads, ctas;
  size_t smem;
};
Grid norm_grid(int64_t rows, int d, int es, int bufs, NormArgs* a) {
  const bool bwd = bufs > 1;
  const int tpr = threads_per_row(d), slot = (d * es + 15) / 16 * 16 + (d * es % 16 ? 16 : 0);
  const int groups = bwd ? BWD_NT / tpr : (tpr == 32 ? 4 : 1);
  int per = bwd ? 1 : 65536 / (tpr * groups * FWD_REGS);
  const size_t place = (size_t)bufs * slot;
  while (per > 1 && per * 2 * (groups * place + 1024) > SMEM_SM) --per;
  int ring = (int)((SMEM_SM / per - 1024) / (groups * place));
  ring = ring > RING ? RING : (ring < 2 ? 2 : ring);
  Grid g;
  g.threads = tpr * groups;
  g.smem = ring * groups * place;
  const size_t sums = groups > 1 ? (size_t)groups * 2 * d * 4 : 0;  // the backward's groups' sums take the ring's place
  if (bwd && g.smem < sums) g.smem = sums;
  const int64_t need = bwd ? rows : (rows + groups - 1) / groups, most = (int64_t)sm_count() * per;
  g.ctas = (int)(need < most ? need : most);
  if (a != nullptr) {
    a->tpr = tpr;
    a->slot = slot;
    a->ring = ring;
  }
  return g;
}

template <typename K>
cudaError_t launch_rows(K kernel, const Grid& g, const NormArgs& a, bool* attr_done, cudaStream_t st) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  if (!attr_done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_SM);
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  return launch_pdl(kernel, dim3(g.ctas), dim3(g.threads), g.smem, st, a);
}

template <typename T, bool WHOLE>
cudaError_t fwd_w(NormArgs& a, cudaStream_t st) {
  static bool done[64] = {false};
  const Grid g = norm_grid(a.rows, a.d, sizeof(T), 1, &a);
  return launch_rows(norm_fwd_kernel<T, WHOLE>, g, a, done, st);
}
template <typename T, bool WHOLE>
cudaError_t bwd_w(NormArgs& a, cudaStream_t st) {
  static bool done[2][64] = {{false}};
  const Grid g = norm_grid(a.rows, a.d, sizeof(T), a.dres ? 3 : 2, &a);
  a.parts = g.ctas;
  return a.dres ? launch_rows(norm_bwd_kernel<T, WHOLE, true>, g, a, done[1], st)
                : launch_rows(norm_bwd_kernel<T, WHOLE, false>, g, a, done[0], st);
}
template <typename T, int VN>
cudaError_t fwd_wide(const NormArgs& a, cudaStream_t st) {
  const int64_t most = (int64_t)sm_count() * 4;
  return launch_pdl(norm_fwd_wide_kernel<T, VN>, dim3((unsigned)(a.rows < most ? a.rows : most)), dim3(WIDE_NT), 0, st, a);
}
// Row slices of the columns' sums: about 16 CTAs an SM
int wide_slices(int64_t rows, int d) {
  const int64_t tiles = (d + COL_NT * 8 - 1) / (COL_NT * 8), most = ((int64_t)sm_count() * 16 + tiles - 1) / tiles;
  return (int)(rows < most ? rows : most);
}
template <typename T, int VN>
cudaError_t bwd_wide(NormArgs& a, cudaStream_t st) {
  a.parts = wide_slices(a.rows, a.d);
  cudaError_t e = launch_pdl(norm_bwd_columns_kernel<T, VN>, dim3((a.d + COL_NT * VN - 1) / (COL_NT * VN), a.parts),
                             dim3(COL_NT), 0, st, a);
  if (e != cudaSuccess) return e;
  const int64_t most = (int64_t)sm_count() * 4;
  return launch_pdl(norm_bwd_wide_kernel<T, VN>, dim3((unsigned)(a.rows < most ? a.rows : most)), dim3(WIDE_NT), 0, st, a);
}
bool vectors(const float* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
template <typename T>
cudaError_t fwd_t(NormArgs& a, cudaStream_t st) {
  const bool whole = a.d % Vec<T>::N == 0;
  if (wide(a.d)) return whole && vectors(a.gamma) && vectors(a.beta) ? fwd_wide<T, Vec<T>::N>(a, st) : fwd_wide<T, 1>(a, st);
  return whole ? fwd_w<T, true>(a, st) : fwd_w<T, false>(a, st);
}
template <typename T>
cudaError_t bwd_t(NormArgs& a, cudaStream_t st) {
  const bool whole = a.d % Vec<T>::N == 0;
  if (wide(a.d)) return whole && vectors(a.gamma) ? bwd_wide<T, Vec<T>::N>(a, st) : bwd_wide<T, 1>(a, st);
  return whole ? bwd_w<T, true>(a, st) : bwd_w<T, false>(a, st);
}

}  // namespace

cudaError_t launch_norm_fwd(int64_t rows, int d, bool bf16, const void* x, const float* gamma, const float* beta,
                            float eps, void* y, float* mean, float* rstd, uint32_t* err, cudaStream_t st) {
  NormArgs a{};
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.eps = eps;
  a.out = y;
  a.mean = mean;
  a.rstd = rstd;
  a.rows = rows;
  a.d = d;
  a.err = err;
  LaunchScope ls(KK_NORM_FWD, st);
  return bf16 ? fwd_t<__nv_bfloat16>(a, st) : fwd_t<float>(a, st);
}

size_t norm_ws_bytes(int64_t rows, int d) {
  const int ctas = wide(d) ? wide_slices(rows, d) : norm_grid(rows, d, 2, 2, nullptr).ctas;
  return (size_t)ctas * 2 * d * 4;
}

cudaError_t launch_norm_bwd(int64_t rows, int d, bool bf16, const void* x, const void* dy, const float* gamma,
                            const float* mean, const float* rstd, const void* dres, void* dx, float* dgamma,
                            float* dbeta, int accumulate, void* ws, uint32_t* err, cudaStream_t st) {
  NormArgs a{};
  a.x = x;
  a.dy = dy;
  a.dres = dres;
  a.gamma = gamma;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.out = dx;
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.partial = static_cast<float*>(ws);
  a.rows = rows;
  a.d = d;
  a.accumulate = accumulate;
  a.err = err;
  {
    LaunchScope ls(KK_NORM_BWD, st);
    const cudaError_t e = bf16 ? bwd_t<__nv_bfloat16>(a, st) : bwd_t<float>(a, st);
    if (e != cudaSuccess) return e;
  }
  LaunchScope ls(KK_NORM_BWD_REDUCE, st);
  return launch_pdl(norm_bwd_reduce_kernel, dim3((2 * d + RED_COLS - 1) / RED_COLS), dim3(RED_COLS * RED_STRIPS), 0,
                    st, a);
}

}  // namespace moe
