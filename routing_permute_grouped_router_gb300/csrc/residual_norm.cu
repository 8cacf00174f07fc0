// The residual path between two blocks with the norms on either side of it.
//
//   u   = y ry gamma_post,  out = rs x + bs row_gate gate u,  h = out ro gamma_next
//
// and its backward; formulas are in moe.h.
//
// Both passes are bound by HBM: the forward reads x and y and writes out and h,
// the backward reads dh, out, dout and y and writes dx and dy.  Up to 512 threads
// share a row, 16 elements each, while copies bring the next rows into a ring in
// shared memory.  A row has two reductions, of which the second needs the first:
// the second of a row and the first of the row after it share one barrier.
// Threads keep their columns' weights and, in the backward, the columns' sums in
// registers over all rows of the CTA; a second kernel adds the CTAs' sums in
// CTA order, so results do not depend on timing.  Statistics and sums are fp32.
//
// Rows that the ring has no room for (over 8192 elements; in the backward, whose
// weights take up to 64 KB of shared memory beside it, float32 rows over 5152 where
// dh, out, dout and y are all there, and over 6868 of three of them) have one CTA
// each and are walked in a loop, again from cache for each pass.  There the columns' sums are taken in a
// pass of their own before anything is written (dx and dy may be dh or dout).
#include <algorithm>
#include <atomic>

#include "row_ring.cuh"
#include "step.h"

namespace moe {
namespace {

// A thread's registers in the forward: three CTAs of 256 fit an SM with 80, two
// with 96.  (32768 x 4096 bf16 178 us with 80, 169 with 96; 16384 x 8192 197 and
// 170; 32768 x 2048 97 and 101; 16384 x 4096 float32 175 and 184.)
constexpr int fwd_regs(int es) { return es == 2 ? 96 : 80; }
constexpr int BWD_NT = 512;    // most threads of the backward's CTAs, one an SM
constexpr int MAX_GROUPS = BWD_NT / 32;
constexpr int BWD_SMEM = 230400;  // a CTA's dynamic shared memory there: 227 KB less its static part
constexpr int WIDE_NT = 512;   // threads of a wide row's CTA
constexpr int COL_NT = 128;
constexpr int RED_COLS = 32, RED_STRIPS = 32;

struct JoinK {
  const void *x, *y, *dh, *dout;
  void *out, *h, *dx, *dy;
  const float *gamma_post, *gamma_next, *gate, *row_gate;
  float *rstd_post, *rstd_next;
  float *dgamma_post, *dgamma_next, *dgate, *drow_gate;
  float* mean_vn;  // [rows]: sum(v n) / d
  float* partial;  // [parts][2][d]: sums of dh n, and of row_gate D m
  int64_t rows;
  int d, parts, accumulate;
  int tpr, slot, ring;  // threads that share a row, bytes of a tensor's row in the ring, places
  float rs, bs, eps;
  uint32_t* err;
};

// ------------------------------ rows in the ring --------------------------- //
// A group of tpr threads, its rows (first, first + step, ...) of up to four
// tensors, and its ring.  The group's first thread starts the copies.
template <typename T, bool WHOLE>
struct JoinRows {
  const void *t0, *t1, *t2, *t3;  // null where there is none; the others follow one another in a place
  int nbuf;
  char* base;
  uint64_t* bars;
  int64_t first, step, rows;
  int d, slot, ring;
  int at = 0;          // the place of the row in work
  uint32_t phase = 0;  // and its barrier's phase
  __device__ __forceinline__ JoinRows(const void* a, const void* b, const void* c, const void* e)
      : t0(a), t1(b), t2(c), t3(e), nbuf((a != nullptr) + (b != nullptr) + (c != nullptr) + (e != nullptr)) {}
  __device__ __forceinline__ void start(int64_t row, int p) const {
    if (row >= rows) return;
    const Span sp = row_span<T, WHOLE>(row, rows, d);
    const uint32_t bar = sm_addr(bars + p);
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(sp.bytes * nbuf) : "memory");
    if (sp.bytes <= 0) return;
    uint32_t to = sm_addr(place(p, sp));
    auto copy = [&](const void* t) {
      if (t == nullptr) return;
      copy_row(to, static_cast<const char*>(t) + sp.at, sp.bytes, bar);
      to += slot;
    };
    copy(t0);
    copy(t1);
    copy(t2);
    copy(t3);
  }
  __device__ __forceinline__ void wait(uint32_t* err) const {
    if (!ring_ready(sm_addr(bars + at), phase)) ring_wait(sm_addr(bars + at), phase, err);
  }
  // of the first tensor's row: as far into a 128-byte line as it is in memory
  __device__ __forceinline__ char* place(int p, const Span& sp) const {
    return base + (size_t)(p * nbuf) * slot + (WHOLE ? 0 : (int)(sp.at & 112));
  }
  __device__ __forceinline__ void next() {
    if (++at == ring) {
      at = 0;
      phase ^= 1u;
    }
  }
};

extern __shared__ __align__(128) char join_smem[];

// The ends of rows that are no whole units, in functions of their own: they are
// few, and as part of the kernels their registers and branches slow every row
// (32768 x 1007 bf16 backward: 143 us).
//
// Zeros for the elements of other rows in a unit of nbuf tensors in shared
// memory, `slot` apart; c is the unit's first element in the row of d.
template <int ES>
__device__ __noinline__ void trim_unit(uint32_t at, int slot, int nbuf, int c, int d) {
  constexpr int VN = 16 / ES;
  const int lo = c < 0 ? -c * 8 * ES : 0, hi = c + VN > d ? (d - c) * 8 * ES : 128;  // the row's bits
  uint64_t m0 = lo < 64 ? ~0ull << lo : 0ull, m1 = lo < 64 ? ~0ull : ~0ull << (lo - 64);
  if (hi <= 64) m1 = 0ull;
  else if (hi < 128) m1 &= (1ull << (hi - 64)) - 1;
  if (hi < 64) m0 &= (1ull << hi) - 1;
  for (int b = 0; b < nbuf; ++b, at += slot)
    asm volatile(
        "{\n\t.reg .b64 x, y;\n\tld.shared.v2.b64 {x, y}, [%0];\n\tand.b64 x, x, %1;\n\tand.b64 y, y, %2;\n\t"
        "st.shared.v2.b64 [%0], {x, y};\n\t}" ::"r"(at), "l"(m0), "l"(m1)
        : "memory");
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // a copy will write there again
}
// The same for a unit that the copy has cut off at the tensors' end: from memory, `byte` bytes into the tensors.
template <typename T>
__device__ __noinline__ void load_cut(const void* t0, const void* t1, const void* t2, const void* t3, int64_t byte,
                                      uint32_t at, int slot, int c, int d) {
  const void* t[4] = {t0, t1, t2, t3};
#pragma unroll
  for (int b = 0; b < 4; ++b) {
    if (t[b] == nullptr) continue;
    const T* p = reinterpret_cast<const T*>(static_cast<const char*>(t[b]) + byte);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j)
      if (c + j >= 0 && c + j < d) {
        if constexpr (sizeof(T) == 2) w[j / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(p + j) << (j % 2 * 16);
        else w[j] = *reinterpret_cast<const uint32_t*>(p + j);
      }
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
    at += slot;
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// The row's elements of a unit to memory.
template <typename T>
__device__ __noinline__ void store_edge(T* to, uint4 u, int c, int d) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < Vec<T>::N; ++j)
    if (c + j >= 0 && c + j < d) {
      if constexpr (sizeof(T) == 2) *reinterpret_cast<uint16_t*>(to + j) = (uint16_t)(w[j / 2] >> (j % 2 * 16));
      else *reinterpret_cast<uint32_t*>(to + j) = w[j];
    }
}

// A thread's chunks of rows in the ring: 16-byte units of the tensor, of which
// the first and the last may hold elements of the rows around.  A CTA's rows are
// a multiple of VN apart, so they all begin as many elements, `skip`, into their
// first unit, and a thread has the same columns in each (rows that are whole
// units, WHOLE, have no skip).  What is past the row's end is read from 16 bytes
// of zeros: a load a chunk and no branch.
template <typename T, bool WHOLE>
struct Mine {
  static constexpr int VN = Vec<T>::N, CN = VN / 2, NC = EPT / VN;
  int r, tpr, d, slot, skip;
  uint32_t zeros, off[NC];
  bool in[NC], edge[NC];  // the chunk has elements of the row; and others
  __device__ __forceinline__ Mine(const JoinK& a, int r_, uint32_t zeros_)
      : r(r_), tpr(a.tpr), d(a.d), slot(a.slot), skip(WHOLE ? 0 : (int)((int64_t)blockIdx.x * a.d % VN)), zeros(zeros_) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      off[i] = (r + i * tpr) * 16;
      in[i] = column(i) < d;
      edge[i] = !WHOLE && in[i] && (column(i) < 0 || column(i) + VN > d);
    }
  }
  // of the chunk's first element; the elements of the row are 0 to d - 1
  __device__ __forceinline__ int column(int i) const { return (r + i * tpr) * VN - skip; }
  __device__ __forceinline__ void get(const char* at, int b, int i, float2 (&v)[CN]) const {
    float w[VN];
    unpack(lds(in[i] ? sm_addr(at) + b * slot + off[i] : zeros), w);
#pragma unroll
    for (int c = 0; c < CN; ++c) v[c] = make_float2(w[2 * c], w[2 * c + 1]);
  }
  // Once a row is there: the thread's own units of it get zeros where they have
  // elements of other rows, and what a copy has cut off at the tensor's end.
  __device__ __forceinline__ void patch(const JoinRows<T, WHOLE>& R, int64_t row) const {
    if constexpr (!WHOLE) {
      const Span sp = row_span<T, WHOLE>(row, R.rows, d);
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (edge[i]) {
          const uint32_t at = sm_addr(R.place(R.at, sp)) + off[i];
          if ((int)off[i] + 16 > sp.bytes) {
            load_cut<T>(R.t0, R.t1, R.t2, R.t3, sp.at + off[i], at, slot, column(i), d);
          } else {
            trim_unit<sizeof(T)>(at, slot, R.nbuf, column(i), d);
          }
        }
    }
  }
  __device__ __forceinline__ void set(void* tensor, const Span& sp, int i, const float2 (&v)[CN]) const {
    float w[VN];
#pragma unroll
    for (int c = 0; c < CN; ++c) {
      w[2 * c] = v[c].x;
      w[2 * c + 1] = v[c].y;
    }
    char* to = static_cast<char*>(tensor) + sp.at + off[i];
    const uint4 u = pack(w);
    if (!WHOLE && edge[i]) store_edge<T>(reinterpret_cast<T*>(to), u, column(i), d);
    else if (in[i]) stg16(to, u);
  }
  // the columns' weights times `by`, `by` where there are none; 0 outside the row
  __device__ __forceinline__ float weight(const float* p, const float* p2, float by, int col) const {
    return col < 0 || col >= d ? 0.f : by * (p ? __ldg(p + col) : 1.f) * (p2 ? __ldg(p2 + col) : 1.f);
  }
  __device__ __forceinline__ void take_weights(const float* p, const float* p2, float by, float2 (&v)[EPT / 2]) const {
#pragma unroll
    for (int c = 0; c < EPT; ++c) (c & 1 ? v[c / 2].y : v[c / 2].x) = weight(p, p2, by, column(c / VN) + c % VN);
  }
  // the same in shared memory, 16 bytes of a chunk at a time so that neighbouring lanes read neighbouring ones
  __device__ __forceinline__ void keep_weights(float* w, const float* p, const float* p2, float by) const {
    for (int c = threadIdx.x; c < EPT * tpr; c += blockDim.x) {
      const int q = c / VN, j = c % VN;
      w[(j / 4 * NC * tpr + q) * 4 + j % 4] = weight(p, p2, by, c - skip);
    }
  }
  __device__ __forceinline__ void weights(uint32_t w, int i, float2 (&v)[CN]) const {
#pragma unroll
    for (int j = 0; j < CN / 2; ++j) {
      const uint4 u = lds(w + j * (NC * tpr * 16) + off[i]);
      v[2 * j] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
      v[2 * j + 1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
  }
  __device__ __forceinline__ static uint4 lds(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
  }
};

// The barriers, and the first rows on their way.
template <typename T, bool WHOLE>
__device__ __forceinline__ void begin(JoinRows<T, WHOLE>& R, const JoinK& a, uint64_t* bars, int r, int before = 0) {
  const int groups = blockDim.x / a.tpr, g = threadIdx.x / a.tpr;  // rows go to all CTAs before a second group of any
  R.base = join_smem + before + (size_t)g * a.ring * R.nbuf * a.slot;
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
}

// BRANCH: there is a y; FOLLOWING: there is an h.  (As run-time flags they cost
// branches in every chunk of a row: the backward 371 us at 32768 x 4096 bf16, not 347.)
template <typename T, bool WHOLE, bool BRANCH, bool FOLLOWING>
__global__ void __maxnreg__(fwd_regs(sizeof(T))) join_fwd_kernel(const JoinK a) {
  constexpr int CN = Mine<T, WHOLE>::CN;
  __shared__ float scratch[2][2][16];
  __shared__ uint64_t bars[MAX_GROUPS * RING];
  __shared__ __align__(16) uint4 zeros;
  if (threadIdx.x == 0) zeros = make_uint4(0, 0, 0, 0);
  int turn = 0;
  const Group<false> grp(a.tpr);
  const int r = grp.r, nw = grp.warps, lane = threadIdx.x % 32;
  const bool upper = lane >= 16, post = BRANCH && a.gamma_post != nullptr;
  JoinRows<T, WHOLE> R(a.x, BRANCH ? a.y : nullptr, nullptr, nullptr);
  constexpr int bx = 0, by_ = 1;
  begin<T, WHOLE>(R, a, bars, r);
  const Mine<T, WHOLE> mine(a, r, sm_addr(&zeros));
  const float inv = 1.f / (float)a.d;
  float2 ga[EPT / 2], gn[EPT / 2];
  mine.take_weights(a.gamma_post, a.gate, a.bs, ga);
  mine.take_weights(a.gamma_next, nullptr, 1.f, gn);
  // both sums over the group, the first in the lower half of the lanes
  auto sums = [&](float u, float v) {
    float m = half_sums(u, v, upper);
    if (nw > 1) {
      if ((lane & 15) == 0) scratch[turn][upper][threadIdx.x / 32] = m;
      grp.sync();
      m = sum_over(scratch[turn][upper][lane & (nw - 1)], nw);
      turn ^= 1;
    }
    __syncwarp();
    return m;
  };
  // the thread's part of sum(y^2) of the row at place R.at
  auto squares = [&](int64_t row) {
    const Span sp = row_span<T, WHOLE>(row, a.rows, a.d);
    float2 s = both(0.f);
#pragma unroll
    for (int i = 0; i < EPT / 2 / CN; ++i) {
      float2 v[CN];
      mine.get(R.place(R.at, sp), by_, i, v);
#pragma unroll
      for (int c = 0; c < CN; ++c) s = fma2(v[c], v[c], s);
    }
    return s.x + s.y;
  };
  float first = 0.f;  // the mean of y^2 of the row in work
  if (R.first < a.rows) {
    R.wait(a.err);
    mine.patch(R, R.first);
    if (post) first = __shfl_sync(0xffffffffu, sums(squares(R.first), 0.f), 0) * inv;
  }
#pragma unroll 1
  for (int64_t row = R.first; row < a.rows; row += R.step) {
    const Span sp = row_span<T, WHOLE>(row, a.rows, a.d);
    const float ry = post ? rsqrtf(first + a.eps) : 1.f;
    const float2 by = both(ry * (a.row_gate ? __ldg(a.row_gate + row) : 1.f)), rs = both(a.rs);
    float2 o[EPT / 2 / CN][CN], s2 = both(0.f);
#pragma unroll
    for (int i = 0; i < EPT / 2 / CN; ++i) {
      mine.get(R.place(R.at, sp), bx, i, o[i]);
      float2 v[CN];
      if (BRANCH) mine.get(R.place(R.at, sp), by_, i, v);
#pragma unroll
      for (int c = 0; c < CN; ++c) {
        o[i][c] = mul2(o[i][c], rs);
        if (BRANCH) o[i][c] = fma2(mul2(v[c], by), ga[i * CN + c], o[i][c]);
        s2 = fma2(o[i][c], o[i][c], s2);
      }
    }
    const int place = R.at;
    float s1 = 0.f;
    R.next();
    if (row + R.step < a.rows) {
      R.wait(a.err);
      mine.patch(R, row + R.step);
      if (post) s1 = squares(row + R.step);
    }
    const float m = sums(s2.x + s2.y, s1) * inv;
    if (r == 0) R.start(row + R.ring * R.step, place);  // everyone has read the row
    const float ro = rsqrtf(__shfl_sync(0xffffffffu, m, 0) + a.eps);
    first = __shfl_sync(0xffffffffu, m, 16);
    const float2 ro2 = both(ro);
#pragma unroll
    for (int i = 0; i < EPT / 2 / CN; ++i) {
      if (a.out) mine.set(a.out, sp, i, o[i]);
      if (FOLLOWING) {
#pragma unroll
        for (int c = 0; c < CN; ++c) o[i][c] = mul2(mul2(o[i][c], ro2), gn[i * CN + c]);
        mine.set(a.h, sp, i, o[i]);
      }
    }
    if (r == 0) {
      if (a.rstd_post) a.rstd_post[row] = ry;
      if (a.rstd_next) a.rstd_next[row] = ro;
    }
  }
}

// The columns' weights are in shared memory.  With the two sums,
// D and y they are more than the 128 registers of 512 threads, and what is
// spilled is waited for in every chunk (32768 x 4096 bf16: 411 us).
template <typename T, bool WHOLE, bool BRANCH, bool FOLLOWING, bool DOUT>
__global__ void __launch_bounds__(BWD_NT, 1) join_bwd_kernel(const JoinK a) {
  constexpr int VN = Vec<T>::N, CN = Mine<T, WHOLE>::CN, NC = EPT / VN;
  __shared__ float4 scratch[2 * 16];
  __shared__ uint64_t bars[MAX_GROUPS * RING];
  __shared__ __align__(16) uint4 zeros;
  if (threadIdx.x == 0) zeros = make_uint4(0, 0, 0, 0);
  const Group<true> grp(a.tpr);
  const int r = grp.r;
  const bool post = BRANCH && a.gamma_post != nullptr;
  JoinRows<T, WHOLE> R(FOLLOWING ? a.dh : nullptr, FOLLOWING ? a.out : nullptr, DOUT ? a.dout : nullptr, BRANCH ? a.y : nullptr);
  constexpr int bh = 0, bo = 1, bd = FOLLOWING ? 2 : 0, by_ = bd + DOUT;
  const int wbytes = EPT * a.tpr * 4;
  begin<T, WHOLE>(R, a, bars, r, 2 * wbytes);
  const Mine<T, WHOLE> mine(a, r, sm_addr(&zeros));
  const float inv = 1.f / (float)a.d;
  const uint32_t gn_s = sm_addr(join_smem), ga_s = gn_s + wbytes;  // weights
  mine.keep_weights(reinterpret_cast<float*>(join_smem), a.gamma_next, nullptr, 1.f);
  mine.keep_weights(reinterpret_cast<float*>(join_smem + wbytes), a.gamma_post, a.gate, a.bs);
  __syncthreads();
  float2 sn[EPT / 2], sm[EPT / 2];  // the columns' sums of dh n and row_gate D m
#pragma unroll
  for (int c = 0; c < EPT / 2; ++c) sn[c] = sm[c] = both(0.f);
  // ro, ry and the gate of a row, loaded two rows ahead of their use
  auto stats = [&](int64_t row) {
    const bool in = row < a.rows;
    return make_float3(in && FOLLOWING ? __ldg(a.rstd_next + row) : 0.f, in && post ? __ldg(a.rstd_post + row) : 1.f,
                       in && a.row_gate ? __ldg(a.row_gate + row) : 1.f);
  };
  // the warp's sum of v n of the row at place R.at, and its part of the columns' sums
  auto along = [&](int64_t row, float ro) {
    R.wait(a.err);
    mine.patch(R, row);
    if (!FOLLOWING) return 0.f;
    const Span sp = row_span<T, WHOLE>(row, a.rows, a.d);
    float2 s = both(0.f);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float2 n[CN], v[CN], gn[CN];
      mine.weights(gn_s, i, gn);
      mine.get(R.place(R.at, sp), bo, i, n);
      mine.get(R.place(R.at, sp), bh, i, v);
#pragma unroll
      for (int c = 0; c < CN; ++c) {  // past the row's end dh is 0
        v[c] = mul2(n[c], v[c]);
        sn[i * CN + c] = fma2(v[c], both(ro), sn[i * CN + c]);
        s = fma2(v[c], gn[c], s);
      }
    }
    return warp_sum(s.x + s.y) * ro;
  };
  const bool alone = grp.warps == 1;
  int turn = 0;
  // both sums over the group
  auto sums = [&](float u, float v) {
    if (alone) {
      __syncwarp();
      return make_float2(u, v);
    }
    grp.give(make_float4(u, v, 0.f, 0.f), scratch, turn);
    grp.sync();
    const float4 w = grp.get(scratch, turn);
    turn ^= 1;
    return make_float2(sum_over(w.x, grp.warps), sum_over(w.y, grp.warps));
  };
  float3 st = stats(R.first), st1 = stats(R.first + R.step);
  float mvn = 0.f;
  if (R.first < a.rows) mvn = sums(0.f, along(R.first, st.x)).y * inv;
#pragma unroll 1
  for (int64_t row = R.first; row < a.rows; row += R.step) {
    const float3 st2 = stats(row + 2 * R.step);
    const Span sp = row_span<T, WHOLE>(row, a.rows, a.d);
    const float2 ro = both(st.x), by = both(st.y * st.z), k = both(-mvn * st.x);
    float2 D[NC][CN], y[NC][CN], s = both(0.f);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (DOUT) {
        mine.get(R.place(R.at, sp), bd, i, D[i]);
      } else {
#pragma unroll
        for (int c = 0; c < CN; ++c) D[i][c] = both(0.f);
      }
      if (FOLLOWING) {
        float2 n[CN], v[CN], gn[CN];
        mine.weights(gn_s, i, gn);
        mine.get(R.place(R.at, sp), bo, i, n);
        mine.get(R.place(R.at, sp), bh, i, v);
#pragma unroll
        for (int c = 0; c < CN; ++c) D[i][c] = fma2(ro, fma2(v[c], gn[c], mul2(n[c], k)), D[i][c]);
      }
      if (BRANCH) {
        float2 ga[CN];
        mine.weights(ga_s, i, ga);
        mine.get(R.place(R.at, sp), by_, i, y[i]);
#pragma unroll
        for (int c = 0; c < CN; ++c) {  // m = y ry
          const float2 t = mul2(D[i][c], y[i][c]);
          sm[i * CN + c] = fma2(t, by, sm[i * CN + c]);
          s = fma2(t, ga[c], s);
        }
      }
    }
    const int place = R.at;
    float ahead = 0.f;
    R.next();
    const float own = BRANCH ? warp_sum(s.x + s.y) * st.y : 0.f;
    if (row + R.step < a.rows) ahead = along(row + R.step, st1.x);
    const float2 t = sums(own, ahead);
    if (r == 0) {
      R.start(row + R.ring * R.step, place);  // everyone has read the row
      if (a.drow_gate) a.drow_gate[row] = t.x;
    }
    mvn = t.y * inv;
    const float2 rs = both(a.rs), ky = both(post ? -t.x * st.z * inv * st.y * st.y : 0.f);  // of y in dy
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (BRANCH) {
        float2 ga[CN];
        mine.weights(ga_s, i, ga);
#pragma unroll
        for (int c = 0; c < CN; ++c) y[i][c] = fma2(mul2(D[i][c], ga[c]), by, mul2(y[i][c], ky));
        mine.set(a.dy, sp, i, y[i]);
      }
      if (a.dx) {
#pragma unroll
        for (int c = 0; c < CN; ++c) D[i][c] = mul2(D[i][c], rs);
        mine.set(a.dx, sp, i, D[i]);
      }
    }
    st = st1;
    st1 = st2;
  }
  __syncthreads();
  // the CTA's sums, over its groups in order, are one row pair of the partials
  const int groups = blockDim.x / a.tpr;
  float* dst = a.partial + (size_t)blockIdx.x * 2 * a.d;
  float* sums_at = groups == 1 ? dst : reinterpret_cast<float*>(join_smem) + (size_t)grp.g * 2 * a.d;
#pragma unroll
  for (int c = 0; c < EPT; ++c) {
    const int col = mine.column(c / VN) + c % VN;
    if (col >= 0 && col < a.d) {
      sums_at[col] = c & 1 ? sn[c / 2].y : sn[c / 2].x;
      sums_at[a.d + col] = c & 1 ? sm[c / 2].y : sm[c / 2].x;
    }
  }
  if (groups == 1) return;
  __syncthreads();
  const float* all = reinterpret_cast<const float*>(join_smem);
  for (int i = threadIdx.x; i < 2 * a.d; i += blockDim.x) {
    float u = 0.f;
#pragma unroll 4
    for (int g = 0; g < groups; ++g) u += all[(size_t)g * 2 * a.d + i];
    dst[i] = u;
  }
}

// ------------------------------ wide rows ---------------------------------- //
__device__ __forceinline__ float row_sum(float v, float* scratch, int& turn) {
  v = warp_sum(v);
  if (threadIdx.x % 32 == 0) scratch[turn * 16 + threadIdx.x / 32] = v;
  __syncthreads();
  v = warp_sum(threadIdx.x % 32 < WIDE_NT / 32 ? scratch[turn * 16 + threadIdx.x % 32] : 0.f);
  turn ^= 1;
  return v;
}
// a weight of each channel, 1 where there is none (vectors need not be aligned)
template <int VN>
__device__ __forceinline__ void ld_or_one(const float* p, int i, float (&v)[VN]) {
#pragma unroll
  for (int j = 0; j < VN; ++j) v[j] = p == nullptr ? 1.f : __ldg(p + i + j);
}

template <typename T, int VN>
__global__ void __launch_bounds__(WIDE_NT) join_fwd_wide_kernel(const JoinK a) {
  pdl_enter();
  __shared__ float scratch[2 * 16];
  int turn = 0;
  const float inv = 1.f / (float)a.d;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.d;
    const T* y = static_cast<const T*>(a.y) + (a.y ? row * a.d : 0);
    float ry = 1.f, ro = 0.f;
    if (a.gamma_post) {
      float s = 0.f;
      for (int i = threadIdx.x * VN; i < a.d; i += WIDE_NT * VN) {
        float v[VN];
        ld_n<T, VN>(y + i, v);
#pragma unroll
        for (int j = 0; j < VN; ++j) s = fmaf(v[j], v[j], s);
      }
      ry = rsqrtf(fmaf(row_sum(s, scratch, turn), inv, a.eps));
    }
    const float by = a.bs * (a.row_gate ? a.row_gate[row] : 1.f) * ry;
    auto joined = [&](int i, float (&o)[VN]) {
      ld_n<T, VN>(x + i, o);
#pragma unroll
      for (int j = 0; j < VN; ++j) o[j] *= a.rs;
      if (a.y) {
        float v[VN], g[VN], w[VN];
        ld_n<T, VN>(y + i, v);
        ld_or_one<VN>(a.gamma_post, i, g);
        ld_or_one<VN>(a.gate, i, w);
#pragma unroll
        for (int j = 0; j < VN; ++j) o[j] = fmaf(v[j] * by, g[j] * w[j], o[j]);
      }
    };
    if (a.gamma_next) {
      float s = 0.f;
      for (int i = threadIdx.x * VN; i < a.d; i += WIDE_NT * VN) {
        float o[VN];
        joined(i, o);
#pragma unroll
        for (int j = 0; j < VN; ++j) s = fmaf(o[j], o[j], s);
      }
      ro = rsqrtf(fmaf(row_sum(s, scratch, turn), inv, a.eps));
    }
    for (int i = threadIdx.x * VN; i < a.d; i += WIDE_NT * VN) {
      float o[VN];
      joined(i, o);
      if (a.out) st_n<T, VN>(static_cast<T*>(a.out) + row * a.d + i, o);
      if (a.gamma_next) {
        float g[VN];
        ld_or_one<VN>(a.gamma_next, i, g);
#pragma unroll
        for (int j = 0; j < VN; ++j) o[j] *= ro * g[j];
        st_n<T, VN>(static_cast<T*>(a.h) + row * a.d + i, o);
      }
    }
    if (threadIdx.x == 0) {
      if (a.rstd_post) a.rstd_post[row] = ry;
      if (a.rstd_next) a.rstd_next[row] = ro;
    }
  }
}

// D of VN elements of a row, from the mean of v n
template <typename T, int VN>
__device__ __forceinline__ void stream_grad(const JoinK& a, int64_t row, int i, float ro, float mvn, float (&D)[VN]) {
  if (a.dout) {
    ld_n<T, VN>(static_cast<const T*>(a.dout) + row * a.d + i, D);
  } else {
#pragma unroll
    for (int j = 0; j < VN; ++j) D[j] = 0.f;
  }
  if (a.gamma_next) {
    float n[VN], v[VN], g[VN];
    ld_n<T, VN>(static_cast<const T*>(a.out) + row * a.d + i, n);
    ld_n<T, VN>(static_cast<const T*>(a.dh) + row * a.d + i, v);
    ld_or_one<VN>(a.gamma_next, i, g);
#pragma unroll
    for (int j = 0; j < VN; ++j) D[j] = fmaf(ro, fmaf(v[j], g[j], -(n[j] * ro) * mvn), D[j]);
  }
}

// sum(v n) / d of each row
template <typename T, int VN>
__global__ void __launch_bounds__(WIDE_NT) join_bwd_stats_kernel(const JoinK a) {
  pdl_enter();
  __shared__ float scratch[2 * 16];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float s = 0.f;
    if (a.gamma_next) {
      for (int i = threadIdx.x * VN; i < a.d; i += WIDE_NT * VN) {
        float n[VN], v[VN], g[VN];
        ld_n<T, VN>(static_cast<const T*>(a.out) + row * a.d + i, n);
        ld_n<T, VN>(static_cast<const T*>(a.dh) + row * a.d + i, v);
        ld_or_one<VN>(a.gamma_next, i, g);
#pragma unroll
        for (int j = 0; j < VN; ++j) s = fmaf(v[j] * g[j], n[j], s);
      }
      s = row_sum(s, scratch, turn) * a.rstd_next[row] / (float)a.d;
    }
    if (threadIdx.x == 0) a.mean_vn[row] = s;
  }
}

// The sums of VN columns a thread over the rows blockIdx.y, + gridDim.y, ...
template <typename T, int VN>
__global__ void __launch_bounds__(COL_NT) join_bwd_columns_kernel(const JoinK a) {
  pdl_enter();
  const int i = (blockIdx.x * COL_NT + threadIdx.x) * VN;
  if (i >= a.d) return;
  float sn[VN], sm[VN];
#pragma unroll
  for (int j = 0; j < VN; ++j) sn[j] = sm[j] = 0.f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float ro = a.gamma_next ? a.rstd_next[row] : 0.f;
    if (a.gamma_next) {
      float n[VN], v[VN];
      ld_n<T, VN>(static_cast<const T*>(a.out) + row * a.d + i, n);
      ld_n<T, VN>(static_cast<const T*>(a.dh) + row * a.d + i, v);
#pragma unroll
      for (int j = 0; j < VN; ++j) sn[j] = fmaf(v[j], n[j] * ro, sn[j]);
    }
    if (a.y) {
      const float by = (a.row_gate ? a.row_gate[row] : 1.f) * (a.gamma_post ? a.rstd_post[row] : 1.f);
      float D[VN], m[VN];
      stream_grad<T, VN>(a, row, i, ro, a.mean_vn[row], D);
      ld_n<T, VN>(static_cast<const T*>(a.y) + row * a.d + i, m);
#pragma unroll
      for (int j = 0; j < VN; ++j) sm[j] = fmaf(D[j], m[j] * by, sm[j]);
    }
  }
  float* out = a.partial + (size_t)blockIdx.y * 2 * a.d;
#pragma unroll
  for (int j = 0; j < VN; ++j) {
    out[i + j] = sn[j];
    out[a.d + i + j] = sm[j];
  }
}

template <typename T, int VN>
__global__ void __launch_bounds__(WIDE_NT) join_bwd_wide_kernel(const JoinK a) {
  pdl_enter();
  __shared__ float scratch[2 * 16];
  int turn = 0;
  const float inv = 1.f / (float)a.d;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const float ro = a.gamma_next ? a.rstd_next[row] : 0.f, ry = a.gamma_post ? a.rstd_post[row] : 1.f;
    const float mvn = a.mean_vn[row], rg = a.row_gate ? a.row_gate[row] : 1.f;
    const T* y = static_cast<const T*>(a.y) + (a.y ? row * a.d : 0);
    float mwm = 0.f;
    if (a.gamma_post || a.drow_gate) {
      float s = 0.f;  // sum of bs gate gamma_post D m
      for (int i = threadIdx.x * VN; i < a.d; i += WIDE_NT * VN) {
        float D[VN], m[VN], g[VN], w[VN];
        stream_grad<T, VN>(a, row, i, ro, mvn, D);
        ld_n<T, VN>(y + i, m);
        ld_or_one<VN>(a.gate, i, g);
        ld_or_one<VN>(a.gamma_post, i, w);
#pragma unroll
        for (int j = 0; j < VN; ++j) s = fmaf(a.bs * D[j] * g[j] * w[j], m[j] * ry, s);
      }
      s = row_sum(s, scratch, turn);
      if (a.drow_gate && threadIdx.x == 0) a.drow_gate[row] = s;
      mwm = s * rg * inv;
    }
    for (int i = threadIdx.x * VN; i < a.d; i += WIDE_NT * VN) {
      float D[VN], o[VN], m[VN], g[VN], w[VN];
      stream_grad<T, VN>(a, row, i, ro, mvn, D);
      if (a.y) {
        ld_n<T, VN>(y + i, m);
        ld_or_one<VN>(a.gate, i, g);
        ld_or_one<VN>(a.gamma_post, i, w);
#pragma unroll
        for (int j = 0; j < VN; ++j) {
          const float G = a.bs * rg * g[j] * D[j];
          o[j] = a.gamma_post ? ry * fmaf(G, w[j], -(m[j] * ry) * mwm) : G;
        }
      }
#pragma unroll
      for (int j = 0; j < VN; ++j) D[j] *= a.rs;
      if (a.dx) st_n<T, VN>(static_cast<T*>(a.dx) + row * a.d + i, D);
      if (a.dy) st_n<T, VN>(static_cast<T*>(a.dy) + row * a.d + i, o);
    }
  }
}

// The parameters' gradients from the partials [parts][2][d], added in part
// order within RED_STRIPS interleaved strips and then over the strips.  The sum
// S of row_gate D m gives both that of gamma_post and that of the gate.
__global__ void __launch_bounds__(RED_COLS * RED_STRIPS) join_bwd_reduce_kernel(const JoinK a) {
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
  if (strip != 0 || col >= 2 * a.d) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < RED_STRIPS; ++i) s += tile[i][c];
  auto give = [&](float* dst, float v) { *dst = a.accumulate ? *dst + v : v; };
  if (col < a.d) {
    if (a.dgamma_next) give(a.dgamma_next + col, s);
    return;
  }
  const int i = col - a.d;
  s *= a.bs;
  if (a.dgamma_post) give(a.dgamma_post + i, a.gate ? s * a.gate[i] : s);
  if (a.dgate) give(a.dgate + i, a.gamma_post ? s * a.gamma_post[i] : s);
}

JoinK kernel_args(const JoinArgs& a, uint32_t* err) {
  JoinK k{};
  k.x = a.x;
  k.y = a.y;
  k.dh = a.dh;
  k.dout = a.dout;
  k.out = a.out;
  k.h = a.h;
  k.dx = a.dx;
  k.dy = a.dy;
  k.gamma_post = a.p.gamma_post;
  k.gamma_next = a.p.gamma_next;
  k.gate = a.p.gate;
  k.row_gate = a.p.row_gate;
  k.rstd_post = a.rstd_post;
  k.rstd_next = a.rstd_next;
  k.dgamma_post = a.g.dgamma_post;
  k.dgamma_next = a.g.dgamma_next;
  k.dgate = a.g.dgate;
  k.drow_gate = a.g.drow_gate;
  k.rows = a.p.rows;
  k.d = a.p.d;
  k.accumulate = a.accumulate;
  k.rs = a.p.residual_scale;
  k.bs = a.p.branch_scale;
  k.eps = a.p.eps;
  k.err = err;
  return k;
}

unsigned row_ctas(int64_t rows) {
  const int64_t most = (int64_t)sm_count() * 4;
  return (unsigned)(rows < most ? rows : most);
}
// Row slices of the columns' sums: about 16 CTAs an SM
int wide_slices(int64_t rows, int d) {
  const int64_t tiles = (d + COL_NT * 8 - 1) / (COL_NT * 8), most = ((int64_t)sm_count() * 16 + tiles - 1) / tiles;
  return (int)(rows < most ? rows : most);
}

template <typename T, int VN>
cudaError_t fwd_wide(const JoinK& a, cudaStream_t st) {
  return launch_pdl(join_fwd_wide_kernel<T, VN>, dim3(row_ctas(a.rows)), dim3(WIDE_NT), 0, st, a);
}
template <typename T, int VN>
cudaError_t bwd_wide(JoinK& a, cudaStream_t st) {
  a.parts = wide_slices(a.rows, a.d);
  cudaError_t e = launch_pdl(join_bwd_stats_kernel<T, VN>, dim3(row_ctas(a.rows)), dim3(WIDE_NT), 0, st, a);
  if (e != cudaSuccess) return e;
  e = launch_pdl(join_bwd_columns_kernel<T, VN>, dim3((a.d + COL_NT * VN - 1) / (COL_NT * VN), a.parts), dim3(COL_NT), 0,
                 st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(join_bwd_wide_kernel<T, VN>, dim3(row_ctas(a.rows)), dim3(WIDE_NT), 0, st, a);
}
// Sizes of a launch over rows in the ring of `bufs` tensors.  Forward: CTAs of one
// group of threads, or of four warps with rows of their own, as many as the
// registers allow.  Backward: one CTA an SM, of as many groups as leave the ring
// two places (three: 46 us at 4099 x 1021 float32, not 40).  ring < 2: no room, the wide kernels.
struct Grid {
  int threads, ctas, tpr, slot, ring;
  size_t smem;
};
Grid grid_of(int64_t rows, int d, int es, int bufs, bool bwd) {
  Grid g{};
  const bool whole = d * es % 16 == 0;
  const int most_units = whole ? d * es / 16 : (d * es + 15 + 16 - es) / 16;  // of a row
  if (most_units * 16 > MAX_TPR * EPT * es) return g;
  g.tpr = threads_per_row(most_units * 16 / es);
  g.slot = whole ? most_units * 16 : (most_units * 16 + 112 + 127) / 128 * 128;
  const size_t place = (size_t)bufs * g.slot, weights = bwd ? 2 * EPT * g.tpr * 4 : 0;
  int groups = bwd ? BWD_NT / g.tpr : (g.tpr == 32 ? 4 : 1), per = bwd ? 1 : 65536 / (g.tpr * groups * fwd_regs(es));
  const size_t room = bwd ? BWD_SMEM - weights : SMEM_SM;
  if (bwd) groups = std::max(1, std::min(groups, (int)(room / (2 * place))));
  while (per > 1 && per * 2 * (groups * place + 1024) > room) --per;
  g.ring = (int)std::min<size_t>(RING, (bwd ? room : SMEM_SM / per - 1024) / (groups * place));
  g.threads = g.tpr * groups;
  g.smem = weights + g.ring * groups * place;
  const size_t sums = groups > 1 ? (size_t)groups * 2 * d * 4 : 0;  // the backward's groups' sums take the ring's place
  if (bwd && g.smem < sums) g.smem = sums;
  const int64_t need = bwd ? rows : (rows + groups - 1) / groups;
  g.ctas = (int)std::min<int64_t>(need, (int64_t)sm_count() * per);
  // the rows of a CTA are as many CTAs apart, and begin alike in their first units: a multiple of a unit's elements
  if (!whole) g.ctas = g.ctas < 8 ? 8 : std::min(g.ctas + 7, sm_count() * per) / 8 * 8;
  return g;
}

template <typename K>
cudaError_t launch_ring(K kernel, const Grid& g, JoinK& a, std::atomic<bool>* attr_done, cudaStream_t st) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  if (!attr_done[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, std::max(SMEM_SM, BWD_SMEM));
    if (e != cudaSuccess) return e;
    attr_done[dev] = true;
  }
  a.tpr = g.tpr;
  a.slot = g.slot;
  a.ring = g.ring;
  a.parts = g.ctas;
  return launch_pdl(kernel, dim3(g.ctas), dim3(g.threads), g.smem, st, a);
}
template <typename T, bool WHOLE, bool BRANCH, bool FOLLOWING>
cudaError_t fwd_ring(const Grid& g, JoinK& a, cudaStream_t st) {
  static std::atomic<bool> done[64];
  return launch_ring(join_fwd_kernel<T, WHOLE, BRANCH, FOLLOWING>, g, a, done, st);
}
template <typename T, bool WHOLE, bool BRANCH, bool FOLLOWING, bool DOUT>
cudaError_t bwd_ring(const Grid& g, JoinK& a, cudaStream_t st) {
  static std::atomic<bool> done[64];
  return launch_ring(join_bwd_kernel<T, WHOLE, BRANCH, FOLLOWING, DOUT>, g, a, done, st);
}
template <typename T, bool WHOLE>
cudaError_t fwd_w(JoinK& a, cudaStream_t st) {
  const Grid g = grid_of(a.rows, a.d, sizeof(T), a.y ? 2 : 1, false);
  if (g.ring < 2) return fwd_wide<T, WHOLE ? Vec<T>::N : 1>(a, st);
  if (!a.y) return a.gamma_next ? fwd_ring<T, WHOLE, false, true>(g, a, st) : fwd_ring<T, WHOLE, false, false>(g, a, st);
  return a.gamma_next ? fwd_ring<T, WHOLE, true, true>(g, a, st) : fwd_ring<T, WHOLE, true, false>(g, a, st);
}
template <typename T, bool WHOLE>
cudaError_t bwd_w(JoinK& a, cudaStream_t st) {
  const int bufs = (a.gamma_next ? 2 : 0) + (a.dout ? 1 : 0) + (a.y ? 1 : 0);
  const Grid g = grid_of(a.rows, a.d, sizeof(T), bufs, true);
  if (g.ring < 2) return bwd_wide<T, WHOLE ? Vec<T>::N : 1>(a, st);
  if (!a.gamma_next)  // dout is there then
    return a.y ? bwd_ring<T, WHOLE, true, false, true>(g, a, st) : bwd_ring<T, WHOLE, false, false, true>(g, a, st);
  if (a.y) return a.dout ? bwd_ring<T, WHOLE, true, true, true>(g, a, st) : bwd_ring<T, WHOLE, true, true, false>(g, a, st);
  return a.dout ? bwd_ring<T, WHOLE, false, true, true>(g, a, st) : bwd_ring<T, WHOLE, false, true, false>(g, a, st);
}
template <typename T>
cudaError_t fwd_t(JoinK& a, cudaStream_t st) {
  return a.d % Vec<T>::N == 0 ? fwd_w<T, true>(a, st) : fwd_w<T, false>(a, st);
}
template <typename T>
cudaError_t bwd_t(JoinK& a, cudaStream_t st) {
  return a.d % Vec<T>::N == 0 ? bwd_w<T, true>(a, st) : bwd_w<T, false>(a, st);
}
size_t partial_bytes(int64_t rows, int d) {
  return (size_t)std::max<int64_t>(wide_slices(rows, d), std::min<int64_t>(rows + 7, std::max(sm_count(), 8))) * 2 * d * 4;
}

}  // namespace

size_t join_ws_bytes(int64_t rows, int d) {
  return rows == 0 ? 0 : (partial_bytes(rows, d) + 255) / 256 * 256 + (size_t)rows * 4;
}

cudaError_t launch_join_fwd(const JoinArgs& args, uint32_t* err, cudaStream_t st) {
  JoinK a = kernel_args(args, err);
  LaunchScope ls(KK_RESIDUAL_NORM_FWD, st);
  return args.p.dtype == MOE_BF16 ? fwd_t<__nv_bfloat16>(a, st) : fwd_t<float>(a, st);
}

cudaError_t launch_join_bwd(const JoinArgs& args, uint32_t* err, cudaStream_t st) {
  JoinK a = kernel_args(args, err);
  a.partial = static_cast<float*>(args.ws);
  a.mean_vn = reinterpret_cast<float*>(static_cast<char*>(args.ws) + (partial_bytes(a.rows, a.d) + 255) / 256 * 256);
  {
    LaunchScope ls(KK_RESIDUAL_NORM_BWD, st);
    const cudaError_t e = args.p.dtype == MOE_BF16 ? bwd_t<__nv_bfloat16>(a, st) : bwd_t<float>(a, st);
    if (e != cudaSuccess) return e;
  }
  if (!a.dgamma_post && !a.dgamma_next && !a.dgate) return cudaSuccess;
  LaunchScope ls(KK_RESIDUAL_NORM_REDUCE, st);
  return launch_pdl(join_bwd_reduce_kernel, dim3((2 * a.d + RED_COLS - 1) / RED_COLS), dim3(RED_COLS * RED_STRIPS), 0,
                    st, a);
}

}  // namespace moe
