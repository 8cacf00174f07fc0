// Softmax cross entropy over a large vocabulary and its gradient, the logits
// formed a piece at a time and never kept; formulas are in moe.h.
//
// The labelled tokens are listed first and their rows of x packed, padded with
// zero rows to whole tiles: ignored tokens cost nothing further, and what their
// rows hold reaches no product.  float32 rows are split into bf16 parts on the
// way.  The products run on the tensor cores (vocab_loss_tc.cu); the forward's
// leaves two floats a row and 128 words, which loss_combine_kernel joins.  The
// backward goes over the vocabulary in equal pieces: dz of a piece, then its
// part of dx (added up in fp32) and its rows of dW.
#include <algorithm>

#include "common.cuh"
#include "vocab_loss.h"

namespace moe {
namespace {

constexpr int LIST_NT = 1024, LIST_EACH = 8;        // labels a thread takes at a time
constexpr int ROW_NT = 256;
constexpr int MAX_SLICES = 64;
constexpr int64_t PIECE_VALUES = (int64_t)1 << 28;  // of a part of dz: 512 MB at most, or a tile's columns

// The labelled tokens in order, each token's place among them, their number.
__global__ void __launch_bounds__(LIST_NT) loss_rows_kernel(const LossWork w, const int32_t* labels) {
  pdl_enter();
  __shared__ int before[32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int base = 0;
  for (int t0 = 0; t0 < w.T; t0 += LIST_NT * LIST_EACH) {
    const int first = t0 + threadIdx.x * LIST_EACH;
    int label[LIST_EACH], mine = 0;
#pragma unroll
    for (int i = 0; i < LIST_EACH; ++i) label[i] = first + i < w.T ? labels[first + i] : -1;
#pragma unroll
    for (int i = 0; i < LIST_EACH; ++i) {
      if (label[i] >= w.V) {
        report_error(w.err, DEV_BAD_LABEL, (uint32_t)(first + i) & 0xFFFFFFu);
        label[i] = -1;
      }
      mine += label[i] >= 0;
    }
    int upto = mine;  // in this warp
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      upto += lane >= o ? v : 0;
    }
    __syncthreads();
    if (lane == 31) before[warp] = upto;
    __syncthreads();
    int at = base + upto - mine, all = 0;
    for (int i = 0; i < LIST_NT / 32; ++i) {
      at += i < warp ? before[i] : 0;
      all += before[i];
    }
#pragma unroll
    for (int i = 0; i < LIST_EACH; ++i) {
      if (first + i >= w.T) continue;
      w.pos[first + i] = label[i] >= 0 ? at : -1;
      if (label[i] >= 0) w.list[at++] = first + i;
    }
    base += all;
  }
  if (threadIdx.x == 0) *w.count = base;
}

// Three bf16 parts of 8 bits each whose sum is v; an infinity is its first part alone.
__device__ __forceinline__ void split3(float v, __nv_bfloat16 (&p)[MAX_PARTS]) {
  float rest = v;
#pragma unroll
  for (int i = 0; i < MAX_PARTS; ++i) {
    const float top = __uint_as_float(__float_as_uint(rest) & 0xffff0000u);
    p[i] = __float2bfloat16_rn(isnan(v) ? v : top);
    rest = isfinite(v) ? rest - top : 0.f;
  }
}

// Four elements of a float32 row as parts at dst, dst + ld, dst + 2 ld.
__device__ __forceinline__ void put_parts(__nv_bfloat16* dst, int ld, const float (&v)[4]) {
  __nv_bfloat16 p[4][MAX_PARTS];
#pragma unroll
  for (int i = 0; i < 4; ++i) split3(v[i], p[i]);
#pragma unroll
  for (int j = 0; j < MAX_PARTS; ++j) {
    __nv_bfloat162 q[2] = {__nv_bfloat162(p[0][j], p[1][j]), __nv_bfloat162(p[2][j], p[3][j])};
    *reinterpret_cast<uint2*>(dst + (size_t)j * ld) = *reinterpret_cast<uint2*>(q);
  }
}

struct PackArgs {
  const void* x;
  const int32_t* labels;
  const float* lse;    // backward
  const float* dloss;  // backward, or null
  float* loss;         // forward: 0 for the ignored tokens
  float* lse_out;
};
// A CTA a row at a time: the labelled rows of x, zeros up to a whole tile; what
// the epilogues want of each row; in the forward 0 for the ignored tokens.
template <typename T>
__global__ void __launch_bounds__(ROW_NT) loss_pack_kernel(const LossWork w, const PackArgs a) {
  pdl_enter();
  const int n = *w.count, rows = (n + LOSS_TILE - 1) / LOSS_TILE * LOSS_TILE;
  constexpr int VN = Vec<T>::N;
  for (int r = blockIdx.x; r < rows; r += gridDim.x) {
    const int t = r < n ? w.list[r] : 0;
    const T* src = static_cast<const T*>(a.x) + (int64_t)t * w.d;
    __nv_bfloat16* dst = w.xp + (int64_t)r * w.parts * w.ldx;
    for (int i = threadIdx.x * VN; i < w.ldx; i += ROW_NT * VN) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (r < n && i < w.d) u = ldg16(src + i);
      if constexpr (VN == 8) {
        stg16(dst + i, u);
      } else {
        float v[4];
        unpack(u, v);
        put_parts(dst + i, w.ldx, v);
      }
    }
    if (threadIdx.x == 0) {
      w.label[r] = r < n ? a.labels[t] : -1;
      if (a.lse != nullptr) {
        w.lse[r] = r < n ? a.lse[t] : 0.f;
        w.grad[r] = r < n ? (a.dloss ? a.dloss[t] : 1.f) : 0.f;
      }
    }
  }
  if (a.loss != nullptr)
    for (int t = blockIdx.x * ROW_NT + threadIdx.x; t < w.T; t += gridDim.x * ROW_NT)
      if (w.pos[t] < 0) a.loss[t] = a.lse_out[t] = 0.f;
}

// The parts of a float32 W, zeros up to ldw, a warp a row.  Infinities count as
// the largest bf16: as one part they would meet the zeros of the other operand's
// parts.
__global__ void __launch_bounds__(ROW_NT) loss_split_kernel(const LossWork w, const float* W, __nv_bfloat16* out) {
  pdl_enter();
  for (int row = blockIdx.x * (ROW_NT / 32) + threadIdx.x / 32; row < w.V; row += gridDim.x * (ROW_NT / 32)) {
    const float* src = W + (int64_t)row * w.d;
    __nv_bfloat16* dst = out + (int64_t)row * MAX_PARTS * w.ldw;
#pragma unroll 4
    for (int c = threadIdx.x % 32 * 4; c < w.ldw; c += 128) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (c < w.d) u = ldg16(src + c);
      float v[4];
      unpack(u, v);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (isinf(v[j])) v[j] = copysignf(0x1.fep127f, v[j]);
      put_parts(dst + c, w.ldw, v);
    }
  }
}

// 32 labelled tokens a CTA, their partial sums in 32 strips: lse, the loss.
__global__ void __launch_bounds__(1024) loss_combine_kernel(const LossWork w, int parts, float* loss, float* lse) {
  pdl_enter();
  __shared__ float tops[32][33], sums[32][33];
  const int n = *w.count, lane = threadIdx.x % 32, strip = threadIdx.x / 32;
  for (int r0 = blockIdx.x * 32; r0 < n; r0 += gridDim.x * 32) {
    const int r = r0 + lane;  // Tp is a multiple of 32: the row is there
    float top = -INFINITY, sum = 0.f;
#pragma unroll 4
    for (int i = strip; i < parts; i += 32) {
      const float2 p = w.partial[(int64_t)i * w.Tp + r];
      const float best = fmaxf(top, p.x), at = base_of(best);
      sum = sum * expf(top - at) + p.y * expf(p.x - at);
      top = best;
    }
    tops[strip][lane] = top;
    sums[strip][lane] = sum;
    __syncthreads();
    // a warp joins one token's strips
    top = tops[lane][strip];
    float best = top;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, o));
    const float at = base_of(best);
    sum = warp_sum(sums[lane][strip] * expf(top - at));
    if (lane == 0 && r0 + strip < n) {
      const int t = w.list[r0 + strip];
      const float v = best + logf(sum);
      lse[t] = v;
      // lse and the logit share the maximum: their difference is formed without it
      loss[t] = (best - w.picked[r0 + strip]) + logf(sum);
    }
    __syncthreads();
  }
}

// The sum of the losses, in token order within each thread, and the number of labelled tokens.
__global__ void __launch_bounds__(LIST_NT) loss_total_kernel(const LossWork w, const float* loss, float* total) {
  pdl_enter();
  __shared__ double scratch[32];
  double s = 0.0;
#pragma unroll 8
  for (int t = threadIdx.x; t < w.T; t += LIST_NT) s += loss[t];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (threadIdx.x % 32 == 0) scratch[threadIdx.x / 32] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    s = 0.0;
    for (int i = 0; i < LIST_NT / 32; ++i) s += scratch[i];
    total[0] = (float)s;
    total[1] = (float)*w.count;
  }
}

// dx of the labelled tokens from acc, 0 for the others.  A bf16 dx comes from dz
// in one part of 8 bits.  One term, the label's, is as large as all the others
// together, so its rounding would be dx's: what the part left of it is added
// here (8192 x 2048 x 50257: dx off by 0.17 % with it, its own rounding; 0.36 %
// without).
template <typename T>
__global__ void __launch_bounds__(ROW_NT) loss_dx_kernel(const LossWork w, const T* W, T* dx) {
  pdl_enter();
  constexpr int VN = Vec<T>::N;
  const float scale = w.mean ? 1.f / (float)*w.count : 1.f;
  for (int t = blockIdx.x; t < w.T; t += gridDim.x) {
    const int r = w.pos[t];
    if (r < 0) {
      for (int i = threadIdx.x * VN; i < w.d; i += ROW_NT * VN) stg16(dx + (int64_t)t * w.d + i, make_uint4(0, 0, 0, 0));
      continue;
    }
    const float* src = w.acc + (int64_t)r * w.d;
    const T* word = W + (int64_t)w.label[r] * w.d;
    const float off = sizeof(T) == 2 ? w.off[r] : 0.f;
    for (int i = threadIdx.x * VN; i < w.d; i += ROW_NT * VN) {
      float v[VN];
#pragma unroll
      for (int j = 0; j < VN; ++j) v[j] = 0.f;
#pragma unroll 4
      for (int s = 0; s < w.slices; ++s) {
        const float* from = src + (int64_t)s * w.Tp * w.d + i;
#pragma unroll
        for (int j = 0; j < VN; j += 4) {
          const float4 f = *reinterpret_cast<const float4*>(from + j);
          v[j] += f.x;
          v[j + 1] += f.y;
          v[j + 2] += f.z;
          v[j + 3] += f.w;
        }
      }
      if constexpr (sizeof(T) == 2) {
        float u[VN];
        unpack(ldg16(word + i), u);
#pragma unroll
        for (int j = 0; j < VN; ++j) v[j] = fmaf(off, u[j], v[j]);
      }
#pragma unroll
      for (int j = 0; j < VN; ++j) v[j] *= scale;
      stg16(dx + (int64_t)t * w.d + i, pack(v));
    }
  }
}

// ------------------------------ host side ---------------------------------- //
size_t up(size_t n, size_t a = 256) { return (n + a - 1) / a * a; }

// Equal pieces of the vocabulary, whole tiles each.
int piece_of(int64_t Tp, int64_t V) {
  const int64_t all = up(V, LOSS_TILE), most = PIECE_VALUES / Tp / LOSS_TILE * LOSS_TILE;
  if (most >= all) return (int)all;
  const int64_t pieces = (V + (most < LOSS_TILE ? LOSS_TILE : most) - 1) / (most < LOSS_TILE ? LOSS_TILE : most);
  return (int)up((V + pieces - 1) / pieces, LOSS_TILE);
}

// Slices of a piece for dx: two tiles of it are at most a pair's share of both
// gradients' work.  (64 tokens, d 4096, V 128000: 16 tiles of dx alone kept 16 of
// the 76 pairs busy for 800 us.)  It goes by T, not by how many tokens are labelled.
int slices_of(const LossWork& w) {
  const int64_t cols = (w.d + 255) / 256, k = w.piece / 128;
  const int64_t seg = w.parts == 1 ? 1 : 6, dx = w.Tp / LOSS_TILE * cols * k * seg;
  const int64_t both = dx + w.piece / LOSS_TILE * cols * (w.Tp / 128) * (w.parts == 1 ? w.dzp : 6);
  const int64_t s = (2 * k * seg * (sm_count() / 2) + both - 1) / both;
  const int64_t most = std::min<int64_t>(std::min<int64_t>(MAX_SLICES, k), ((int64_t)1 << 28) / ((int64_t)w.Tp * w.d));
  return (int)std::max<int64_t>(1, std::min(s, most));
}

// What dz and acc are given in the workspace: enough for as many tokens and for any
// fewer.  Equal pieces and slices of whole tiles take less of some larger batches
// than of smaller ones (bf16, 4096 x 128000: 617 MB for 2304 tokens, 1048 for 2048),
// and a buffer for the largest batch has to do for the last, shorter one.
//
// A piece has at most PIECE_VALUES values of a part, or a tile's columns of each row.
int64_t dz_values(int64_t Tp, int64_t V) {
  return std::max(std::min(Tp * (int64_t)up(V, LOSS_TILE), PIECE_VALUES), Tp * LOSS_TILE);
}
// Rows of acc.  slices_of is the ceiling of n / m for m tiles of tokens, n a ratio
// of the sizes that has neither tokens nor the piece in it, so slices * m < n + m
// below n tiles, and m from there on; and no more than its caps give.
int64_t acc_rows(const LossWork& w) {
  const int64_t seg = w.parts == 1 ? 1 : 6, cols = (w.d + 255) / 256, m = w.Tp / LOSS_TILE;
  const int64_t both = cols * (seg + (w.parts == 1 ? w.dzp : 6)), n = (2 * seg * (sm_count() / 2) + both - 1) / both;
  const int64_t most = std::min<int64_t>(MAX_SLICES, (int64_t)up(w.V, LOSS_TILE) / 128) * m;
  const int64_t tiles = std::min({n + std::min(m, n) - 1, most, ((int64_t)1 << 28) / ((int64_t)LOSS_TILE * w.d)});
  return std::max(m, tiles) * LOSS_TILE;
}

// What a call keeps in the workspace, from `base` on (null: its size alone); returns its end.
size_t lay_out(LossWork* w, char* base, int T, int d, int V, bool bf16, bool backward, int dzp) {
  size_t end = 0;
  auto take = [&](size_t bytes) {
    char* p = base + end;
    end += up(bytes);
    return base == nullptr ? nullptr : p;
  };
  w->T = T;
  w->Tp = (int)up(T, LOSS_TILE);
  w->d = d;
  w->V = V;
  w->parts = bf16 ? 1 : MAX_PARTS;
  w->ldx = w->ldw = bf16 ? d : (int)up(d, 128);
  w->dzp = dzp;
  w->piece = piece_of(w->Tp, V);
  const size_t Tp = w->Tp, parts = w->parts;
  w->list = reinterpret_cast<int32_t*>(take((size_t)T * 4));
  w->pos = reinterpret_cast<int32_t*>(take((size_t)T * 4));
  w->count = reinterpret_cast<int32_t*>(take(4));
  w->label = reinterpret_cast<int32_t*>(take(Tp * 4));
  w->xp = reinterpret_cast<__nv_bfloat16*>(take(Tp * parts * w->ldx * 2));
  if (!bf16) w->wp = reinterpret_cast<__nv_bfloat16*>(take((size_t)V * parts * w->ldw * 2));
  if (!backward) {
    w->picked = reinterpret_cast<float*>(take(Tp * 4));
    w->partial = reinterpret_cast<float2*>(take(up(V, LOSS_TILE) / LOSS_PART * Tp * 8));
  } else {
    w->lse = reinterpret_cast<float*>(take(Tp * 4));
    w->grad = reinterpret_cast<float*>(take(Tp * 4));
    w->off = reinterpret_cast<float*>(take(Tp * 4));
    w->dz = reinterpret_cast<__nv_bfloat16*>(take((size_t)dzp * dz_values(Tp, V) * 2));
    w->slices = slices_of(*w);
    w->acc = reinterpret_cast<float*>(take((size_t)acc_rows(*w) * d * 4));
  }
  return end;
}

#define LAUNCH(kind, ...)                            \
  do {                                               \
    LaunchScope ls(kind, st);                        \
    const cudaError_t e = launch_pdl(__VA_ARGS__);   \
    if (e != cudaSuccess) return e;                  \
  } while (0)

unsigned few(int64_t n, int per_sm) {
  const int64_t most = (int64_t)sm_count() * per_sm;
  return (unsigned)(n < most ? n : most);
}

// The labelled tokens' rows and W as the products read them.
cudaError_t prepare(LossWork* w, const LossArgs& a, const PackArgs& p, cudaStream_t st) {
  LAUNCH(KK_LOSS_ROWS, loss_rows_kernel, dim3(1), dim3(LIST_NT), 0, st, *w, a.labels);
  LAUNCH(KK_LOSS_ROWS, a.bf16 ? loss_pack_kernel<__nv_bfloat16> : loss_pack_kernel<float>, dim3(few(w->Tp, 8)),
         dim3(ROW_NT), 0, st, *w, p);
  if (a.bf16) {
    w->wp = static_cast<const __nv_bfloat16*>(a.W);
    return cudaSuccess;
  }
  LAUNCH(KK_LOSS_ROWS, loss_split_kernel, dim3(few((w->V + ROW_NT / 32 - 1) / (ROW_NT / 32), 16)), dim3(ROW_NT), 0, st,
         *w, static_cast<const float*>(a.W), const_cast<__nv_bfloat16*>(w->wp));
  return cudaSuccess;
}

}  // namespace

size_t loss_ws_bytes(int T, int d, int V, bool bf16, bool training) {
  if (T == 0) return 0;
  LossWork w{};
  size_t fwd = loss_few_bytes();  // that of more tokens may be less, of a small vocabulary
  if (!loss_is_few(T, d, bf16)) fwd = std::max(fwd, lay_out(&w, nullptr, T, d, V, bf16, false, 0));
  if (!training) return fwd;
  size_t most = fwd;
  for (int dzp = bf16 ? 1 : MAX_PARTS; dzp <= (bf16 ? 2 : MAX_PARTS); ++dzp)
    most = std::max(most, lay_out(&w, nullptr, T, d, V, bf16, true, dzp));
  return most;
}

cudaError_t launch_loss_fwd(const LossArgs& a, uint32_t* err, cudaStream_t st) {
  if (loss_is_few(a.T, a.d, a.bf16)) return launch_loss_few(a, err, st);
  LossWork w{};
  w.err = err;
  lay_out(&w, static_cast<char*>(a.ws), a.T, a.d, a.V, a.bf16, false, 0);
  cudaError_t e = prepare(&w, a, PackArgs{a.x, a.labels, nullptr, nullptr, a.loss, a.lse}, st);
  if (e != cudaSuccess) return e;
  e = tc_loss_logits(w, st);
  if (e != cudaSuccess) return e;
  LAUNCH(KK_LOSS_COMBINE, loss_combine_kernel, dim3(few((a.T + 31) / 32, 2)), dim3(1024), 0, st, w,
         (a.V + LOSS_PART - 1) / LOSS_PART, a.loss, a.lse);
  if (a.total) LAUNCH(KK_LOSS_FINISH, loss_total_kernel, dim3(1), dim3(LIST_NT), 0, st, w, (const float*)a.loss, a.total);
  return cudaSuccess;
}

cudaError_t launch_loss_bwd(const LossArgs& a, uint32_t* err, cudaStream_t st) {
  LossWork w{};
  w.err = err;
  // as many bits of dz as the results can use
  const int dzp = !a.bf16 ? MAX_PARTS : a.dW != nullptr && !a.dw_bf16 ? 2 : 1;
  lay_out(&w, static_cast<char*>(a.ws), a.T, a.d, a.V, a.bf16, true, dzp);
  w.mean = a.dloss == nullptr;
  cudaError_t e = prepare(&w, a, PackArgs{a.x, a.labels, a.lse, a.dloss, nullptr, nullptr}, st);
  for (w.v0 = 0; w.v0 < a.V; w.v0 += w.piece) {
    if (e == cudaSuccess) e = tc_loss_dlogits(w, st);
    if (e == cudaSuccess) e = tc_loss_grads(w, a.dx != nullptr, a.dW, a.dw_bf16, a.accumulate != 0, st);
    if (e != cudaSuccess) return e;
  }
  if (a.dx == nullptr) return cudaSuccess;
  if (a.bf16)
    LAUNCH(KK_LOSS_FINISH, loss_dx_kernel<__nv_bfloat16>, dim3(few(a.T, 8)), dim3(ROW_NT), 0, st, w,
           static_cast<const __nv_bfloat16*>(a.W), static_cast<__nv_bfloat16*>(a.dx));
  else
    LAUNCH(KK_LOSS_FINISH, loss_dx_kernel<float>, dim3(few(a.T, 8)), dim3(ROW_NT), 0, st, w,
           static_cast<const float*>(a.W), static_cast<float*>(a.dx));
  return cudaSuccess;
}

}  // namespace moe
