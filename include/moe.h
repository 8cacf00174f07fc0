/*
 * moe.h -- C ABI of the GB300 (sm_103a) mixture-of-experts layer step.
 *
 * One MoE layer step on one GPU: router scoring, top-k with a capacity factor
 * and overflow drop, permutation into contiguous per-expert buffers, the
 * experts' SwiGLU FFN as grouped GEMMs, the inverse permutation with a
 * gate-weighted combine, and the matching backward.  The sequence follows
 * "The step timeline: dispatch, expert GEMM, combine" on the
 * gpu_expert_parallel page: with every expert local, the dispatch and combine
 * all-to-alls reduce to the permute and the unpermute.
 *
 * Conventions shared by every call
 * --------------------------------
 * - All pointers are device pointers on the calling thread's current CUDA
 *   device unless a parameter says otherwise.  The library never allocates,
 *   frees or keeps caller memory; the caller owns every buffer.
 * - Every call that takes a stream is asynchronous on that stream (NULL = the
 *   legacy default stream) and never synchronises with the host, except
 *   moe_get_device_error and moe_profiler_read.
 * - Tensors are dense and row-major.  Activations and expert weights use
 *   cfg->dtype (MOE_F32 or MOE_BF16); router weights, router bias, gates,
 *   probabilities and every gradient buffer except dx are float32; index
 *   tensors are int32.
 * - Activation and weight pointers must be 16-byte aligned.
 * - MOE_BF16 needs d_model and d_ff to be multiples of 256 (the grouped GEMM
 *   tiles); MOE_F32 needs them to be multiples of 4.  1 <= k <= min(E, 8),
 *   1 <= E <= 128.
 * - Argument, shape and alignment errors are detected on the host before any
 *   work is queued and are returned as a status.  Launch failures return
 *   MOE_ERR_CUDA.  Problems found by the kernels (a corrupt routing state, an
 *   out-of-range row, a pipeline wait that exceeded its time limit) are
 *   recorded in a per-device error word and reported by
 *   moe_get_device_error; the offending access is skipped, never performed.
 *
 * Shapes (T tokens, d = d_model, f = d_ff, E experts, k picks per token)
 * -------------------------------------------------------------------------
 *   x, y, dy, dx          [T, d]           dtype
 *   W_r                   [d, E]           float32   router weight
 *   bias                  [E]              float32   fixed router bias (optional)
 *   W1, W3                [E, d, f]        dtype     x W1 -> gate path, x W3 -> up path
 *   W2                    [E, f, d]        dtype
 *   ids, slot, row_of     [T, k]           int32
 *   gates                 [T, k]           float32
 *   probs                 [T, E]           float32
 *   counts                [E]              int32     kept assignments per expert
 *   offsets               [E + 1]          int32     first row of each expert
 *   src_token             [max_rows]       int32     token of each row, -1 on pad rows
 *   x_perm, y_perm, dy_perm, dx_perm [max_rows, d]  dtype
 *   a, b, h, da, db       [max_rows, f]    dtype
 *   dW1, dW3              [E, d, f]        float32
 *   dW2                   [E, f, d]        float32
 *   dW_r                  [d, E]           float32
 *
 * Permutation map layout: the rows of expert e are
 * [offsets[e], offsets[e] + counts[e]), in slot order, followed by zero pad
 * rows up to offsets[e+1]; offsets[e] is a multiple of 128, offsets[0] = 0.
 * max_rows (moe_max_rows) bounds offsets[E] for every routing outcome.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; declared here so the header needs no CUDA headers. */
typedef struct CUstream_st* moe_stream_t;

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,  /* NULL where a pointer is required, bad flag value */
  MOE_ERR_SHAPE = 2,        /* sizes outside the supported range */
  MOE_ERR_DTYPE = 3,        /* unknown dtype */
  MOE_ERR_ALIGNMENT = 4,    /* a pointer is not 16-byte aligned */
  MOE_ERR_WORKSPACE = 5,    /* workspace missing or smaller than moe_workspace_size */
  MOE_ERR_CUDA = 6,         /* a CUDA runtime call or kernel launch failed */
  MOE_ERR_DEVICE_CHECK = 7, /* a kernel found an invalid index (see moe_get_device_error) */
  MOE_ERR_TIMEOUT = 8,      /* a kernel pipeline wait exceeded its time limit */
  MOE_ERR_UNSUPPORTED = 9   /* the device is not sm_103 */
} moe_status;

typedef enum { MOE_F32 = 0, MOE_BF16 = 1 } moe_dtype;

typedef struct {
  int32_t T;                /* tokens in this (micro-)batch, >= 0 */
  int32_t d_model;          /* d */
  int32_t d_ff;             /* f */
  int32_t E;                /* experts */
  int32_t k;                /* experts per token (top-k) */
  float capacity_factor;    /* C = ceil(cf * T * k / E); <= 0 means dropless */
  int32_t capacity;         /* >= 0: use this exact capacity instead of the factor; < 0: use the factor */
  int32_t dtype;            /* moe_dtype of activations and expert weights */
  float aux_loss_coeff;     /* >= 0; > 0 adds the auxiliary load-balancing loss to the backward (moe_aux_loss) */
} moe_config;

/* Expert and router parameters (device pointers, read only). */
typedef struct {
  const float* W_r;   /* [d, E] */
  const float* bias;  /* [E] or NULL */
  const void* W1;     /* [E, d, f] */
  const void* W3;     /* [E, d, f] */
  const void* W2;     /* [E, f, d] */
} moe_weights;

/* Routing state and activations that the forward keeps for the backward.
 * Keeping the assignment indices and the permutation map lets the backward
 * reuse the routing instead of recomputing it ("Recomputation re-runs the
 * dispatch unless you save the permutation", gpu_expert_parallel page).
 * Sizes are in the shape table above.  Recompute variant: with a, b and h all
 * NULL the forward keeps only the routing state, x_perm and y_perm, and the
 * backward recomputes a, b and h with the same up product (bit for bit the
 * forward's); the workspace is then moe_workspace_size(cfg, 2) for both calls. */
typedef struct {
  int32_t* ids;
  float* gates;
  int32_t* slot;
  int32_t* row_of;
  int32_t* src_token;
  int32_t* counts;
  int32_t* offsets;
  float* probs;
  void* x_perm;
  void* a;
  void* b;
  void* h;
  void* y_perm;
} moe_saved;

/* float32 gradient buffers of the parameters (accumulated across calls when
 * accumulate != 0, overwritten otherwise). */
typedef struct {
  float* dW_r;
  float* dW1;
  float* dW3;
  float* dW2;
  float* aux_loss;  /* device fp32 scalar that receives the auxiliary loss, or NULL */
} moe_grads;

/* Human-readable name of a status code (static storage). */
const char* moe_status_string(moe_status s);

/* Expert capacity: *C = ceil(cf * T * k / E) computed in double from the
 * float capacity factor, or cfg->capacity when that is >= 0, or -1 when the
 * layer is dropless.  Capacity-factor passage, "The Capacity Factor: A Dial
 * Between Imbalance and Dropping" (distributed-training tutorial, Expert
 * Parallelism section).  Host only. */
moe_status moe_capacity(const moe_config* cfg, int32_t* C);

/* Upper bound on offsets[E] (rows of the per-expert buffers), a multiple of
 * 128: min(T*k + 127*E, E * roundup128(C)) rounded up to 128.  Host only. */
moe_status moe_max_rows(const moe_config* cfg, int64_t* rows);

/* Bytes of workspace that moe_layer_fwd (training = 0) or moe_layer_fwd and
 * moe_layer_bwd (training = 1; 2 with a, b, h recomputed, see moe_saved) need.  The workspace holds the routing
 * histograms, the forward intermediates when no moe_saved is given, and the
 * backward scratch.  Host only; for bf16 layers the router-weight gradient's
 * partial sums scale with the SM count of the current device, so ask with the
 * device that will run the layer current. */
moe_status moe_workspace_size(const moe_config* cfg, int training, size_t* bytes);

/* Router scoring, softmax, top-k and capacity slotting (steps "the router
 * scores every token" and the capacity dial).
 *   logits l = x W_r + bias in fp32; probs = softmax(l) in fp32;
 *   ids[t, 0..k-1] = experts of the k largest logits, descending, ties to the
 *   lower index; gates: k = 1 -> probs[t, ids[t,0]]; k > 1 -> the picked
 *   probabilities renormalised over the picks;
 *   slot: assignments are visited choice-major then in token order; each
 *   expert hands out slots 0, 1, ...; an assignment at slot >= C is dropped
 *   (slot = -1, row_of = -1);  counts[e] = kept assignments of expert e;
 *   offsets, row_of, src_token as described at the top of this file.
 * probs may be NULL.  Deterministic.  ws must hold moe_workspace_size(cfg, 0). */
moe_status moe_router_topk(const moe_config* cfg, const void* x, const float* W_r, const float* bias,
                           int32_t* ids, float* gates, float* probs, int32_t* slot, int32_t* row_of,
                           int32_t* src_token, int32_t* counts, int32_t* offsets, void* ws, size_t ws_bytes,
                           moe_stream_t stream);

/* Permute tokens into the per-expert buffers ("tokens are permuted into
 * contiguous per-destination buffers"): x_perm[row_of[t,j]] = x[t] for every
 * kept assignment; pad rows [offsets[e] + counts[e], offsets[e+1]) are zeroed.
 * Rows at or beyond offsets[E] are not touched. */
moe_status moe_permute(const moe_config* cfg, const void* x, const int32_t* row_of, const int32_t* counts,
                       const int32_t* offsets, void* x_perm, moe_stream_t stream);

/* The experts' feed-forward as grouped GEMMs over the ragged row segments
 * ("Sorting tokens by destination is what lets the expert computation become
 * a batched or grouped matrix multiply"):
 *   a = X_e W1_e, b = X_e W3_e, h = silu(a) * b, y_perm = h W2_e
 * with fp32 accumulation; silu(z) = z / (1 + exp(-z)).  h is required; a and b
 * may be NULL (they are stored only for the backward).  Pad rows give zero. */
moe_status moe_grouped_ffn(const moe_config* cfg, const void* x_perm, const int32_t* counts,
                           const int32_t* offsets, const void* W1, const void* W3, const void* W2, void* h,
                           void* y_perm, void* a, void* b, moe_stream_t stream);

/* Inverse permutation with the gate-weighted combine ("the inverse permutation
 * restores the original token order"): y[t] = sum over kept j of
 * gates[t,j] * y_perm[row_of[t,j]], summed in fp32 in j order; a token whose
 * assignments were all dropped gets 0. */
moe_status moe_unpermute_combine(const moe_config* cfg, const void* y_perm, const int32_t* row_of,
                                 const float* gates, void* y, moe_stream_t stream);

/* Whole forward: moe_router_topk, moe_permute, moe_grouped_ffn,
 * moe_unpermute_combine.  With saved == NULL the intermediates live in ws;
 * with saved != NULL every field of *saved must be set and receives the state
 * moe_layer_bwd needs. */
moe_status moe_layer_fwd(const moe_config* cfg, const moe_weights* w, const void* x, void* y,
                         const moe_saved* saved, void* ws, size_t ws_bytes, moe_stream_t stream);

/* Backward of the combine (token-gradient routing, the reverse of the combine
 * all-to-all in "Backward walks the same path in reverse"):
 *   dy_perm[row_of[t,j]] = gates[t,j] * dy[t];  dg[t,j] = <dy[t], y_perm[row_of[t,j]]>
 * (0 for dropped assignments); pad rows of dy_perm are zeroed; and the logit
 * gradient dl [T, E] (float32): k > 1 -> dl[t, ids_j] = g_j (dg_j - sum_i g_i dg_i)
 * and 0 elsewhere; k = 1 -> dl[t, :] = g dg (onehot(ids_0) - probs[t, :]).
 * probs may be NULL when k > 1. */
moe_status moe_combine_bwd(const moe_config* cfg, const void* dy, const void* y_perm, const int32_t* ids,
                           const int32_t* row_of, const float* gates, const float* probs,
                           const int32_t* counts, const int32_t* offsets, void* dy_perm, float* dg, float* dl,
                           moe_stream_t stream);

/* Expert backward as grouped GEMMs (dgrad and wgrad):
 *   dH = dY_e W2_e^T;  da = dH * b * s * (1 + a (1 - s)), s = sigmoid(a);  db = dH * silu(a)
 *   dx_perm = da W1_e^T + db W3_e^T
 *   dW1_e (+)= X_e^T da;  dW3_e (+)= X_e^T db;  dW2_e (+)= H_e^T dY_e     (float32)
 * accumulate = 0 overwrites dW1/dW3/dW2, 1 adds to them (gradient
 * accumulation over micro-batches).  da and db are caller scratch of shape
 * [max_rows, f]. */
moe_status moe_grouped_ffn_bwd(const moe_config* cfg, const void* x_perm, const void* a, const void* b,
                               const void* h, const void* dy_perm, const int32_t* counts, const int32_t* offsets,
                               const void* W1, const void* W3, const void* W2, void* da, void* db, void* dx_perm,
                               float* dW1, float* dW3, float* dW2, int accumulate, moe_stream_t stream);

/* Auxiliary load-balancing loss of the router and its logit gradient.  The
 * tutorial's MoE configuration example names an "aux_loss" coefficient
 * (distributed-training tutorial, "The Conflict Between EP and TP") without a
 * formula; the usual expert-balance form is taken:
 *   f_e = (assignments (t, j) with ids[t,j] = e, before the capacity drop) / (T k)
 *   P_e = (1/T) sum_t probs[t,e]
 *   L   = c * E * sum_e f_e P_e,          c = cfg->aux_loss_coeff
 * f is a count and carries no gradient, so
 *   dl[t,e'] += c * E / T * probs[t,e'] * (f_e' - sum_e f_e probs[t,e]).
 * probs [T, E] fp32 and ids [T, k] int32 as moe_router_topk writes them; dl
 * [T, E] fp32 is updated in place (moe_combine_bwd's output); *loss (device
 * fp32, may be NULL) receives L.  Sums run in a fixed order (bitwise
 * reproducible).  ws must hold moe_workspace_size(cfg, 1).  When the
 * coefficient is 0 (or T = 0) dl is left as it is and *loss, if given, is set
 * to 0. */
moe_status moe_aux_loss(const moe_config* cfg, const float* probs, const int32_t* ids, float* loss, float* dl,
                        void* ws, size_t ws_bytes, moe_stream_t stream);

/* Inverse permutation of the token gradient plus the router backward ("Its
 * gradient behaves like any other shared parameter", gpu_expert_parallel page):
 *   dx[t] = sum over kept j of dx_perm[row_of[t,j]] + dl[t] W_r^T
 *   dW_r (+)= x^T dl        (float32, fixed summation order; no bias gradient)
 * ws must hold moe_workspace_size(cfg, 1). */
moe_status moe_unpermute_dx_router_bwd(const moe_config* cfg, const void* x, const void* dx_perm,
                                       const int32_t* row_of, const float* dl, const float* W_r, void* dx,
                                       float* dW_r, int accumulate, void* ws, size_t ws_bytes,
                                       moe_stream_t stream);

/* Whole backward from the state saved by moe_layer_fwd (no re-routing):
 * moe_combine_bwd, moe_aux_loss (when cfg->aux_loss_coeff > 0; saved->probs is
 * then required for every k and grads->aux_loss may receive the loss),
 * moe_grouped_ffn_bwd, moe_unpermute_dx_router_bwd.
 * grads receives dW_r, dW1, dW3, dW2 (accumulate as above); dx [T, d] in dtype. */
moe_status moe_layer_bwd(const moe_config* cfg, const moe_weights* w, const void* x, const void* dy,
                         const moe_saved* saved, void* dx, const moe_grads* grads, int accumulate, void* ws,
                         size_t ws_bytes, moe_stream_t stream);

/* Bytes of device memory the library reserves, on every GPU that loads it and
 * until the process exits, for moe_router_topk_noalloc. */
#define MOE_NOALLOC_SCRATCH_BYTES (4u << 20)

/* moe_router_topk for callers that cannot allocate device memory: a plugin
 * hosted by a program that owns every allocation, a path whose memory budget
 * is fixed at start-up, or a latency-critical loop that cannot afford the
 * implicit device synchronisation of cudaMalloc/cudaFree.  No workspace is
 * passed; the routing histograms, their scan and (bf16 layers of at least
 * 128 tokens) the three bf16 parts of W_r live in a static device array of
 * MOE_NOALLOC_SCRATCH_BYTES owned by the library (the pages have no
 * counterpart of this entry point; it is a deployment convenience).
 * It runs the same kernels as moe_router_topk for the same layer, so
 * arguments, results (bit for bit) and errors are those of moe_router_topk,
 * plus MOE_ERR_WORKSPACE, returned before anything is queued, when the layer
 * needs more than MOE_NOALLOC_SCRATCH_BYTES of scratch:
 * 2 * E * k * ceil(T/64) * 4 bytes of histograms and scan, plus
 * 3 * E_pad * d * 2 bytes of W_r parts for bf16 layers with T >= 128
 * (E_pad = E rounded up to 16, 32, 64 or 128), plus under 2 KB of alignment
 * (E = 32, k = 4, d = 4096 fits up to about 210,000 tokens).  The call
 * allocates nothing.
 * The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call
 * before any stream capture.  Every call on a device shares the one array and
 * it keeps the previous call's contents (the kernels rewrite or clear all of
 * it they read), so calls that overlap on the GPU -- on two streams, or from
 * two host threads -- race and must be serialised by the caller. */
moe_status moe_router_topk_noalloc(const moe_config* cfg, const void* x, const float* W_r, const float* bias,
                                   int32_t* ids, float* gates, float* probs, int32_t* slot, int32_t* row_of,
                                   int32_t* src_token, int32_t* counts, int32_t* offsets, moe_stream_t stream);

/* ---- Operators around the layer in a transformer block ----
 * The block is out = x + dropout(layer(norm(x))): moe_norm_fwd in front of the
 * layer, moe_dropout_add behind it, their backward passes, and the whole layer
 * for the few tokens of a serving step.  (The pages have no counterpart.)
 * Rows are dense; x, y, dy, dx, out and the residuals use `dtype` (moe_dtype)
 * and are 16-byte aligned, gamma, beta, the statistics and dgamma, dbeta are
 * float32.  1 <= d <= 65536, of any parity; rows * d <= 2^40. */

/* Most tokens of one moe_layer_decode call. */
#define MOE_DECODE_MAX_T 64

/* Bytes of workspace that moe_layer_decode needs for cfg.  Host only; it
 * scales with the SM count of the current device, so ask with the device that
 * will run the layer current. */
moe_status moe_decode_workspace_size(const moe_config* cfg, size_t* bytes);

/* The whole layer for a few tokens (T <= MOE_DECODE_MAX_T) in one kernel:
 *   y[t] = residual[t] + sum over kept j of gates[t,j] * (silu(x_t W1_e) * (x_t W3_e)) W2_e,
 * e = ids[t, j].  Routing, ties, gates, capacity and dropped assignments are
 * those of moe_router_topk; residual (NULL: none), ids and gates (NULL: not
 * wanted) as there.  Only the weights of experts with kept rows are read.  a
 * and b are fp32 sums and are not rounded to the activations' type, so y
 * carries one rounding to it.
 * Deterministic.  It is a cooperative launch of one block an SM for bf16 and of
 * two for float32: on a GPU that other streams keep busy it starts when all its
 * blocks fit.  Calls that may overlap want a workspace each.  residual may be y;
 * x must not overlap y. */
moe_status moe_layer_decode(const moe_config* cfg, const moe_weights* w, const void* x, const void* residual, void* y,
                            int32_t* ids, float* gates, void* ws, size_t ws_bytes, moe_stream_t stream);

/* Layer norm of each row:
 *   mean = sum(x) / d;  rstd = 1 / sqrt(sum((x - mean)^2) / d + eps)
 *   y = (x - mean) * rstd * gamma + beta
 * with fp32 statistics.  mean and rstd [rows] may be NULL (inference).  y may
 * be x.  eps >= 0. */
moe_status moe_norm_fwd(int64_t rows, int32_t d, int32_t dtype, const void* x, const float* gamma, const float* beta,
                        float eps, void* y, float* mean, float* rstd, moe_stream_t stream);

/* Bytes of workspace that moe_norm_bwd needs: partial sums of dgamma and
 * dbeta, at most two rows of d an SM, four where d > 8192.  Host only; device as
 * above. */
moe_status moe_norm_workspace_size(int64_t rows, int32_t d, size_t* bytes);

/* Backward of moe_norm_fwd, n = (x - mean) * rstd, v = dy * gamma:
 *   dx = rstd * (v - sum(v) / d - n * sum(v n) / d) + dres
 *   dgamma (+)= sum over rows of dy * n;  dbeta (+)= sum over rows of dy
 * dres (NULL: none) is the gradient that reaches x past the norm, on the
 * residual branch; dx may be x, dy or dres.  accumulate as in moe_layer_bwd.
 * Sums run in an order fixed by the sizes and the device. */
moe_status moe_norm_bwd(int64_t rows, int32_t d, int32_t dtype, const void* x, const void* dy, const float* gamma,
                        const float* mean, const float* rstd, const void* dres, void* dx, float* dgamma, float* dbeta,
                        int accumulate, void* ws, size_t ws_bytes, moe_stream_t stream);

/* Dropout of n elements behind the layer, with the residual added:
 *   out[i] = residual[i] + (u_i >= cut ? y[i] * 65536 / (65536 - cut) : 0)
 * cut = floor(65536 p + 1/2); 0 <= p < 1 and cut < 65536.  u_i are 16-bit
 * draws of Philox-4x32-10: element i takes 16-bit part i % 8 (low half of a
 * 32-bit word first) of the block whose counter is the 64-bit pair
 * (i / 8, offset) and whose key is seed.  The mask depends on (seed, offset, i)
 * alone and is never stored: give each layer and step its own offset.  A
 * dropped element contributes 0 whatever y[i] is.  residual may be NULL; out
 * may be y or residual. */
moe_status moe_dropout_add(int64_t n, int32_t dtype, const void* y, const void* residual, void* out, float p,
                           uint64_t seed, uint64_t offset, moe_stream_t stream);

/* Its gradient, with the mask drawn again from the same seed and offset:
 *   dy[i] = u_i >= cut ? dout[i] * 65536 / (65536 - cut) : 0
 * (the residual's gradient is dout itself).  dy may be dout. */
moe_status moe_dropout_bwd(int64_t n, int32_t dtype, const void* dout, void* dy, float p, uint64_t seed,
                           uint64_t offset, moe_stream_t stream);

/* ---- From blocks to a training step ----
 * The residual path between two blocks with the norms on either side of it,
 * the loss at the end of the stack, and the clipping of the accumulated
 * gradients.  (The pages have no counterpart.)  Conventions as above: dense
 * rows, tensors of `dtype` 16-byte aligned unless a parameter says otherwise,
 * float32 vectors 4-byte aligned.  A workspace's contents are of one call alone;
 * calls that may overlap want one each. */

/* The residual path between two blocks, per row t and channel c:
 *   u   = y * ry * gamma_post,  ry = 1 / sqrt(sum(y^2) / d + eps)     (gamma_post NULL: u = y)
 *   out = residual_scale * x + branch_scale * row_gate[t] * gate[c] * u   (a gate that is NULL is 1; y NULL: no branch)
 *   h   = out * ro * gamma_next,  ro = 1 / sqrt(sum(out^2) / d + eps)  (gamma_next NULL: no h)
 * y is the block's output, x the residual stream in front of it, h the next
 * block's input.  Without y it is the norm in front of the first block, without
 * gamma_next the path behind the last.  Squares are summed in fp32. */
typedef struct {
  int64_t rows;
  int32_t d;                 /* 1 <= d <= 65536, rows * d <= 2^40 */
  int32_t dtype;             /* of x, y, out, h and their gradients */
  const float* gamma_post;   /* [d] or NULL */
  const float* gamma_next;   /* [d] or NULL */
  const float* gate;         /* [d] or NULL: a gate of each channel */
  const float* row_gate;     /* [rows] or NULL: a gate of each row */
  float residual_scale;
  float branch_scale;
  float eps;                 /* >= 0 */
} moe_residual_norm;

/* Gradients of the parameters, float32; each NULL where it is not wanted, and
 * where the forward has no such parameter. */
typedef struct {
  float* dgamma_post;  /* [d] */
  float* dgamma_next;  /* [d] */
  float* dgate;        /* [d] */
  float* drow_gate;    /* [rows], overwritten whatever `accumulate` says */
} moe_residual_norm_grads;

/* Writes out and h.  out may be NULL where it is not wanted; h is required with
 * gamma_next and NULL without.  rstd_post and rstd_next [rows] (ry and ro) are
 * kept for the backward, or NULL.  h is formed from out before its rounding.
 * out and h may be x or y. */
moe_status moe_residual_norm_fwd(const moe_residual_norm* p, const void* x, const void* y, void* out, void* h,
                                 float* rstd_post, float* rstd_next, moe_stream_t stream);

/* Bytes of workspace that moe_residual_norm_bwd needs.  Host only; it scales
 * with the SM count of the current device. */
moe_status moe_residual_norm_workspace_size(int64_t rows, int32_t d, size_t* bytes);

/* Backward of moe_residual_norm_fwd from out and y as they are in memory and
 * the kept ry and ro.  n = out ro, m = y ry (m = y without gamma_post):
 *   D  = dout + ro (v - n sum(v n) / d),  v = dh gamma_next
 *   dx = residual_scale D;  G = branch_scale row_gate gate D;  w = G gamma_post
 *   dy = ry (w - m sum(w m) / d)   (G without gamma_post)
 *   dgamma_next (+)= sum over rows of dh n;  dgamma_post (+)= sum over rows of G m
 *   dgate (+)= sum over rows of branch_scale row_gate D u
 *   drow_gate[t] = sum over channels of branch_scale gate D u
 * dout (NULL: none) is the gradient that reaches out past the next norm; dh is
 * required with gamma_next.  dx may be NULL, dout or dh; dy may be dh or dout. out and
 * rstd_next are read with gamma_next only, y and dy are required where the
 * forward had a branch and NULL where it had none.  accumulate as in
 * moe_layer_bwd.  Sums run in an order fixed by the sizes and the device. */
moe_status moe_residual_norm_bwd(const moe_residual_norm* p, const void* out, const void* y, const void* dh,
                                 const void* dout, const float* rstd_post, const float* rstd_next, void* dx, void* dy,
                                 const moe_residual_norm_grads* grads, int accumulate, void* ws, size_t ws_bytes,
                                 moe_stream_t stream);

/* One gradient tensor: n elements of `dtype` at src, aligned to their own size. */
typedef struct {
  const void* src;
  void* dst;      /* receives the clipped gradient: src itself, another tensor of n elements, or NULL (norm only) */
  int64_t n;      /* 0 <= n <= 2^40 */
  int32_t dtype;  /* moe_dtype */
} moe_grad;

/* Most tensors of one moe_clip_grads call. */
#define MOE_CLIP_MAX_TENSORS 65536

/* Bytes of workspace that moe_clip_grads needs for `count` tensors.  Host only;
 * device as above. */
moe_status moe_clip_workspace_size(int32_t count, size_t* bytes);

/* The 2-norm of all tensors together, and the gradients clipped to it:
 *   norm = sqrt(sum over tensors of sum(src^2));  dst = src * min(1, max_norm / norm)
 * `grads` is a HOST array, read during the call alone.  *norm is a device
 * float.  max_norm is positive; INFINITY clips nothing.  A norm that is not
 * finite (a gradient holds an infinity or a NaN, or the norm itself passes
 * float32) clips nothing either: dst = src, and the caller sees *norm.  Where
 * nothing is clipped a tensor whose dst is its src is not written.  Squares are summed
 * without overflow or underflow whatever the values, in an order fixed by the
 * sizes, each src's place modulo 16 bytes and the device (elsewhere modulo 16 the
 * same values may give a norm whose last bit differs); subnormal float32 gradients
 * count.  A dst must not overlap another tensor's src or dst, or its own src but for
 * being the same (MOE_ERR_INVALID_ARG). */
moe_status moe_clip_grads(const moe_grad* grads, int32_t count, float max_norm, float* norm, void* ws, size_t ws_bytes,
                          moe_stream_t stream);

/* Softmax cross entropy over a vocabulary of V, x [T, d] and W [V, d] of `dtype`, whose
 * logits z = x W^T are formed a piece at a time and never kept:
 *   lse[t] = log sum_v exp(z[t, v]);  loss[t] = lse[t] - z[t, labels[t]]
 * labels [T] int32.  A token whose label is negative is ignored: loss and lse are
 * 0, whatever its row of x holds.  A label >= V is ignored too and recorded in
 * the device error word.  total (NULL: not wanted) receives two floats: the sum
 * of the losses and the number of labelled tokens.  0 <= T <= 2^24,
 * 1 <= V <= 2^24, T V <= 2^44, 1 <= d <= 65536, d a multiple of 8 for MOE_BF16
 * and of 4 for MOE_F32.  Infinities in a float32 W count as the largest bf16 of
 * their sign, and a float32 x with an infinity has no finite loss.  A logit of -inf adds
 * nothing; with one of +inf (or past float32) lse is inf and the loss inf, or NaN
 * where it is the label's.  Products are added up in fp32, but cut off and not
 * rounded over d of 1024 at a time (512 of MOE_F32; 256 of at most 64 MOE_BF16
 * tokens): some 1e-6 of the sum of their magnitudes, 2^-17 at most.  Deterministic. */
moe_status moe_vocab_loss_fwd(int32_t T, int32_t d, int32_t V, int32_t dtype, const void* x, const void* W,
                              const int32_t* labels, float* loss, float* lse, float* total, void* ws, size_t ws_bytes,
                              moe_stream_t stream);

/* Bytes of workspace of moe_vocab_loss_fwd (training = 0) or of both calls
 * (training = 1).  As many bytes do for any fewer tokens too, with the same d, V
 * and dtype.  MOE_F32 calls hold W in bf16 parts there, 6 bytes an element (but for
 * the forward of few tokens: up to 48; 24, 12 and none of d past 13312, 26624 and
 * 53248); the backward holds up to 2^28 values of dz, 2 bytes for each of its 1 to 3
 * parts.  Host only; device as above. */
moe_status moe_vocab_loss_workspace_size(int32_t T, int32_t d, int32_t V, int32_t dtype, int training, size_t* bytes);

/* Its gradient, the logits formed again:
 *   dz[t, v] = dloss[t] (exp(z[t, v] - lse[t]) - [v = labels[t]])   (0 for ignored tokens)
 *   dx = dz W [T, d] in dtype;  dW (+)= dz^T x [V, d] in dw_dtype
 * dloss [T] is the gradient that reaches each loss; NULL is that of the mean
 * over the labelled tokens.  dw_dtype is MOE_F32, or MOE_BF16 in a bf16 call;
 * in a bf16 call dz is held in 16 significant bits for a float32 dW and in 8 for
 * dx and a bf16 dW.  dx or dW may be NULL, not both.
 * accumulate as in moe_layer_bwd, for dW. */
moe_status moe_vocab_loss_bwd(int32_t T, int32_t d, int32_t V, int32_t dtype, int32_t dw_dtype, const void* x,
                              const void* W, const int32_t* labels, const float* lse, const float* dloss, void* dx,
                              void* dW, int accumulate, void* ws, size_t ws_bytes, moe_stream_t stream);

/* Waits for the current device to finish, then reads the device error word:
 * *code is MOE_OK, MOE_ERR_DEVICE_CHECK or MOE_ERR_TIMEOUT, *detail says which
 * kernel and check; clear != 0 resets the word.  Either output may be NULL. */
moe_status moe_get_device_error(int32_t* code, int32_t* detail, int clear);

/* Self-test of failure detection (the pages have no counterpart; it checks
 * this library's own safeguard).  Every mbarrier wait in the tensor-core
 * kernels gives up after a time limit, records MOE_ERR_TIMEOUT in the device
 * error word, drains and exits, so a stalled pipeline is reported rather than
 * hanging the GPU.  This launches one thread that waits with that same helper
 * on a barrier nothing arrives at (arrive = 0) or one that another warp
 * arrives at (arrive = 1, the control), giving up after limit_ns nanoseconds
 * (1e6 <= limit_ns <= 2e9).  Afterwards moe_get_device_error reports
 * MOE_ERR_TIMEOUT (arrive = 0) or MOE_OK (arrive = 1); the GPU stays usable. */
moe_status moe_selftest_bounded_wait(int64_t limit_ns, int arrive, moe_stream_t stream);

/* Kernel launches the library has issued in this process (all devices). */
uint64_t moe_launch_count(void);

/* Optional per-kernel timing with CUDA events recorded on the launch stream
 * around every kernel.  moe_profiler_enable(1) clears earlier records and
 * starts recording; moe_profiler_enable(0) stops.  moe_profiler_read
 * synchronises on the recorded events and fills, for kernel id 0 <= id <
 * moe_kernel_kinds(), the launches and total milliseconds. */
moe_status moe_profiler_enable(int on);
int32_t moe_kernel_kinds(void);
/* Restricts the profiler to launches of kernel kind id (0 <= id <
 * moe_kernel_kinds()), or to every kind when id < 0 (the default).  Applies to
 * launches issued after the call; records already taken are kept. */
moe_status moe_profiler_filter(int32_t id);
const char* moe_kernel_name(int32_t id);
/* NVTX ranges for timeline tools (off by default; the pages have no
 * counterpart).  While on, every kernel launch is bracketed by an NVTX range
 * named after its kernel kind (moe_kernel_name) and every moe_layer_fwd /
 * moe_layer_bwd call by a range of that name, pushed and popped on the
 * calling host thread, so an nsys or ncu timeline can be cut by layer step and
 * kernel.  Without a tool attached a range costs a few nanoseconds.  Host only. */
moe_status moe_nvtx_enable(int on);
moe_status moe_profiler_read(int32_t id, int64_t* launches, double* total_ms);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
