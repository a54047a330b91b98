/*
 * libttc: forward and backward of a rank-gated tensor-train (TT) linear layer
 * on one NVIDIA GB300 GPU (sm_103a).
 *
 * The layer (CoMERA project page, "Learn the ranks while training", figure of
 * a tensor-train layer with rank-control diagonals):
 *   W (M x N), N = n_1*...*n_d, M = m_1*...*m_d, is a chain of 2d cores
 *   G_k of shape (r_{k-1}, s_k, r_k), r_0 = r_2d = 1, input modes first:
 *   s = (n_1..n_d, m_1..m_d).  A diagonal D_k sits on every internal link
 *   k = 1..2d-1; the rank of a link is the number of nonzeros of D_k, and a
 *   zero entry drops the matching slice of both neighbouring cores.
 *   With j = (j_1..j_d), i = (i_1..i_d) row-major (first mode most
 *   significant):
 *     W[i,j] = G_1[0,j_1,:] D_1 G_2[:,j_2,:] ... D_d ... G_2d[:,i_d,0]
 *   forward   y[t,i] = sum_j W[i,j] x[t,j]                (no bias)
 *   backward  for L = sum dy[t,i] y[t,i]:  dx = dy W,  dG_k = dL/dG_k,
 *             dD_k = dL/dD_k, except that dD_k[a] is returned as 0 where
 *             D_k[a] == 0 (the rank-truncated layer has no such parameter).
 * The contraction order is the one of the project page, "Making small tensor
 * operations fast on GPUs", bullet "One contraction order for both passes":
 * the input-side cores are merged into A (N x r_d), the output-side cores
 * into B (r_d x M), and x is contracted through them
 * (y = ((x A) diag(D_d)) B).
 *
 * Conventions for every call:
 *  - All device pointers are plain CUDA device addresses owned by the caller.
 *    The library allocates no device memory at run time; it uses the
 *    caller's workspace.  It does hold a few module-scope device arrays,
 *    which every GPU that loads the library keeps until the process exits,
 *    whether or not it calls the functions that use them: the
 *    tt_forward_noalloc scratch (32 MiB), the status words and the TT-matrix
 *    lookup's unit constants (a few bytes).
 *  - Calls on different streams may overlap on the GPU when each has its own
 *    workspace: everything a call writes (grid-barrier counters included)
 *    lives in its workspace or its outputs.  Calls that share a workspace
 *    must be ordered (one stream, or events).
 *  - stream is a cudaStream_t passed as void* (NULL = legacy default stream).
 *    Calls only enqueue work; none synchronises, except
 *    tt_get_device_status.
 *  - Argument errors are reported before anything is enqueued.  A failed
 *    launch returns TT_ERR_CUDA.  Errors found on the device (a bounded wait
 *    that ran out, a failed consistency check) are recorded in a status word
 *    that the library keeps in device memory, one per GPU (a module-scope
 *    variable, zero at load), and read back by tt_get_device_status.
 *  - Activations of the TT layers: x is (T, N), y is (T, M), dy is (T, M), dx is (T, N), all
 *    row-major, dense, in the plan's activation type (f32 or bf16), 16-byte
 *    aligned.  Cores, diagonals and their gradients are f32.
 *  - Packed parameters: one f32 buffer holding G_1..G_2d, each
 *    (r_{k-1}, s_k, r_k) row-major, followed by D_1..D_{2d-1}
 *    (tt_param_layout gives the offsets).  dparams has the same layout.
 */
#ifndef TTC_H
#define TTC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define TT_MAX_D 4 /* order 2d <= 8 */

typedef enum tt_status {
  TT_OK = 0,
  TT_ERR_INVALID_ARG = 1, /* bad descriptor, NULL or misaligned pointer, T < 0 */
  TT_ERR_UNSUPPORTED = 2, /* valid layer the library has no kernel for */
  TT_ERR_WORKSPACE = 3,   /* workspace missing or smaller than tt_workspace_size */
  TT_ERR_CUDA = 4,        /* a CUDA runtime call or launch failed */
  TT_ERR_TIMEOUT = 5,     /* a bounded device-side wait ran out (device status) */
  TT_ERR_DEVICE = 6       /* a device-side consistency check failed (device status) */
} tt_status;

/* Activation types.  TT_DT_E4M3: x and dy are one-byte OCP FP8 E4M3
 * ("e4m3fn": bias 7, 3 mantissa bits, largest finite 448, NaN 0x7F/0xFF)
 * codes, y and dx are bf16; the cores, diagonals and gradients stay fp32 and
 * every product accumulates in fp32.  This is the FP8/FP32 mixed precision of
 * the CoMERA poster digest (its FP8-mix speedup table and the mixed-precision
 * DLRM results), read as FP8 storage of the activations. */
typedef enum tt_dtype { TT_DT_F32 = 0, TT_DT_BF16 = 1, TT_DT_E4M3 = 2 } tt_dtype;

/* flags of tt_desc */
#define TT_ACCUMULATE 1u /* backward adds into dparams instead of overwriting */
/* The backward reuses the merged cores that the forward left in the
 * workspace, as the CoMERA project page describes for its contraction path
 * (the forward keeps its intermediate results for the backward pass).  The
 * caller guarantees that a tt_forward call with the same plan, the same
 * params and the same workspace came before, with nothing else using the
 * workspace in between; then tt_backward skips re-merging the cores (a
 * backward of T == 0 tokens ignores the flag: a forward of none does no work).  In an
 * FFN plan (both descs must carry the same flags) each layer then keeps its
 * merges in a workspace region of its own. */
#define TT_REUSE_MERGE 2u
/* Implies TT_REUSE_MERGE.  On the tensor-core path (bf16 or E4M3 activations)
 * the forward also keeps z' = (x A) diag(D_d) for every token in the
 * workspace (bf16, T x 64 values: 128 more bytes a token, counted by
 * tt_workspace_size), and the backward reads it instead of computing x A
 * again, so it streams x once instead of twice.  The caller guarantees in
 * addition that the backward gets the forward's x and T.  The f32 path
 * ignores it.  In a bf16 FFN plan (and a bf16 multi-layer plan) every layer
 * keeps its z' the same way; without the flag the fused FFN and multi-layer
 * backward compute them first (one more pass over x). */
#define TT_REUSE_Z 4u
/* Bit-reproducible gradients: the same inputs give the same dx and dparams
 * bit for bit, run after run, on a given GPU model.  Every sum over tokens
 * is taken in a fixed order: 128-token tiles, each CTA adding its tiles in
 * order into a slot of its own (TMA bulk add with completion awaited between
 * tiles), the slots then summed in CTA order by one more kernel; the merge
 * backward runs without atomic K splits (split partials reduced in split
 * order, one more engine phase); the f32 path reduces without atomics; a
 * bf16 FFN pair runs layer by layer.  Costs workspace (up to 160 slots of
 * (N + M + 4) x 64 floats, counted by tt_workspace_size) and time.  The
 * CoMERA pages do not discuss reproducibility; this is the training
 * requirement of a library boundary. */
#define TT_DETERMINISTIC 8u

typedef struct tt_desc {
  int d;                        /* 1..TT_MAX_D: number of input (= output) modes */
  int in_modes[TT_MAX_D];       /* n_1..n_d, each >= 1 */
  int out_modes[TT_MAX_D];      /* m_1..m_d, each >= 1 */
  int ranks[2 * TT_MAX_D + 1];  /* r_0..r_2d; r_0 = r_2d = 1, others >= 1 */
  int act;                      /* tt_dtype of x, y, dx, dy (E4M3: y, dx bf16) */
  unsigned flags;               /* TT_ACCUMULATE | TT_REUSE_MERGE | TT_REUSE_Z | TT_DETERMINISTIC */
} tt_desc;

typedef struct tt_plan_s tt_plan_t; /* opaque, immutable host object */

/* Rank caps read off the printed rank table (project page, "Results",
 * "Internal tensor-train ranks of each layer in one encoder block"):
 * r_k = min(R, prod s_<=k, prod s_>k), r_0 = r_2d = 1.  ranks receives 2d+1
 * values.  Host only. */
tt_status tt_default_ranks(int d, const int* in_modes, const int* out_modes, int R,
                           int* ranks);

/* Validate desc and build a plan (host only; no device work, no allocation on
 * the device).  *out is owned by the caller and freed with tt_destroy.
 * TT_ERR_INVALID_ARG for a malformed desc (a rank outside 1..4096 among
 * them); TT_ERR_UNSUPPORTED for N or M above 2^20 or a merged intermediate
 * (the packed parameters, a prefix product of the cores, the merged A or B)
 * of 2^31 elements or more; TT_ERR_UNSUPPORTED as well for an E4M3 layer
 * outside the fused tensor-core kernels' shapes (N, M multiples of 16 and at
 * least 128, middle rank r_d <= 64): E4M3 has no other path. */
tt_status tt_plan(const tt_desc* desc, tt_plan_t** out);

/* FFN pair y = TT_down(GELU(TT_up(x))) with GELU(h) = h Phi(h).  Up's
 * output width must equal down's input width and both must use the same act
 * type and flags (F32 or BF16; E4M3 gives TT_ERR_UNSUPPORTED).  A bf16 pair
 * whose layers fit the tensor-core kernels runs fused, h never leaving the
 * SM, with Phi(h) = (1 + tanh(sqrt(2/pi)(h + 0.044715 h^3))) / 2 (Hendrycks
 * and Gimpel's tanh form; |Phi error| <= 1.8e-4, below a bf16 rounding of
 * h); every other pair evaluates erf to within 1.5e-7 (Abramowitz and
 * Stegun 7.1.26). */
tt_status tt_ffn_plan(const tt_desc* up, const tt_desc* down, tt_plan_t** out);

void tt_destroy(tt_plan_t* plan);

/* Offsets (in floats) of every core and diagonal inside the packed parameter
 * buffer: core_off receives 2d values, diag_off 2d-1, *n_floats the total.
 * For an FFN plan these describe the up layer (use tt_ffn_param_layout), for
 * a multi-layer plan its first layer (use tt_multi_param_layout). */
tt_status tt_param_layout(const tt_plan_t* plan, size_t* core_off, size_t* diag_off,
                          size_t* n_floats);
tt_status tt_ffn_param_layout(const tt_plan_t* plan, int layer /*0 up, 1 down*/,
                              size_t* core_off, size_t* diag_off, size_t* n_floats);

/* Bytes of device workspace a forward or backward call with T tokens needs
 * (the same value serves both).  The workspace must be 256-byte aligned. */
tt_status tt_workspace_size(const tt_plan_t* plan, int64_t T, size_t* bytes);

/* y = x W^T for T tokens.  T == 0 is a no-op. */
tt_status tt_forward(const tt_plan_t* plan, int64_t T, const void* x, const float* params,
                     void* y, void* ws, size_t ws_bytes, void* stream);

/* dx = dy W and dparams = dL/dparams (overwritten, or added to under
 * TT_ACCUMULATE).  Recomputes what the forward computed; needs no state from
 * a forward call.  T == 0 writes zero gradients (or leaves them under
 * TT_ACCUMULATE). */
tt_status tt_backward(const tt_plan_t* plan, int64_t T, const void* x, const void* dy,
                      const float* params, void* dx, float* dparams, void* ws,
                      size_t ws_bytes, void* stream);

/* The forward above for callers that cannot allocate device memory (a
 * plain-C host or plugin without a device allocator of its own, or a process
 * that must not call cudaMalloc once running).  The CoMERA pages have no
 * counterpart of this call; it only changes where scratch comes from.
 * Scratch is a fixed 32 MiB device array inside the library, held on every
 * GPU that loads it until exit; the caller passes only inputs and outputs.
 * Returns TT_ERR_WORKSPACE when tt_workspace_size(plan, T) exceeds 32 MiB.
 * The first call on a device looks the array's address up (once per device)
 * and should come before any stream capture.  All calls share the array:
 * calls that overlap on the GPU race on it.  Nothing in it needs to start at
 * zero.  Otherwise behaves like tt_forward. */
tt_status tt_forward_noalloc(const tt_plan_t* plan, int64_t T, const void* x,
                             const float* params, void* y, void* stream);

/* FFN pair: params_up / params_down are the two packed buffers. */
tt_status tt_ffn_forward(const tt_plan_t* plan, int64_t T, const void* x,
                         const float* params_up, const float* params_down, void* y, void* ws,
                         size_t ws_bytes, void* stream);
tt_status tt_ffn_backward(const tt_plan_t* plan, int64_t T, const void* x, const void* dy,
                          const float* params_up, const float* params_down, void* dx,
                          float* dparams_up, float* dparams_down, void* ws, size_t ws_bytes,
                          void* stream);

/* ---- several layers on one input --------------------------------------------
 * Up to TT_MULTI_MAX layers that read the same x: the Q, K and V projections
 * of an encoder block's attention (CoMERA project page, "Results", rank
 * table: the attention rows, 768 x 768 at rank 30 each).  The results are
 * those of one tt_forward / tt_backward per layer, except that the backward
 * returns the sum dx = sum_g dy_g W_g (the gradient of x, which feeds every
 * layer).  A bf16 plan whose layers all fit the tensor-core kernels (and
 * without TT_DETERMINISTIC) runs every token pass as one kernel over all
 * layers, streaming x once for all of them (twice in a backward without
 * TT_REUSE_Z); otherwise the layers run one after another and dx is their
 * sum, taken in layer order.  params, y, dy, dparams are host arrays of n
 * device pointers, one per layer, in the descs' order. */
#define TT_MULTI_MAX 3
/* descs: n (1..TT_MULTI_MAX) layers with the same input modes, act type and
 * flags (else TT_ERR_INVALID_ARG); other errors as tt_plan. */
tt_status tt_multi_plan(const tt_desc* descs, int n, tt_plan_t** out);
/* The packed parameter layout of layer `layer` (0..n-1) of a multi plan. */
tt_status tt_multi_param_layout(const tt_plan_t* plan, int layer, size_t* core_off,
                                size_t* diag_off, size_t* n_floats);
tt_status tt_multi_forward(const tt_plan_t* plan, int64_t T, const void* x,
                           const float* const* params, void* const* y, void* ws,
                           size_t ws_bytes, void* stream);
tt_status tt_multi_backward(const tt_plan_t* plan, int64_t T, const void* x,
                            const void* const* dy, const float* const* params, void* dx,
                            float* const* dparams, void* ws, size_t ws_bytes, void* stream);

/* Rank-adaptive step [CoMERA project page, "Learn the ranks while
 * training": the early-stage objective L(G, D) + gamma S_hat(D) + beta ||G||^2,
 * with S_hat an l1 penalty on the diagonals (read here as sum_k |D_k|_1 over
 * every internal link) and ||G||^2 = sum_k ||G_k||_F^2].  Works in place on
 * one layer's packed params / dparams (the tt_param_layout layout, fp32,
 * device pointers), enqueued on `stream`:
 *   lr == 0: dparams += the penalty's sub-gradient:
 *            dG_k += (2 beta) G_k,  dD_k += gamma sign(D_k), sign(0) = 0;
 *            params untouched.
 *   lr > 0:  one proximal gradient step on the whole objective:
 *            G_k <- G_k - lr (dG_k + (2 beta) G_k),
 *            D_k <- soft_threshold(D_k - lr dD_k, lr gamma),
 *            soft_threshold(v, t) = sign(v) max(|v| - t, 0) (entries with
 *            |v| <= t become exactly +0: pruned, and compacted out by the
 *            next forward / backward); dparams untouched.
 * Every step is one float32 operation, rounded to nearest, in the order
 * written (no fused multiply-add).  TT_ERR_INVALID_ARG for a null pointer,
 * an FFN plan (update each layer with its own single-layer plan), or a
 * negative or non-finite gamma, beta or lr.  The CoMERA pages give no
 * optimiser; this is the plainest step on the objective they state. */
typedef struct tt_rank_opts {
  float gamma; /* weight of the l1 penalty on the diagonals, >= 0 */
  float beta;  /* weight of the squared l2 penalty on the cores, >= 0 */
  float lr;    /* step size, >= 0; 0 selects the gradient-only form */
} tt_rank_opts;
tt_status tt_rank_update(const tt_plan_t* plan, float* params, float* dparams,
                         const tt_rank_opts* opts, void* stream);

/* tt_backward followed by tt_rank_update on the same params / dparams, with
 * the step run as the last phase of the backward's merge program (after a
 * grid barrier that follows every read of params) instead of a launch of its
 * own: the early-stage objective's gradient (lr == 0: dparams = dL/dparams +
 * the penalty's sub-gradient) or one proximal step (lr > 0: params updated in
 * place, dparams = dL/dparams).  Arguments and errors as tt_backward and
 * tt_rank_update (params is written when lr > 0); a single-layer plan only.
 * The result equals the two calls in a row. */
tt_status tt_backward_rank_update(const tt_plan_t* plan, int64_t T, const void* x,
                                  const void* dy, float* params, void* dx, float* dparams,
                                  const tt_rank_opts* opts, void* ws, size_t ws_bytes,
                                  void* stream);

/* ---- TT-matrix (TTM) embedding lookup ---------------------------------------
 * [CoMERA project page, "Making small tensor operations fast on GPUs", bullet
 * "Embedding lookup without repeated work": keep only the unique rows of a
 * batch, contract neighbouring cores in pairs so each shared part is computed
 * once, and assemble the rows with one batched product; the table is in
 * tensor-train-matrix format (project page, "Learn the ranks while training";
 * poster digest, TT/TTM figure)].
 * The table E (V x Dm), V = prod m_k rows, Dm = prod n_k columns, is
 *     E[i, j] = F_1[0, i_1, j_1, :] D_1 F_2[:, i_2, j_2, :] D_2 ... F_d[:, i_d, j_d, 0]
 * with i = (i_1..i_d) and j = (j_1..j_d) row-major (first mode most
 * significant).  Packed params: F_1..F_d, each (r_{k-1}, m_k, n_k, r_k)
 * row-major, then D_1..D_{d-1}, fp32 (tt_param_layout describes a TTM plan
 * too: d core offsets, d-1 diagonal offsets).  d is 2 or 3; ranks 1..64;
 * n_1 n_2 r_2 <= 8192, r_1 n_2 r_2 <= 16384 and Dm <= 8192 (else
 * TT_ERR_UNSUPPORTED). */
typedef struct tt_ttm_desc {
  int d;               /* 2 or 3 cores */
  int row_modes[4];    /* m_1..m_d (the vocabulary V = prod m_k, <= 2^24) */
  int col_modes[4];    /* n_1..n_d (the embedding width Dm = prod n_k) */
  int ranks[5];        /* r_0..r_d, r_0 = r_d = 1 */
  unsigned flags;      /* TT_ACCUMULATE (backward adds into dparams),
                          TT_REUSE_MERGE (see tt_ttm_lookup_backward) */
} tt_ttm_desc;
tt_status tt_ttm_plan(const tt_ttm_desc* desc, tt_plan_t** out);

/* out[b, :] = E[idx[b], :] for b < B (out: B x Dm fp32, row-major; idx:
 * int32 device array).  Each distinct row and each distinct (i_1, i_2)
 * prefix is computed once.  An index outside [0, V) is skipped (its output
 * row is left unwritten) and recorded in the device status word
 * (TT_ERR_DEVICE from tt_get_device_status).  Workspace: tt_workspace_size
 * with T = B.  B == 0 is a no-op. */
tt_status tt_ttm_lookup(const tt_plan_t* plan, int64_t B, const int32_t* idx,
                        const float* params, float* out, void* ws, size_t ws_bytes,
                        void* stream);

/* Gradients of L = <dout, lookup(idx)> (dout: B x Dm fp32): every dF_k and
 * dD_k into dparams (overwritten, or added to under TT_ACCUMULATE); repeated
 * indices add up.  dD_k[a] is 0 where D_k[a] == 0 (as for the TT layers).
 * Recomputes the forward's unique rows; needs no state from a lookup call.
 * Under TT_REUSE_MERGE it also takes the batch's distinct rows and prefixes
 * from the workspace instead of finding them again: the caller guarantees
 * that a tt_ttm_lookup with the same plan, the same idx and B and the same
 * workspace came before, with nothing but such backward calls using the
 * workspace in between.
 * Gradient sums are reduced with atomics (summation order not fixed). */
tt_status tt_ttm_lookup_backward(const tt_plan_t* plan, int64_t B, const int32_t* idx,
                                 const float* dout, const float* params, float* dparams,
                                 void* ws, size_t ws_bytes, void* stream);

/* After a lookup or backward on ws (synchronises stream): the number of
 * distinct rows and of distinct (i_1, i_2) prefixes of that batch. */
tt_status tt_ttm_stats(const tt_plan_t* plan, const void* ws, int64_t* unique_rows,
                       int64_t* unique_pairs, void* stream);

/* ---- layer normalisation ------------------------------------------------------
 * The normalisation between an encoder block's TT layers, with the residual
 * sum in front of it.  The CoMERA pages leave it uncompressed and do not
 * describe it; the definition is Ba, Kiros and Hinton's.  For a row t of N
 * values
 *   s = x + res  (s = x without res),   mean = sum_j s_j / N,
 *   rstd = 1 / sqrt(sum_j (s_j - mean)^2 / N + eps),
 *   y_j = (s_j - mean) rstd gamma_j + beta_j.
 * Row statistics and sums are fp32; y and s are rounded once, s after y was
 * computed from its unrounded value. */
typedef struct tt_norm_desc {
  int64_t N;      /* width of a row, 1 .. 2^20 */
  float eps;      /* > 0, finite */
  int act;        /* tt_dtype of x, res, s, y and their gradients: F32 or BF16 */
  unsigned flags; /* TT_ACCUMULATE: the backward adds into dgamma and dbeta */
} tt_norm_desc;
/* Host only.  TT_ERR_INVALID_ARG for a bad field, TT_ERR_UNSUPPORTED for E4M3
 * or N above 2^20. */
tt_status tt_norm_plan(const tt_norm_desc* desc, tt_plan_t** out);
/* T rows.  x, res, sum and y are (T, N), dense, 16-byte aligned; res may be
 * NULL (no residual), sum may be NULL (s not wanted); sum or y may be x or res
 * itself.  gamma and beta: N fp32 each, either may be NULL (1 and 0).
 * stats: T x 2 fp32 (mean, rstd of each row), for the backward; may be NULL.
 * Needs no workspace.  T == 0 is a no-op. */
tt_status tt_norm_forward(const tt_plan_t* plan, int64_t T, const void* x, const void* res,
                          const float* gamma, const float* beta, void* sum, void* y,
                          float* stats, void* stream);
/* Gradients of L = <dy, y> + <dsum, s>.  s: what was normalised (x, or the
 * forward's sum); stats: the forward's.  With g = dy gamma, h = (s - mean) rstd:
 *   dx = rstd (g - sum_j g_j / N - h sum_j g_j h_j / N) + dsum   (the gradient
 * of x, and of res: they are equal), dgamma = sum_t dy h, dbeta = sum_t dy.
 * dsum (the gradient that reaches s along the residual path) may be NULL;
 * dgamma and dbeta (fp32, overwritten, or added to under TT_ACCUMULATE) may
 * each be NULL.  dx may be dy or dsum itself.  Sums over tokens are taken in a fixed order: the
 * same inputs give the same bits on a given GPU model.  Workspace:
 * tt_workspace_size(plan, T).  T == 0 writes zero dgamma and dbeta (or leaves
 * them under TT_ACCUMULATE). */
tt_status tt_norm_backward(const tt_plan_t* plan, int64_t T, const void* s, const void* dy,
                           const void* dsum, const float* gamma, const float* stats, void* dx,
                           float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                           void* stream);

/* ---- attention with a sliding window and first tokens that stay visible ------
 * The attention between the Q, K, V projections and O.  The CoMERA pages
 * leave it uncompressed; the definition is scaled dot-product attention
 * (Vaswani et al.) under the mask below.
 * Sequence b has queries q rows q_begin[b] .. q_end[b] and keys k rows
 * k_begin[b] .. k_end[b] (lq and lk of them).  Its query row t (0-based)
 * stands at position i = t + lk - lq: with lq == lk that is self-attention,
 * with lq < lk the queries are the last ones of a longer cache.  Key j
 * (0-based) is visible to it when
 *   (right < 0 or j <= i + right)  and  (left < 0 or j >= i - left or j < sinks)
 * so right = 0 is causal, left = W - 1 a window of W tokens, and the first
 * `sinks` tokens never leave it.  Query head h reads key head h / (heads /
 * kv_heads).  Over the visible j:
 *   z_j = scale q_i . k_j,  lse = log sum_j exp(z_j),  p_j = exp(z_j - lse),
 *   o_i = sum_j p_j v_j.
 * A row that sees no key gets o = 0 and lse = -infinity, and zero gradients.
 * Keys that no query of their sequence sees are not used: what they hold (a
 * cache's unwritten rows, NaN) reaches no output.  A key that some query sees
 * must hold finite values: the products are taken over tiles, where a weight of
 * zero times a value that is not finite is NaN, so such a value may reach every
 * query within 128 rows of one that sees it (in a backward, a query's q, o or
 * dout likewise every key within 128 of one that it sees).
 * Scores, softmax statistics and all sums are fp32: a weight's relative error grows
 * with its score, some 2^-22 |z| (a thousandth at scores of 5000).  With bf16 activations
 * the weights p (and in the backward z's gradient) are rounded to bf16 for
 * the tensor-core products. */
typedef struct tt_attn_desc {
  int heads;     /* query heads, 1 .. 1024 */
  int kv_heads;  /* key / value heads, a divisor of heads */
  int dim;       /* width of a head, 1 .. 256 */
  int left;      /* tokens to the left that stay visible; < 0: all */
  int right;     /* tokens to the right; < 0: all */
  int sinks;     /* first tokens that the left bound does not hide, >= 0 */
  float scale;   /* 0: 1 / sqrt(dim) */
  int act;       /* tt_dtype of q, k, v, o and their gradients: F32 or BF16 */
  unsigned flags; /* 0 */
} tt_attn_desc;
/* Host only.  TT_ERR_INVALID_ARG for a bad field, TT_ERR_UNSUPPORTED for E4M3
 * or dim above 256. */
tt_status tt_attn_plan(const tt_attn_desc* desc, tt_plan_t** out);

/* The rows of a batch's sequences.  The four arrays are device memory, B
 * int32 each; packed self-attention passes one array of B + 1 offsets as
 * begin and the same array + 1 as end, for queries and keys alike.  Query
 * ranges must not overlap; key ranges must not overlap in a backward.
 * max_q and max_k bound lq and lk (they size the launch).  A sequence with a
 * negative length, a row outside [0, Tq) / [0, Tk), or longer than max_q /
 * max_k is skipped (its rows left unwritten) and recorded in the device
 * status word (TT_ERR_DEVICE).  Rows of no sequence are left unwritten. */
typedef struct tt_attn_seqs {
  int B;                 /* sequences, 0 .. 2^20 */
  int max_q, max_k;      /* 0 .. 2^29 */
  int64_t Tq, Tk;        /* rows of the q and k buffers, < 2^31 */
  const int32_t* q_begin;
  const int32_t* q_end;
  const int32_t* k_begin;
  const int32_t* k_end;
} tt_attn_seqs;
/* A tensor of heads: element (t, h, c) is at p[t * row + h * head + c] (row
 * and head in elements, >= 0).  p is aligned to its type; the tensor-core kernels
 * additionally take p 16-byte aligned and, in bf16, row, head and dim
 * multiples of 8 with dim <= 128; anything else runs on the general kernels. */
typedef struct tt_heads {
  void* p;
  int64_t row, head;
} tt_heads;

/* Bytes of workspace (256-byte aligned) for a forward or a backward of seqs
 * (its device arrays are not read).  Either can be the larger: one buffer for
 * both passes takes the maximum of the two sizes. */
tt_status tt_attn_workspace_size(const tt_plan_t* plan, const tt_attn_seqs* seqs, int backward,
                                 size_t* bytes);
/* q and o: (Tq, heads, dim), k and v: (Tk, kv_heads, dim); lse: (heads, Tq)
 * fp32, may be NULL. */
tt_status tt_attn_forward(const tt_plan_t* plan, const tt_attn_seqs* seqs, const tt_heads* q,
                          const tt_heads* k, const tt_heads* v, const tt_heads* o, float* lse,
                          void* ws, size_t ws_bytes, void* stream);
/* Gradients of L = <dout, o>: dq, dk and dv (overwritten; the gradient of a
 * shared key head is the sum over its query heads), with o and lse as the
 * forward left them.  Every sum is taken in a fixed order. */
tt_status tt_attn_backward(const tt_plan_t* plan, const tt_attn_seqs* seqs, const tt_heads* q,
                           const tt_heads* k, const tt_heads* v, const tt_heads* o,
                           const float* lse, const tt_heads* dout, const tt_heads* dq,
                           const tt_heads* dk, const tt_heads* dv, void* ws, size_t ws_bytes,
                           void* stream);

/* ---- norm of queries and keys for each head, and their rotation by position ----
 * Between the Q, K projections and the attention.  The CoMERA pages do not
 * describe positions; the definitions are root mean square normalisation
 * (Zhang and Sennrich) of each head and rotary position embedding (Su et al.).
 * For a token at position pos and a head x of dim values, with a weight g of dim
 * values for all query heads and one for all key heads:
 *   u_c = x_c g_c / sqrt(sum_c x_c^2 / dim + eps)    (u = x when eps == 0)
 *   (y_a, y_b) = (u_a cos - u_b sin, u_a sin + u_b cos) of the angle pos f_i
 * for the pairs i < rot / 2, (a, b) = (i, i + rot / 2), or (2 i, 2 i + 1) when
 * interleaved; y_c = u_c for c >= rot.  f_i = base^(-2 i / rot), or freqs[i].
 * All arithmetic is fp32 and y is rounded once (finite values whose squares' sum is beyond
 * fp32 give zeros); angles are reduced to a turn without rounding (64-bit fractions of a
 * turn), so far positions keep theirs. */
typedef struct tt_rope_desc {
  int heads;           /* query heads, 1 .. 1024 */
  int kv_heads;        /* key / value heads, a divisor of heads */
  int dim;             /* width of a head, 1 .. 256 */
  int rot;             /* channels that are rotated: even, 0 .. dim */
  double base;         /* > 0; not read when freqs is given or rot == 0 */
  const double* freqs; /* host array of rot / 2 frequencies (radians a position) or NULL */
  int interleaved;     /* 0: pairs half a rotation apart; else neighbours */
  float eps;           /* >= 0, finite; 0: no norm (then rot > 0) */
  int act;             /* tt_dtype of q, k, v and their gradients: F32 or BF16 */
  unsigned flags;      /* TT_ACCUMULATE: the backward adds into dgq and dgk */
} tt_rope_desc;
/* Host only; freqs is copied.  TT_ERR_INVALID_ARG for a bad field,
 * TT_ERR_UNSUPPORTED for E4M3 or dim above 256. */
tt_status tt_rope_plan(const tt_rope_desc* desc, tt_plan_t** out);
/* T tokens (below 2^31) at positions pos (T int32, device; NULL: 0, 1, ..).
 * q, q_out: (T, heads, dim); k: (T, kv_heads, dim).  gq, gk: dim fp32 each, NULL for
 * ones (and NULL without a norm).  rows == NULL: k_out is (T, kv_heads, dim).
 * With rows (T int32, device): token t's keys go to row rows[t] of k_out,
 * (cache_rows, kv_heads, dim), the other rows stay as they are; a negative row is
 * skipped, one of cache_rows or more too and recorded in the device status word
 * (TT_ERR_DEVICE).  Rows that are not negative must differ from one another.  v and v_out
 * (both or neither): v's heads are copied to the rows of k_out's, unchanged.
 * q_out may be q, and without rows k_out may be k (the same strides).  Any strides
 * (tt_heads); pointers aligned to 16 bytes, with strides, rot / 2 and dim - rot that
 * are multiples of 8 and 16 values (bf16; 4 and 8 in f32), are fastest.  Needs no
 * workspace.  T == 0 is a no-op. */
tt_status tt_rope_forward(const tt_plan_t* plan, int64_t T, const int32_t* pos,
                          const tt_heads* q, const tt_heads* k, const float* gq,
                          const float* gk, const tt_heads* q_out, const tt_heads* k_out,
                          const tt_heads* v, const tt_heads* v_out, const int32_t* rows,
                          int64_t cache_rows, void* stream);
/* Gradients of L = <dq_out, q_out> + <dk_out, k_out> (of the form without rows): dq,
 * dk, and dgq, dgk (dim fp32 each, overwritten or added to under TT_ACCUMULATE; either
 * may be NULL, and both are without a norm).  q and k are the forward's inputs, not
 * read without a norm.  dq may be dq_out or q, dk dk_out or k (the same strides).
 * Sums over tokens and heads are taken in a fixed order: the same inputs give the
 * same bits on a given GPU model.  Workspace: tt_workspace_size(plan, T) bytes or more (it
 * never falls as T grows), 256-byte aligned (none without a norm).  T == 0 writes zero dgq
 * and dgk (or leaves them). */
tt_status tt_rope_backward(const tt_plan_t* plan, int64_t T, const int32_t* pos,
                           const tt_heads* q, const tt_heads* k, const float* gq,
                           const float* gk, const tt_heads* dq_out, const tt_heads* dk_out,
                           const tt_heads* dq, const tt_heads* dk, float* dgq, float* dgk,
                           void* ws, size_t ws_bytes, void* stream);

/* ---- dropout ---------------------------------------------------------------------
 * [Srivastava et al.]  An element stays with probability 1 - p and is then scaled by
 * 1 / (1 - p), else it becomes 0 (whatever it held).  Which ones stay is a function of
 * the element's index i in its dense tensor, the seed, the offset and the site, computed
 * where it is needed and never stored: Philox 4x32 with ten rounds (Salmon et al.,
 * 2011), key = seed, counter words = (low 32 bits of i / 8, its high bits + site 2^16,
 * low and high 32 bits of the offset); element i takes 16 bits, the lower half of word
 * (i % 8) / 2 for even i, the upper for odd, and stays when they are at least
 * cut = floor(65536 p + 1/2).  p is thus taken in steps of 2^-16, and the scale is
 * 65536 / (65536 - cut).  rng is device memory, two int64: seed and offset; a program
 * adds to the offset once a step (in a captured graph as well) and gives each place of
 * its model a site of its own. */
typedef struct tt_dropout_desc {
  float p;  /* 0 .. 1 */
  int site; /* 0 .. 65535 */
  int act;  /* tt_dtype: F32 or BF16 */
} tt_dropout_desc;
/* Host only.  TT_ERR_INVALID_ARG for a bad field, TT_ERR_UNSUPPORTED for E4M3. */
tt_status tt_dropout_plan(const tt_dropout_desc* desc, tt_plan_t** out);
/* y = dropout(x) + res for n elements (n below 2^48), dense, 16-byte aligned; res may
 * be NULL; y may be x or res itself.  Its own backward pass: dx is the dropout of dy
 * with the same rng and site, the gradient of res is dy.  The sum is fp32, rounded
 * once.  n == 0 is a no-op. */
tt_status tt_dropout(const tt_plan_t* plan, int64_t n, const int64_t* rng, const void* x,
                     const void* res, void* y, void* stream);
/* tt_norm_forward and tt_norm_backward with dropout of x in front of the residual sum:
 * s = dropout(x) + res.  `dropout` is a plan of tt_dropout_plan with the same activation type;
 * i = t N + j.  The backward takes the same rng and gives dres, the gradient of s and of
 * res, and dx = dropout(dres); dres may be NULL, and is not dx.  dx and dres may each be
 * dy or dsum.  All else as there. */
tt_status tt_norm_dropout_forward(const tt_plan_t* plan, const tt_plan_t* dropout, int64_t T,
                                  const int64_t* rng, const void* x, const void* res,
                                  const float* gamma, const float* beta, void* sum, void* y,
                                  float* stats, void* stream);
tt_status tt_norm_dropout_backward(const tt_plan_t* plan, const tt_plan_t* dropout, int64_t T,
                                   const int64_t* rng, const void* s, const void* dy,
                                   const void* dsum, const float* gamma, const float* stats,
                                   void* dx, void* dres, float* dgamma, float* dbeta, void* ws,
                                   size_t ws_bytes, void* stream);

/* ---- log probabilities of given tokens, their entropy, top alternatives, gradient ----
 * What follows a model's output layer: the loss of training, the scores of a text,
 * the choice of a next token.  For a row of V logits x, z = scale x:
 *   lse = log sum_v exp(z_v),  p_v = exp(z_v - lse),
 *   logp = z_target - lse,     entropy = lse - sum_v p_v z_v,
 *   top: the indices of the largest logits in order, of equal ones the lowest index
 *   first, and their z - lse.
 * A negative target stands for none: logp = 0 and no gradient of it.  A target of V
 * or more is taken as none and recorded in the device status word (TT_ERR_DEVICE).
 * A logit of -infinity has p = 0; a row of nothing else gives lse = -infinity,
 * entropy 0, logp -infinity and zero gradients.  An lse beyond fp32's range is the infinity
 * of its sign; the row's other results are those of its logits.  A NaN or +infinity makes
 * the row's results NaN (its top indices are valid, their order is not given).  All sums are
 * fp32.
 * Row t of the logits starts at logits[t stride], at any multiple of the element;
 * columns from V on are not read (nor written, in dlogits). */
typedef struct tt_logp_desc {
  int64_t V;    /* 1 .. 2^24 */
  float scale;  /* 1e-6 .. 1e6: 1 / temperature */
  int top;      /* top alternatives, 0 .. min(V, 64) */
  int act;      /* tt_dtype of logits and their gradients: F32 or BF16 */
} tt_logp_desc;
/* Host only.  TT_ERR_INVALID_ARG for a bad field, TT_ERR_UNSUPPORTED for E4M3, V
 * above 2^24 or top above 64. */
tt_status tt_logp_plan(const tt_logp_desc* desc, tt_plan_t** out);
/* T rows (below 2^31).  stride: elements from row to row, V .. 2^31.  targets: T int32 (NULL:
 * no logp).  logp, lse, entropy: T fp32 each, any of them NULL where it is not wanted;
 * top (T x top int32) and top_logp (T x top fp32): both or neither.  Needs no workspace.
 * T == 0 is a no-op. */
tt_status tt_logp_forward(const tt_plan_t* plan, int64_t T, const void* logits, int64_t stride,
                          const int32_t* targets, float* logp, float* lse, float* entropy,
                          int32_t* top, float* top_logp, void* stream);
/* dlogits of L = sum_t dlogp logp + dentropy entropy, from the forward's lse (and entropy
 * where dentropy is given; one of the two gradients may be NULL):
 *   dlogits_v = scale (dlogp ([v = target] - p_v) - dentropy p_v (z_v - lse + entropy)).
 * lse is rounded to fp32, which a weight p_v feels by 2^-24 |lse| of itself.  A row of
 * |lse| above 256 (f32) or 4096 (bf16), infinities among them, has its sum taken again from
 * the logits, so rows of large finite masks have the gradient of tt_logp_loss.
 * dlogits may be logits (the same strides). */
tt_status tt_logp_backward(const tt_plan_t* plan, int64_t T, const void* logits, int64_t stride,
                           const int32_t* targets, const float* lse, const float* dlogp,
                           const float* entropy, const float* dentropy, void* dlogits,
                           int64_t dstride, void* stream);
/* Both in one pass, where the gradients are known beforehand (-1 / T for a mean loss):
 * logp, lse and entropy (each may be NULL) and dlogits; reads the logits once. */
tt_status tt_logp_loss(const tt_plan_t* plan, int64_t T, const void* logits, int64_t stride,
                       const int32_t* targets, const float* dlogp, const float* dentropy,
                       float* logp, float* lse, float* entropy, void* dlogits, int64_t dstride,
                       void* stream);

/* ---- the device-side error path ---------------------------------------------
 * Every wait inside the library's kernels (on a TMA transfer, on another warp
 * of the CTA, on a grid barrier) is bounded: after the limit it records
 * TT_ERR_TIMEOUT in the device status word, tells the CTA's other warps to
 * stop, waits (bounded) for its own copies and MMAs, frees its tensor memory
 * and returns, leaving the context usable.  Not part of the CoMERA method.
 * In the attention kernels a wait's limit counts from the last tile that its CTA
 * worked on: one piece of their work may be as long as the sequences are. */

/* The limit of those waits on the current device, in nanoseconds of the
 * global timer (default 2e9, at least 1000).  Applies to kernels launched
 * afterwards; call it with no library work in flight on the device and
 * outside stream capture.  TT_ERR_INVALID_ARG below 1000 ns. */
tt_status tt_set_wait_limit_ns(uint64_t ns);

/* Test hook: the next launch on the current device of the named kernel skips
 * one arrival in its first CTA, so that a bounded wait of that launch runs
 * out (the launch then reports TT_ERR_TIMEOUT through tt_get_device_status
 * and its outputs are undefined).  It faults nothing and hangs nothing: it is
 * for testing the error path above.  Same calling rules as
 * tt_set_wait_limit_ns. */
#define TT_DEBUG_NONE 0
#define TT_DEBUG_FWD_TOKENS 1    /* forward token kernel: first stage never loaded */
#define TT_DEBUG_BWD_TOKENS 2    /* backward token kernel: first stage never loaded */
#define TT_DEBUG_MERGE_BARRIER 3 /* merge engine (programs of 2+ phases): one grid-barrier arrival */
/* tensor-core attention kernels: the first tile of their lists never loaded */
#define TT_DEBUG_ATTN_FWD 4
#define TT_DEBUG_ATTN_BWD_QUERIES 5 /* the backward's pass over queries (dq) */
#define TT_DEBUG_ATTN_BWD_KEYS 6    /* its pass over keys (dk, dv) */
#define TT_DEBUG_LOGP_LOSS 7 /* tt_logp_loss of many rows of 24 to 108 KB: the first never loaded */
tt_status tt_debug_skip_arrival(int site);

/* Synchronise stream, then read and clear the status word of the current
 * device.  The word is sticky: it holds the first error any libttc kernel
 * on this device recorded since the last read.  Returns TT_OK,
 * TT_ERR_TIMEOUT or TT_ERR_DEVICE (or TT_ERR_CUDA). */
tt_status tt_get_device_status(void* stream);

const char* tt_status_string(tt_status s);

/* ---- measurement hooks (host side, not thread-safe) ------------------------
 * When enabled, every kernel phase the library enqueues is bracketed by CUDA
 * events on the caller's stream, and every kernel launch is counted.  Phases:
 * 0 merge (chain merges, forward), 1 forward token pass, 2 backward token pass,
 * 3 merge backward, 4 elementwise (GELU).  Not part of the CoMERA method:
 * it lets a benchmark time the library's own kernels with CUDA events. */
#define TT_NUM_PHASES 5
void tt_profile_enable(int on); /* on != 0: clear records and start; 0: stop */
/* Synchronise on the recorded events and return the summed milliseconds and
 * the number of bracketed intervals of one phase since the last enable.
 * Calls captured into a CUDA graph record external event nodes: after each
 * replay of that graph this returns the times of that replay. */
tt_status tt_profile_phase(int phase, double* total_ms, int64_t* intervals);
const char* tt_profile_phase_name(int phase);
/* Total kernels this library has launched in this process (monotonic). */
uint64_t tt_launch_count(void);
/* Throughput probe of the fused FFN kernels' GELU arithmetic: `blocks`
 * blocks of 256 threads each carry 16 values through `iters` rounds of the
 * same packed tanh-form GELU (mode 0) or GELU and GELU' (mode 1), in
 * registers, and write one float each to out (device, blocks * 256 floats).
 * Evaluations = blocks * 256 * 16 * iters; time it with CUDA events on
 * `stream`. */
tt_status tt_gelu_rate(int mode, int iters, int blocks, float* out, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TTC_H */
