/*
 * moe.h -- C ABI of the MI355X (gfx950) sparse-MoE FFN forward of GLM-4.5 / GLM-5.
 *
 * What the layer computes (pages as titled):
 *  - "Group Router" (GLM-4.5), How it works: s = sigmoid(x W_g^T), a bias-free
 *    gate evaluated in float32; s' = s + b, the correction bias used only to
 *    choose experts; G contiguous groups scored by the sum of their two largest
 *    s'; the topk_group best groups kept; the top-k experts by s' inside them;
 *    weights w = alpha * s / (sum over the chosen of s + eps) from the raw s
 *    (w = alpha * s without norm_topk_prob).
 *  - "MoE Forward" (GLM-4.5), How it works: each routed expert is a bias-free
 *    SwiGLU, E_i(x) = W_down (SiLU(W_gate x) * W_up x), with gate and up packed
 *    as one (2 d, D) matrix; y_n = sum over the chosen of w E_i(x_n) + E_sh(x_n);
 *    alpha scales only the routed sum; every token uses exactly k routed
 *    experts plus the shared one.
 *  - "GLM-5 . Mixture of experts" and "Shared output": the module layout (router,
 *    routed experts, one shared MLP of width n_shared * d) and the per-expert
 *    token lists that dispatch builds; the expert loop skips the id E, which
 *    marks an empty slot in routing given by the caller.
 *  - "Module 02 -- MoE: Capacity, Work, and Traffic", section 3: the clamped
 *    SwiGLU of that checkpoint (swiglu_limit below).
 *
 * Conventions for every call:
 *  - Buffers: all tensor pointers are device pointers (HBM), row-major and
 *    contiguous, 16-byte aligned, owned by the caller. The library allocates
 *    nothing and frees nothing on these calls; scratch space is the caller's
 *    `workspace` of at least moe_workspace_size() bytes. Calls that may run at
 *    the same time (on different streams) need separate workspaces.
 *  - Streams: `stream` is a hipStream_t (NULL = the null stream). Every call
 *    enqueues its kernels on it and returns without synchronising.
 *  - Errors: configuration and argument errors are detected on the host before
 *    anything is launched and returned as a status; a failed launch returns
 *    MOE_ERR_HIP. No exception crosses the ABI.
 *  - N = 0 is valid and launches nothing (moe_dispatch: one small kernel that zeroes counts and
 *    offsets).
 *  - Inputs must be finite. Router weight, bias, scores and mixture weights are
 *    float32 whatever `dtype` says; indices are int32.
 *  - Readings where the pages are open: discarded groups are excluded from the
 *    top-k; ties go to the lower expert / group index (IEEE comparison, so +0
 *    equals -0); the k slots are in (s' descending, index ascending) order, and
 *    that order fixes the summation order of the weight denominator; alpha is
 *    applied once, inside the weights unless alpha_on_output moves it to the
 *    routed sum; eps is added to the denominator as a float32 (1e-20 rounds to
 *    9.99999968e-21).
 */
#ifndef SPARSE_MOE_LAYER_GATE_AMD_MOE_H
#define SPARSE_MOE_LAYER_GATE_AMD_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1, /* a config field, size or pointer is invalid */
  MOE_ERR_UNSUPPORTED = 2, /* valid per the pages, not supported by these kernels (see moe_check_config) */
  MOE_ERR_WORKSPACE = 3,   /* workspace missing or smaller than moe_workspace_size() */
  MOE_ERR_HIP = 4          /* a HIP launch or runtime call failed */
} moe_status;

typedef enum { MOE_F32 = 0, MOE_BF16 = 1 } moe_dtype;

/* The router / expert fields of the model config ("Group Router": n_group, topk_group,
 * num_experts_per_tok, norm_topk_prob, routed_scaling_factor; "MoE Forward": moe_intermediate_size,
 * n_shared_experts). */
typedef struct {
  int32_t hidden_size;           /* D: multiple of 64 */
  int32_t n_routed_experts;      /* E: 1..512 */
  int32_t n_group;               /* G: divides E, 1..64; E/G >= 2 when G > 1 */
  int32_t topk_group;            /* 1..G */
  int32_t num_experts_per_tok;   /* k: 1..32 and k <= topk_group * E / G */
  int32_t moe_intermediate_size; /* d: multiple of 64 */
  int32_t n_shared_experts;      /* >= 0; the shared MLP has width d * n_shared_experts */
  float routed_scaling_factor;   /* alpha */
  int32_t norm_topk_prob;        /* 0 or 1 */
  float eps;                     /* added to the weight denominator (1e-20 on the pages) */
  int32_t dtype;                 /* moe_dtype of x, the expert weights and y */
  /* Where alpha goes ("MoE Forward", Official code: inside the router or on the routed output, never
   * both). 0: w = alpha * s / (sum s + eps). 1: w = s / (sum s + eps), and the combine multiplies the
   * routed sum by alpha before adding the shared expert. */
  int32_t alpha_on_output;
  /* Clamped SwiGLU ("Module 02 -- MoE: Capacity, Work, and Traffic", section 3), in every expert, routed
   * and shared: with L = swiglu_limit > 0, gate = min(gate, L) (no lower bound) and
   * up = min(max(up, -L), L) before SiLU(gate) * up. 0: plain SwiGLU. Finite and >= 0. */
  float swiglu_limit;
} moe_config;

/* Device pointers to the layer's weights, in the pages' canonical layouts. */
typedef struct {
  const float* w_router; /* [E, D] float32 */
  const float* e_bias;   /* [E] float32 correction bias (selection only) */
  const void* gate_up;   /* [E, 2d, D]: rows [0, d) gate, rows [d, 2d) up */
  const void* down;      /* [E, D, d] */
  const void* sh_gate;   /* [d_sh, D]; NULL iff n_shared_experts == 0 */
  const void* sh_up;     /* [d_sh, D] */
  const void* sh_down;   /* [D, d_sh] */
  /* NULL, or moe_router_prepare's output for w_router (bf16 layers): the forward then reads it and skips
   * splitting w_router on every call; w_router is not read and may be NULL. */
  const void* w_router_prepared;
} moe_weights;

/* moe_route flags. */
#define MOE_ROUTE_SCORES_IN 1u  /* read the float32 scores s [N, E] from `scores`; skip the gate GEMM */
#define MOE_ROUTE_SCORES_OUT 2u /* also write s [N, E] to `scores` (without it `scores` may be NULL) */
#define MOE_ROUTE_PREPARED 4u   /* `w_router` is moe_router_prepare's output, not the float32 weight */

/* Host only. MOE_OK if the config is valid and these kernels support it; otherwise
 * MOE_ERR_INVALID_ARG (not a valid layer) or MOE_ERR_UNSUPPORTED (outside the limits above). */
moe_status moe_check_config(const moe_config* cfg);

/* Host only. Bytes of workspace moe_forward, moe_forward_routed and moe_route need for N tokens (0 for
 * an invalid config): the most any batch of at most N tokens needs, so the size never falls as N grows
 * and a workspace sized for the largest batch serves every smaller one. */
size_t moe_workspace_size(const moe_config* cfg, int64_t N);

/* Host only. Bytes of workspace moe_dispatch needs for N tokens: per-chunk counts for batches of more
 * than 256 tokens, 0 below (one kernel, no scratch). Never falls as N grows. */
size_t moe_dispatch_workspace_size(const moe_config* cfg, int64_t N);

/* Host only. Bytes of the prepared router weight of a bf16 layer: 3 * E * D * 2 (0 for float32 layers,
 * which use w_router as given, or an invalid config). */
size_t moe_router_prepared_size(const moe_config* cfg);

/* Prepare the router weight of a bf16 layer once, for calls that would otherwise split it every time
 * ("Group Router", How it works: the gate is evaluated in float32; the bf16 gate GEMM runs it as three
 * exact bf16 pieces). prepared [3, E, D] bf16 (caller-owned, >= moe_router_prepared_size bytes) receives
 * hi, mid and lo with hi + mid + lo == w_router exactly, each the bf16 rounding of what the pieces before
 * it leave. Pass it as moe_weights.w_router_prepared or to moe_route with MOE_ROUTE_PREPARED; run it
 * again whenever w_router changes. MOE_ERR_INVALID_ARG for float32 layers. Asynchronous on `stream`. */
moe_status moe_router_prepare(const moe_config* cfg, const float* w_router, void* prepared, size_t bytes,
                              void* stream);

/* Router: gate GEMM + sigmoid, then group-restricted top-k and mixture weights ("Group Router").
 *   x        [N, D] of cfg->dtype (ignored with MOE_ROUTE_SCORES_IN)
 *   w_router [E, D] float32, or with MOE_ROUTE_PREPARED the [3, E, D] bf16 output of moe_router_prepare
 *            (ignored with MOE_ROUTE_SCORES_IN)
 *   e_bias   [E] float32
 *   scores   [N, E] float32: read (MOE_ROUTE_SCORES_IN), written (MOE_ROUTE_SCORES_OUT), or unused and
 *            may be NULL (neither flag). SCORES_IN excludes the other two flags.
 *   topk_idx [N, k] int32 out: the chosen experts in slot order
 *   topk_w   [N, k] float32 out: their weights, alpha included (unless alpha_on_output)
 *   workspace, ws_bytes: scratch of at least moe_workspace_size(cfg, N) bytes (unused, may be NULL,
 *            with MOE_ROUTE_SCORES_IN)
 * The logits are float32 dot products (bf16 activations: exact products of x with an exact three-piece
 * bf16 split of w_router, accumulated in float32: on the matrix cores, or with fused multiply-adds for
 * batches of one to four tokens). Given the same float32 scores,
 * indices and weights are bit-identical to a float32 evaluation in the order stated above (correctly
 * rounded add, divide and multiply). */
moe_status moe_route(const moe_config* cfg, int64_t N, const void* x, const void* w_router, const float* e_bias,
                     float* scores, uint32_t flags, int32_t* topk_idx, float* topk_w, void* workspace,
                     size_t ws_bytes, void* stream);

/* Token-choice dispatch: per-expert token lists in the per-expert loop form of "GLM-5 . Mixture of
 * experts", as counts, an exclusive scan and a stable placement (tokens ascending inside each expert).
 *   topk_idx    [N, k] int32 in: expert ids in [0, E); E marks an empty slot
 *   counts      [E] int32 out: (token, slot) pairs per expert
 *   offsets     [E + 1] int32 out: exclusive scan of counts; offsets[E] = N * k less the empty slots
 *   sorted_pair [N * k] int32 out: the flat pair index n * k + slot at each expert-sorted position; the
 *               token is sorted_pair / k (the page's per-expert token index list) and the slot, which
 *               selects the mixture weight, is sorted_pair % k
 *   inv_row     [N * k] int32 out: the position of each pair (inverse of sorted_pair)
 *   workspace, ws_bytes: at least moe_dispatch_workspace_size(cfg, N) bytes (may be NULL when that is 0)
 * Pairs whose id is outside [0, E) are left out of the lists (inv_row = -1); the lists are then
 * shorter than N * k and offsets[E] says so. */
moe_status moe_dispatch(const moe_config* cfg, int64_t N, const int32_t* topk_idx, int32_t* counts,
                        int32_t* offsets, int32_t* sorted_pair, int32_t* inv_row, void* workspace,
                        size_t ws_bytes, void* stream);

/* The whole layer ("MoE Forward", eq. y_n): route, dispatch, the routed SwiGLU experts on bf16 MFMA
 * (float32 accumulation; float32 arithmetic when dtype is MOE_F32), the weighted combine in a fixed
 * order without atomics, and the unscaled shared expert.
 *   x [N, D] and y [N, D] of cfg->dtype; y must not overlap x.
 *   topk_idx_out [N, k], topk_w_out [N, k], counts_out [E]: optional copies of the routing (NULL to skip).
 * Deterministic: the same inputs give bit-identical outputs. */
moe_status moe_forward(const moe_config* cfg, int64_t N, const void* x, const moe_weights* w, void* y,
                       int32_t* topk_idx_out, float* topk_w_out, int32_t* counts_out, void* workspace,
                       size_t ws_bytes, void* stream);

/* moe_forward without a workspace argument, for callers that cannot allocate device memory: code being
 * captured into a HIP graph, serving loops that must not call the allocator, harnesses that forbid it.
 * The scratch is a fixed device array of moe_noalloc_scratch_bytes() (32 MiB) inside the library, one
 * per device, taken from the first call on each device until the process ends. The call allocates and
 * frees nothing; it returns MOE_ERR_WORKSPACE, before launching anything, when the batch needs more than
 * that (moe_workspace_size(cfg, N) > moe_noalloc_scratch_bytes(): on the GLM-5 shape batches of up to
 * 146 tokens fit), and MOE_ERR_HIP if the array's device address cannot be found. Every call on a
 * device shares that device's array: calls that may overlap on one device (other streams, other
 * threads) race and must be serialised by the caller. No part of the array has to start at zero: each
 * call writes every region it reads. Arguments and results otherwise as moe_forward. */
moe_status moe_forward_noalloc(const moe_config* cfg, int64_t N, const void* x, const moe_weights* w, void* y,
                               int32_t* topk_idx_out, float* topk_w_out, int32_t* counts_out, void* stream);
size_t moe_noalloc_scratch_bytes(void);

/* The layer with routing given by the caller ("MoE Forward", Official code: the experts take x, the
 * top-k indices and the top-k weights; "GLM-5 . Mixture of experts": the expert loop skips id E):
 * dispatch, routed experts, combine and shared expert as in moe_forward, without the router.
 *   topk_idx [N, k] int32 in: expert ids; E (or any id outside [0, E)) marks an empty slot, which
 *            adds nothing
 *   topk_w   [N, k] float32 in: the weights, used as given (alpha is applied on the routed sum only
 *            when cfg->alpha_on_output is 1)
 *   x, y, counts_out, workspace, ws_bytes, stream: as for moe_forward.
 * Deterministic: the same inputs give bit-identical outputs. */
moe_status moe_forward_routed(const moe_config* cfg, int64_t N, const void* x, const moe_weights* w,
                              const int32_t* topk_idx, const float* topk_w, void* y, int32_t* counts_out,
                              void* workspace, size_t ws_bytes, void* stream);

/* The dense SwiGLU FFN of the layers before the MoE ones ("Shared output" (GLM-5), the evidence from the
 * shared expert: the dense feed-forward network is the same bias-free SwiGLU MLP,
 * y = W_down (SiLU(W_gate x) * W_up x), at the model's full intermediate width; "MoE Forward": dense
 * prefix layers never enter the MoE module). Runs on the same GEMM kernels as the shared expert.
 *   N, D, dff: tokens, hidden size, intermediate width (D and dff multiples of 64)
 *   dtype: moe_dtype of x, the weights and y; swiglu_limit as in moe_config (0: plain SwiGLU)
 *   x [N, D], gate [dff, D], up [dff, D], down [D, dff], y [N, D] (y must not overlap x)
 *   workspace, ws_bytes: at least moe_dense_workspace_size(N, D, dff, dtype) bytes.
 * Errors as for the other calls; N = 0 launches nothing. */
size_t moe_dense_workspace_size(int64_t N, int32_t D, int32_t dff, int32_t dtype);
moe_status moe_dense_forward(int64_t N, int32_t D, int32_t dff, int32_t dtype, float swiglu_limit, const void* x,
                             const void* gate, const void* up, const void* down, void* y, void* workspace,
                             size_t ws_bytes, void* stream);

/* ---- The operators around the experts --------------------------------------------------------------
 *
 * For models that hold more than the fused layer: the norms, gate and residual on both sides of a block,
 * the experts' products as separate calls (other activations, adapters, training), the combine of their
 * rows, and experts with 4-bit weights. They work on the same lists as the layer (moe_route,
 * moe_dispatch). The conventions at the top hold: 16-byte aligned contiguous device pointers, the
 * caller's stream and workspace, errors found on the host before any launch, no atomics on results (the same
 * inputs give the same bits). Calls that write gradients overwrite them.
 */

/* Norms before and after a block, fused with the block's gate and the residual scale:
 *   h_out = residual_scale * h + gate * (o / rms(o)) * w_post,   u = (h_out / rms(h_out)) * w_pre,
 *   rms(v) = sqrt(mean(v^2) + eps) over the D features of a row.
 * One call closes a block (o is its output) and opens the next (u is its input). Parts that are absent:
 *   o == NULL      the norm before a block alone: u from h. w_post, gate and h_out are NULL, residual_scale
 *                  is not used.
 *   w_pre == NULL  the end of a block alone: h_out. u is NULL.
 *   w_post == NULL o enters as it is, without a norm.   gate == NULL: 1.
 *   h, o, h_out, u [N, D] of dtype; w_post, w_pre [D] of dtype
 *   gate    [ceil(N / gate_rows), D] of dtype: row n uses gate row n / gate_rows (gate_rows >= N: one row
 *           for all; 1: a row per token; a sequence's length: one per sequence)
 * Float32 arithmetic; h_out and u are each rounded once, u from the unrounded h_out. h_out may be h
 * (in place); no other overlap. D: a multiple of 64, at most 16384. N below 2^31, and N * T below 2^32 with T the
 * threads of a row: D / 8 (D / 16 above 8192), rounded up to a multiple of 64. N = 0 launches nothing. */
moe_status moe_block_norm(int64_t N, int32_t D, int32_t dtype, float eps, float residual_scale, const void* h,
                          const void* o, const void* w_post, const void* gate, int64_t gate_rows, const void* w_pre,
                          void* h_out, void* u, void* stream);

/* Gradients of moe_block_norm, from the tensors of the forward call (nothing else is kept):
 *   h_out   [N, D]: the forward's h_out, or its h when o == NULL (not read, and may be NULL, without w_pre)
 *   dh_out, du: the gradients of h_out and u. dh_out may be NULL (zero) when du is given; du is NULL
 *           without w_pre. With o == NULL, dh_out is what reaches h beside the norm.
 *   dh [N, D], d_o [N, D] (NULL without o) of dtype, written
 *   dw_post [D], dgate [ceil(N / gate_rows), D], dw_pre [D] float32, written, or NULL where not wanted:
 *           sums over rows in a fixed order
 *   workspace: at least moe_block_norm_workspace_size(N, D, dtype, gate ? gate_rows : 0) bytes (may be NULL
 *           when no sum is wanted). The size never falls as N grows.
 * dh may be dh_out (in place); no other overlap. residual_scale has no gradient. N below 2^31. N = 0 writes zeros
 * to dw_post and dw_pre. */
size_t moe_block_norm_workspace_size(int64_t N, int32_t D, int32_t dtype, int64_t gate_rows);
moe_status moe_block_norm_backward(int64_t N, int32_t D, int32_t dtype, float eps, float residual_scale,
                                   const void* h_out, const void* o, const void* w_post, const void* gate,
                                   int64_t gate_rows, const void* w_pre, const void* dh_out, const void* du, void* dh,
                                   void* d_o, float* dw_post, float* dgate, float* dw_pre, void* workspace,
                                   size_t ws_bytes, void* stream);

/* The combine as a call of its own ("MoE Forward", eq. y_n, for expert rows that are not weighted yet):
 *   y[n] = alpha * sum over the slots s of topk_w[n, s] * rows[inv_row[n, s]]  +  shared[n]
 *   rows [R, D], shared [N, D] or NULL, y [N, D] of dtype; inv_row [N, k] int32 as moe_dispatch writes it;
 *   topk_w [N, k] float32 or NULL (all 1: the gradient of a gathered token is the sum of its rows').
 * Slots whose entry is outside [0, R) add nothing. Float32 sums in slot order, one rounding. y may be
 * shared (in place) but not rows. k: 1..32; D: a multiple of 64; N k and R below 2^31, and N * T below 2^32 with T
 * the threads of a token: D / 8 rounded up to a multiple of 64, at most 1024. N = 0 launches nothing. */
moe_status moe_combine(int64_t N, int32_t k, int32_t D, int32_t dtype, const void* rows, int64_t R,
                       const int32_t* inv_row, const float* topk_w, const void* shared, float alpha, void* y,
                       void* stream);

/* Gradients of moe_combine:
 *   drows[inv_row[n, s]] = alpha * topk_w[n, s] * dy[n]   (of dtype)
 *   dtopk_w[n, s]        = alpha * <dy[n], rows[inv_row[n, s]]>   (float32; 0 for an empty slot)
 * The entries of inv_row inside [0, R) are distinct, as moe_dispatch writes them; rows that no slot names
 * are left as they were. dtopk_w may be NULL (not wanted; rows may then be NULL too) and is NULL without
 * topk_w. The gradient of shared is dy. drows overlaps neither dy nor rows. Sizes as for moe_combine. */
moe_status moe_combine_backward(int64_t N, int32_t k, int32_t D, int32_t dtype, const void* dy, const void* rows,
                                int64_t R, const int32_t* inv_row, const float* topk_w, float alpha, void* drows,
                                float* dtopk_w, void* stream);

/* A bias-free linear map per expert over rows grouped by expert, ragged sizes, and its gradients. Expert e
 * has the rows r in [offsets[e], offsets[e + 1]):
 *   moe_grouped_linear        y[r]  = W[e] x[src(r)]
 *   moe_grouped_linear_dgrad  dx[r] = W[e]^T dy[r]
 *   moe_grouped_linear_wgrad  dW[e] = sum over the expert's rows of dy[r] x[src(r)]^T   (0 without rows)
 *   W, dW [E, out, in], y, dy [R, out], dx [R, in] of dtype
 *   x       [x_rows, in] of dtype; src(r) = row_index[r] / index_div with row_index [R] int32 (moe_dispatch's
 *           sorted_pair with index_div = k gathers tokens), or r when row_index is NULL (x_rows >= R)
 *   offsets [E + 1] int32 on the device, ascending, as moe_dispatch writes them. Rows outside
 *           [offsets[0], offsets[E]) belong to no expert: no output row of theirs is written.
 *   workspace: at least moe_grouped_workspace_size(E, R, dtype) bytes. The size never falls as R grows.
 * dx holds one row per grouped row: the gradient of a gathered token is moe_combine of its rows with
 * topk_w == NULL. Offsets and indices are read on the device and kept in range there: offsets outside [0, R]
 * or out of order and indices outside [0, x_rows * index_div) give unspecified values, never an access
 * outside the buffers. Float32 sums over the whole reduction, one rounding. E: 1..512; in and out:
 * multiples of 64 up to 2^22, in * out below 2^31; bf16: gathered x below 4 GiB; R below 2^31.
 * Calls whose tiles would take a launch of 2^32 threads are MOE_ERR_UNSUPPORTED (float32: 2^24 tiles of 128 x 128).
 * R = 0 launches nothing (wgrad: writes zeros). No overlap between an output and an input. */
size_t moe_grouped_workspace_size(int32_t E, int64_t R, int32_t dtype);
moe_status moe_grouped_linear(int32_t E, int64_t R, int32_t in, int32_t out, int32_t dtype, const void* x,
                              int64_t x_rows, const int32_t* row_index, int32_t index_div, const void* w,
                              const int32_t* offsets, void* y, void* workspace, size_t ws_bytes, void* stream);
moe_status moe_grouped_linear_dgrad(int32_t E, int64_t R, int32_t in, int32_t out, int32_t dtype, const void* dy,
                                    const void* w, const int32_t* offsets, void* dx, void* workspace, size_t ws_bytes,
                                    void* stream);
moe_status moe_grouped_linear_wgrad(int32_t E, int64_t R, int32_t in, int32_t out, int32_t dtype, const void* dy,
                                    const void* x, int64_t x_rows, const int32_t* row_index, int32_t index_div,
                                    const int32_t* offsets, void* dw, void* workspace, size_t ws_bytes,
                                    void* stream);

/* moe_grouped_linear with 4-bit weights and one scale per group of a weight row:
 *   W[e, m, i] = (q[e, m, i] - 8) * scales[e, m, i / group],   q in 0..15
 *   wq      [E, out, in / 2] uint8: two values a byte, even i in the low four bits
 *   scales  [E, out, in / group] bf16 (one that is not finite shows in the outputs of its weight row, in no other);
 *           group 32, 64 or 128, dividing in
 *   x, y    bf16; x, x_rows, row_index, index_div, offsets, rows as for moe_grouped_linear. With E = 1 offsets
 *           may be NULL: all R rows (a plain 4-bit linear map).
 *   swiglu  1: the rows of W are [0, out / 2) gate and [out / 2, out) up, and y [R, out / 2] is
 *           SiLU(W_gate x) * W_up x, clamped by swiglu_limit > 0 as in moe_config (out a multiple of 128).
 *           0: y [R, out], swiglu_limit 0.
 * Float32 sums of the products x * (q - 8) over a group (which have to stay in float32's range: 8 |x| summed over a
 * group below 2^128), then scaled and added; no weight and no partial sum is rounded to fewer bits, and a weight of
 * q = 8 adds exactly nothing. No workspace. x does not overlap y. R = 0
 * launches nothing. */
moe_status moe_qlinear(int32_t E, int64_t R, int32_t in, int32_t out, int32_t group, const void* x, int64_t x_rows,
                       const int32_t* row_index, int32_t index_div, const void* wq, const void* scales,
                       const int32_t* offsets, int32_t swiglu, float swiglu_limit, void* y, void* stream);

/* Weights for moe_qlinear from w [rows, in] of dtype (rows = E * out): scale = bf16(max|w| / 7) over each
 * group, q = 8 + the nearest integer (ties to even) of the float32 quotient w / scale, kept in 0..15; a
 * group whose scale is 0 has q = 8. w need not be finite: a group that holds a NaN has the scale NaN, any other that
 * holds an infinity the scale infinity, and q = 8, so that every product with the group is NaN. in: a multiple of 64
 * and of group; rows * in at most 2^35 - 2^11. */
moe_status moe_quantize(int32_t dtype, int64_t rows, int32_t in, int32_t group, const void* w, void* wq, void* scales,
                        void* stream);

/* Static string naming a status. */
const char* moe_status_str(moe_status status);

/* Per-stage timing for measurement. moe_profile_begin() starts recording a HIP event pair, on the
 * stream each call is given, around every kernel that moe_forward / moe_route / moe_dispatch launch
 * from the calling thread; moe_profile_end() waits for those events, writes the summed milliseconds and
 * launch counts per stage (up to n_stages entries, indexed as moe_stage_name lists them) and stops
 * recording. The recording state is per thread: calls made by other threads are not recorded, and each
 * thread's begin / end pair is independent. A thread's HIP events are reused across its recordings and
 * live until the process ends. Returns MOE_ERR_HIP if event creation or timing fails. For measurement
 * only: recording adds two event records around every launch. */
moe_status moe_profile_begin(void);
/* As moe_profile_begin, recording only the stages whose bit (1 << stage) is set in stage_mask (fewer
 * events in the stream when only some kernels are to be timed). */
moe_status moe_profile_begin_mask(uint32_t stage_mask);
moe_status moe_profile_end(double* ms_per_stage, int32_t* launches_per_stage, int32_t n_stages);
/* Name of stage i (NULL past the last), and the number of stages. */
const char* moe_stage_name(int32_t stage);
int32_t moe_stage_count(void);

#ifdef __cplusplus
}
#endif

#endif
