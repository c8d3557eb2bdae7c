/*
 * moe.h -- C ABI of libmoe, a DeepSeekMoE layer forward pass for AMD Instinct
 * MI355X (gfx950).
 *
 * The layer is the one of the "DeepSeek-V3 Technical Report" (papers-reader
 * rewrite of arXiv 2412.19437):
 *   §2.1.2  DeepSeekMoE: for the FFN input u_t, the output is the sum of the
 *           N_s shared experts applied to u_t and of the K_r selected routed
 *           experts weighted by their gating values; affinities are
 *           s_{i,t} = sigmoid(u_t . e_i) with e_i the centroid of routed
 *           expert i; gating values are the selected affinities normalised
 *           over the selected experts.
 *   §2.1.2  auxiliary-loss-free balancing: a bias b_i is added to s_{i,t} for
 *           the top-K choice only (the gating value uses the un-biased s);
 *           after each step b_i moves by gamma against expert i's whole-batch
 *           load; node-limited routing keeps a token on at most M groups;
 *           no token is dropped.
 *   §3.3    FP8: activations quantised in 1 x N_c tiles and weights in
 *           N_c x N_c blocks (N_c = 128), each group with its own fp32 scale;
 *           partial sums accumulated in fp32 every N_c products.
 *   §4.2    shape: d = 7168, 1 shared + 256 routed experts, expert
 *           intermediate size 2048, 8 routed experts per token, at most 4
 *           nodes (groups) per token, gamma = 0.001.
 *
 * Conventions for every call
 *   - Return 0 (MOE_OK) or a negative moe_status.  Argument checks run on the
 *     host before any HIP call, so a rejected call touches no device state.
 *     moe_last_error() gives a message for the calling thread's last failure.
 *   - The moe_shape struct is host memory; every array argument is a device
 *     pointer to row-major contiguous storage, owned by the caller.  The
 *     library keeps no pointer after a call returns, but kernels read and
 *     write the buffers until the stream reaches them.
 *   - All work is enqueued on `stream` (a hipStream_t; NULL = the default
 *     stream) without host synchronisation; expert loads never leave the GPU.
 *   - No call allocates device memory: scratch space comes from the caller's
 *     workspace `ws` of `ws_bytes` bytes (size it with moe_workspace_bytes);
 *     the workspace must be 256-byte aligned.
 *   - Matrices of weights are stored [out][in] (the reduction dimension is
 *     contiguous).  bf16 is stored as its 16-bit pattern; e4m3 is OCP E4M3FN
 *     (largest finite 448) in one byte.
 *   - Inputs must be finite; NaN and infinity are not checked (the gate, MX4,
 *     product and update calls say what they make of them).
 *   - Calls on different streams that share a buffer race, workspaces
 *     included (a workspace holds intermediate results and the expert
 *     kernel's tile-queue counters); the library holds no global mutable
 *     state, so calls on different data may overlap.
 */
#ifndef MOE_H_
#define MOE_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = -1,   /* null pointer, non-positive size, bad alignment */
    MOE_ERR_UNSUPPORTED = -2,   /* shape or dtype combination outside the limits below */
    MOE_ERR_WORKSPACE = -3,     /* ws_bytes smaller than moe_workspace_bytes() */
    MOE_ERR_HIP = -4            /* a HIP runtime call or kernel launch failed */
} moe_status;

typedef enum { MOE_F32 = 0, MOE_BF16 = 1, MOE_E4M3 = 2 } moe_dtype;

/* flags */
#define MOE_ADD_RESIDUAL 1u   /* moe_forward / moe_combine add u_t to the output */
/* moe_forward keeps the SwiGLU inputs a = W_gate x and b = W_up x of every
 * routed and shared row (fp32, the gate/up accumulators as they are) in its
 * workspace, which grows by (T*topk + T*n_shared) * 2 * inter * 4 bytes;
 * moe_backward with the same flag then forms the SwiGLU gradient from them
 * instead of recomputing the gate/up product: the same bits, without a second
 * pass over W_gate and W_up.  Forward and backward must agree on this flag. */
#define MOE_SAVE_SWIGLU_INPUTS 2u

/*
 * Shape and numerics of one layer (§2.1.2, §4.2).  Supported combinations
 * (act_dtype, router_dtype, w_dtype, out_dtype):
 *   (F32,  F32,  F32,  F32 )  fp32 everywhere
 *   (BF16, BF16, BF16, BF16)  bf16 storage, fp32 accumulation
 *   (BF16, BF16, E4M3, BF16)  bf16 u and centroids; expert GEMMs in e4m3 with
 *                             1x128 activation / 128x128 weight fp32 scales
 * Limits (MOE_ERR_UNSUPPORTED otherwise): n_routed % n_groups == 0,
 * 1 <= topk_groups <= n_groups <= 64, 1 <= topk <= 32,
 * topk <= topk_groups * n_routed / n_groups, n_routed <= 1024,
 * 0 <= n_shared <= 8, d and inter multiples of 128, quant_block == 128,
 * T * topk < 2^31, T * n_shared < 2^31.
 */
typedef struct moe_shape {
    int64_t T;              /* tokens in the batch (T >= 0; T == 0 is a no-op) */
    int32_t d;              /* hidden size (7168) */
    int32_t n_routed;       /* N_r routed experts (256) */
    int32_t n_shared;       /* N_s shared experts (1) */
    int32_t n_groups;       /* expert groups (nodes) G (8); group g = experts [g*N_r/G, (g+1)*N_r/G) */
    int32_t topk_groups;    /* M: groups a token may use (4) */
    int32_t topk;           /* K_r: routed experts per token (8) */
    int32_t inter;          /* expert intermediate size I (2048) */
    int32_t act_dtype;      /* u, x_perm (non-e4m3), H (non-e4m3) storage: MOE_F32 | MOE_BF16 */
    int32_t router_dtype;   /* centroids gate_w: equal to act_dtype */
    int32_t w_dtype;        /* expert weights and GEMM inputs: act_dtype, or MOE_E4M3 */
    int32_t out_dtype;      /* y_perm, y_shared, out: equal to act_dtype */
    int32_t quant_block;    /* N_c = 128 */
    float routed_scale;     /* factor on every gating value (1.0) */
    uint32_t flags;         /* MOE_ADD_RESIDUAL | MOE_SAVE_SWIGLU_INPUTS, or 0 */
} moe_shape;

/* ------------------------------------------------------------------------ */

/*
 * moe_route -- affinities, group-limited biased top-K, gating values
 * (§2.1.2; the group rule and tie rule are readings of the prose):
 *   s[t][i]  = sigmoid(sum_c u[t][c] * gate_w[i][c])   fp32 accumulation
 *   s'       = s + bias (one fp32 add; used for selection only)
 *   group g score = sum of its two largest s' (its only s' if N_r/G == 1);
 *   the topk_groups best groups are kept, other experts are excluded;
 *   the topk largest s' among kept experts are selected, slot order is
 *   decreasing s'; every tie goes to the lower index;
 *   topk_w[t][j] = routed_scale * s[t][e_j] / (s[t][e_0] + ... + s[t][e_{K-1}])
 *   with the sum taken left to right in fp32.
 * u [T][d] (act_dtype), gate_w [N_r][d] (router_dtype), bias [N_r] fp32.
 * scores_in [T][N_r] fp32 or NULL: when given, u and gate_w are not read and
 * selection runs on these affinities (bit-exact routing checks).
 * scores_out [T][N_r] fp32 or NULL; topk_idx [T][K] int32; topk_w [T][K] fp32.
 * ws: moe_workspace_bytes(shape, MOE_WS_ROUTE) bytes (256-byte aligned): the
 * affinities when scores_out is NULL, and for bf16 layers of 256 routed experts
 * in groups of a multiple of 16 experts with topk <= 16 the chunk partials of
 * a split-K gate GEMM (fp32 partial dot products over chunks of the hidden
 * dimension, summed in chunk order).  Given less workspace (at least the
 * affinities' when scores_out is NULL) the single-pass gate GEMM runs instead:
 * the affinities agree up to the order of the fp32 additions.
 */
int moe_route(const moe_shape *shape, const void *u, const void *gate_w, const float *bias,
              const float *scores_in, float *scores_out, int32_t *topk_idx, float *topk_w,
              void *ws, size_t ws_bytes, void *stream);

/*
 * moe_permute -- dispatch bookkeeping and row gather (§2.1.2: every
 * (token, slot) pair is kept; "whole-batch load" = pairs per expert):
 *   counts[i]   = #{(t, j) : topk_idx[t][j] == i}
 *   offsets     = exclusive prefix sum of counts, offsets[N_r] = T*K
 *   rows offsets[i] .. offsets[i+1]-1 belong to expert i, in increasing t
 *   perm_token[row] = t,   inv_perm[t*K + j] = row
 *   x_perm[row] = u[t]              when w_dtype != E4M3 (act_dtype copy)
 *   x_perm[row] = Q_1x128(u[t]) with x_scales[row][d/128] when w_dtype == E4M3
 *     (Q: scale = amax/448 in fp32, 1 for an all-zero tile; code =
 *      E4M3 round-to-nearest-even of clamp(x/scale, -448, 448); §3.3).
 * x_perm may be NULL (index outputs only); then u and x_scales are ignored.
 * topk_idx entries must lie in [0, N_r) and be distinct within a token.
 * ws: moe_workspace_bytes(shape, MOE_WS_PERMUTE).
 */
int moe_permute(const moe_shape *shape, const int32_t *topk_idx, const void *u,
                int32_t *counts, int32_t *offsets, int32_t *perm_token, int32_t *inv_perm,
                void *x_perm, float *x_scales, void *ws, size_t ws_bytes, void *stream);

/*
 * moe_grouped_ffn -- SwiGLU experts over ragged row groups (§2.1.2 experts;
 * the SwiGLU form is the reading of the unstated expert FFN):
 *   for expert e and each of its rows r in [offsets[e], offsets[e+1]):
 *     a = W_gate[e] x_r,  b = W_up[e] x_r        (fp32 accumulation)
 *     h = SiLU(a) * b,    SiLU(a) = a / (1 + exp(-a)),   stored as
 *         act_dtype, or for E4M3 quantised per 1x128 tile of I (Q above)
 *     y[r] = W_down[e] h  (fp32 accumulation), stored in out_dtype
 *   x_r = x[gather[r]] when gather != NULL, else x[r].
 *   For E4M3 every 128-long block of the reduction is an fp32 partial sum of
 *   code products, multiplied by (activation scale * weight block scale) and
 *   added to the fp32 accumulator (§3.3 promotion every N_c products).
 * n_exp experts; offsets [n_exp+1] int32 on the device, offsets[0] = 0,
 * non-decreasing, offsets[n_exp] <= max_rows.
 * x [*][d] in act_dtype, or e4m3 with x_scales [*][d/128] fp32.
 * w_gate, w_up [n_exp][I][d]; w_down [n_exp][d][I] in w_dtype;
 * w_scales: NULL unless E4M3, then 3 device pointers to fp32 block scales
 * [n_exp][I/128][d/128], [n_exp][I/128][d/128], [n_exp][d/128][I/128]
 * (the array of 3 pointers itself is host memory).
 * y [max_rows][d] out_dtype.  ws: moe_ffn_workspace_bytes(shape, max_rows).
 */
int moe_grouped_ffn(const moe_shape *shape, int32_t n_exp, const int32_t *offsets, int64_t max_rows,
                    const int32_t *gather, const void *x, const float *x_scales,
                    const void *w_gate, const void *w_up, const void *w_down,
                    const float *const *w_scales, void *y, void *ws, size_t ws_bytes, void *stream);

/*
 * moe_combine -- the layer output (§2.1.2 output equation; stripped on the
 * page, read as shared experts plus gate-weighted routed experts):
 *   out[t] = sum_j topk_w[t][j] * y_perm[inv_perm[t*K + j]]
 *          + sum_s y_shared[s][t]  (+ u[t] if MOE_ADD_RESIDUAL)
 * computed in fp32 and rounded once to out_dtype.
 * y_perm [T*K][d], y_shared [N_s][T][d] (NULL when N_s == 0), out [T][d] in
 * out_dtype; residual = u [T][d] (act_dtype), read only with the flag.
 */
int moe_combine(const moe_shape *shape, const void *y_perm, const int32_t *inv_perm, const float *topk_w,
                const void *y_shared, const void *residual, void *out, void *stream);

/*
 * moe_forward -- the whole layer: moe_route, dispatch, the routed and shared
 * grouped FFNs and moe_combine in one enqueue.  For E4M3, u is quantised
 * once per token (1x128) and rows are gathered inside the expert GEMM instead
 * of being copied.
 * routed_w = {W_gate [N_r][I][d], W_up [N_r][I][d], W_down [N_r][d][I]};
 * shared_w = the same with N_s (NULL when N_s == 0).  routed_s / shared_s:
 * the 3 block-scale arrays for E4M3, else NULL.  (Pointer arrays are host
 * memory; their elements are device pointers.)
 * Optional outputs (NULL to skip): topk_idx_out [T][K], topk_w_out [T][K],
 * counts_out [N_r], scores_out [T][N_r].
 * ws: moe_workspace_bytes(shape, MOE_WS_FORWARD).  After the call it holds the
 * layer's saved activations (affinities, selection, gates, dispatch, H and the
 * expert outputs) that moe_backward reads; scores_out, topk_idx_out and
 * topk_w_out receive copies.
 */
int moe_forward(const moe_shape *shape, const void *u, const void *gate_w, const float *bias,
                const void *const *routed_w, const float *const *routed_s,
                const void *const *shared_w, const float *const *shared_s,
                void *out, int32_t *topk_idx_out, float *topk_w_out, int32_t *counts_out,
                float *scores_out, void *ws, size_t ws_bytes, void *stream);

/*
 * moe_forward_timed -- moe_forward that also records caller-created HIP
 * events (hipEvent_t) on `stream` at its stage boundaries, for per-kernel
 * timing without a profiler:
 *   stage_events[0] before the router        [1] after routing (affinities + selection)
 *   [2] after dispatch (and e4m3 quantisation of u)
 *   [3] after the gate/up expert kernel      [4] after the down expert kernel
 *   [5] after the combine
 * NULL entries (or a NULL array, 6 entries otherwise) are skipped.  The array
 * itself is host memory.  Results are identical to moe_forward.
 */
int moe_forward_timed(const moe_shape *shape, const void *u, const void *gate_w, const float *bias,
                      const void *const *routed_w, const float *const *routed_s,
                      const void *const *shared_w, const float *const *shared_s,
                      void *out, int32_t *topk_idx_out, float *topk_w_out, int32_t *counts_out,
                      float *scores_out, void *ws, size_t ws_bytes, void *stream, void *const *stage_events);

/*
 * moe_forward_static -- moe_forward for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc.  The caller passes inputs and outputs only (arguments,
 * results and errors as for moe_forward); the workspace is a buffer of
 * MOE_STATIC_WS_BYTES that the library keeps in device memory, one per GPU it
 * runs on, for the life of the process.  No call allocates or frees memory.
 * Limit: shapes whose moe_workspace_bytes(shape, MOE_WS_FORWARD) exceeds
 * MOE_STATIC_WS_BYTES are rejected with MOE_ERR_WORKSPACE (at the V3 shape,
 * d = 7168 with 256 + 1 experts of I = 2048 in bf16, that is T above about 400
 * tokens: decode-size batches fit); MOE_SAVE_SWIGLU_INPUTS is rejected with
 * MOE_ERR_UNSUPPORTED (the saved activations stay in the library's buffer,
 * where moe_backward cannot read them).  Every call on one GPU shares that
 * GPU's buffer, which keeps the last call's intermediate results: calls that
 * overlap on one GPU (other streams, other host threads) race, so a caller
 * serialises them.
 */
#define MOE_STATIC_WS_BYTES ((size_t)64 << 20)
int moe_forward_static(const moe_shape *shape, const void *u, const void *gate_w, const float *bias,
                       const void *const *routed_w, const float *const *routed_s,
                       const void *const *shared_w, const float *const *shared_s,
                       void *out, int32_t *topk_idx_out, float *topk_w_out, int32_t *counts_out,
                       float *scores_out, void *stream);

/* ------------------------------------------------------------------------ */
/* backward                                                                 */

/*
 * moe_transpose_expert_weights -- the transposed weight copies moe_backward
 * reads (input gradients run through the same grouped expert kernel as the
 * forward, which wants the reduction dimension contiguous):
 *   wt[0] = W_down^T [n][I][d] per expert,
 *   wt[1] = [W_gate^T | W_up^T] [n][d][2I] per expert,
 * from w = {W_gate [n][I][d], W_up [n][I][d], W_down [n][d][I]} in
 * shape->w_dtype.  For E4M3 the 128 x 128 block scales follow their blocks:
 * w_s = the three forward scale grids ([n][I/128][d/128], .., [n][d/128][I/128])
 * and wt_s = {[n][I/128][d/128], [n][d/128][2I/128]}; NULL otherwise.  The
 * copies are bit-exact.  Rebuild them whenever the weights change.
 * n = N_r for the routed and N_s for the shared experts.  (Pointer arrays are
 * host memory; their elements are device pointers.)
 */
int moe_transpose_expert_weights(const moe_shape *shape, int32_t n, const void *const *w, const float *const *w_s,
                                 void *const *wt, float *const *wt_s, void *stream);

/*
 * moe_backward -- gradient of the layer (§2.1.2) for the selection that
 * moe_forward made, given dout = dL/dh'_t [T][d]; the selection and the bias
 * are piecewise constant and take no gradient (reading: the balancing bias
 * moves only by the moe_bias_update rule).  For output row t,
 *   dy_{t,j} = g_{t,j} dout_t,   dg_{t,j} = dout_t . y_{t,j}   (y = expert output)
 *   expert (SwiGLU h = SiLU(a) * b, a = W_gate x, b = W_up x, y = W_down h):
 *     dh = W_down^T dy,  da = dh b SiLU'(a),  db = dh SiLU(a),
 *     dx = W_gate^T da + W_up^T db,
 *     dW_down = sum dy h^T,  dW_gate = sum da x^T,  dW_up = sum db x^T
 *   gate g_j = rs s_j / D, D = sum_k s_k over the selected k (rs = routed_scale):
 *     ds_j = rs (dg_j / D - (sum_k dg_k s_k) / D^2),  dz_j = ds_j s_j (1 - s_j)
 *     (z = u . e, s = sigmoid(z)),
 *   du_t = sum_j dx_{t,j} + sum_shared dx + sum_j dz_j e_{sel_j},
 *   de_i = sum over slots routed to i of dz u_t.
 * E4M3 layers (§3.3: Fprop, Dgrad and Wgrad GEMMs in FP8): the Dgrad GEMMs take
 * dy, dout and [da | db] in 1 x 128 tiles along their reduction with the
 * transposed 128 x 128 weight blocks; the Wgrad GEMMs take both operands in
 * 128 x 1 tiles along each expert's rows (runs of 128 from its first row):
 * dy, dout, [da | db], and the forward's cached 1 x 128 tiles of H and u,
 * re-tiled; fp32 accumulation per run with both column scales.  The router
 * chain (dg, dz, du's centroid term, dgate_w) stays in fp32.
 * (With MOE_ADD_RESIDUAL the residual's own gradient, dout, is the caller's
 * to add: du holds the layer's part only.)
 * Inputs: u, gate_w, the weights and (E4M3) their scales exactly as passed to
 * moe_forward; routed_wt / routed_wt_s from moe_transpose_expert_weights,
 * shared_* likewise (NULL when N_s == 0); *_s and *_wt_s are NULL for
 * fp32 / bf16 layers.  fwd_ws/fwd_ws_bytes: the forward workspace of the
 * moe_forward call whose output dout refers to, untouched since (it holds the
 * scores, selection, dispatch, H and Y, which are the saved activations,
 * and with MOE_SAVE_SWIGLU_INPUTS the SwiGLU inputs a and b).
 * Storage: dout, du and the weight gradients in act_dtype (bf16 for E4M3
 * layers).  Outputs: du [T][d]; optional (NULL to skip): dgate_w [N_r][d]
 * fp32, d_routed_w = {dW_gate, dW_up, dW_down} (layout of the forward weights,
 * act_dtype), d_shared_w likewise, dtopk_w [T][K] fp32 = dL/dg.  Gradients
 * are written, not accumulated.  Sums run in fp32 in a fixed order
 * (deterministic).  ws: moe_backward_workspace_bytes(shape).
 * Errors: MOE_ERR_WORKSPACE when fwd_ws_bytes is smaller than
 * moe_workspace_bytes(shape, MOE_WS_FORWARD); MOE_ERR_INVALID_ARG for a NULL
 * required pointer or scale.
 */
int moe_backward(const moe_shape *shape, const void *u, const void *gate_w, const void *const *routed_w,
                 const float *const *routed_s, const void *const *routed_wt, const float *const *routed_wt_s,
                 const void *const *shared_w, const float *const *shared_s, const void *const *shared_wt,
                 const float *const *shared_wt_s, const void *fwd_ws, size_t fwd_ws_bytes, const void *dout, void *du,
                 float *dgate_w, void *const *d_routed_w, void *const *d_shared_w, float *dtopk_w, void *ws,
                 size_t ws_bytes, void *stream);

/*
 * moe_backward_timed -- moe_backward that also records caller-created HIP
 * events on `stream` at its stage boundaries:
 *   stage_events[0] before the combine gradient   [1] after it (dY, dg; e4m3: their 1 x 128 tiles)
 *   [2] after dH = dY W_down                      [3] after the SwiGLU gradient pass ([dA | dB], tiled)
 *   [4] after dX = [dA | dB] [W_gate ; W_up]      [5] after the token pass (du, dz)
 *   [6] after the centroid gradient               [7] after the weight-gradient operands' tiling
 *   [8] after dW_down                             (e4m3: run bases and 128 x 1 tiles; else empty)
 *   [9] after dW_gate / dW_up
 * NULL entries (or a NULL array, 10 entries otherwise) are skipped; skipped
 * optional outputs leave their stage empty.  Results are identical to
 * moe_backward.
 */
int moe_backward_timed(const moe_shape *shape, const void *u, const void *gate_w, const void *const *routed_w,
                       const float *const *routed_s, const void *const *routed_wt, const float *const *routed_wt_s,
                       const void *const *shared_w, const float *const *shared_s, const void *const *shared_wt,
                       const float *const *shared_wt_s, const void *fwd_ws, size_t fwd_ws_bytes, const void *dout,
                       void *du, float *dgate_w, void *const *d_routed_w, void *const *d_shared_w, float *dtopk_w,
                       void *ws, size_t ws_bytes, void *stream, void *const *stage_events);

/* Workspace bytes for moe_backward (0 when rejected). */
size_t moe_backward_workspace_bytes(const moe_shape *shape);

/* ------------------------------------------------------------------------ */
/* gate: routing from logits                                                */

enum { MOE_SCORE_SIGMOID = 0, MOE_SCORE_SOFTMAX = 1 };

/* moe_gate_rule.flags */
#define MOE_GATE_RENORM 1u      /* weights are divided by their sum */
#define MOE_GATE_GROUP_MAX 2u   /* a group scores its largest choice value, else the sum of its two largest */

/*
 * How a gate scores, chooses and weighs.  Limits (MOE_ERR_UNSUPPORTED
 * otherwise): n_experts <= 1024, n_experts % n_groups == 0,
 * 1 <= topk_groups <= n_groups <= 64, 1 <= topk <= 32,
 * topk <= topk_groups * n_experts / n_groups, T * topk < 2^31.
 */
typedef struct moe_gate_rule {
    int64_t T;              /* tokens (T >= 0; T == 0 is a no-op) */
    int32_t n_experts;
    int32_t n_groups;       /* group g = experts [g * n_experts / n_groups, ...); 1: no groups */
    int32_t topk_groups;    /* groups a token may use */
    int32_t topk;           /* K: experts per token */
    int32_t score;          /* MOE_SCORE_SIGMOID | MOE_SCORE_SOFTMAX */
    int32_t logits_dtype;   /* logits and dlogits: MOE_F32 | MOE_BF16 */
    float routed_scale;     /* factor on every weight */
    uint32_t flags;         /* MOE_GATE_RENORM | MOE_GATE_GROUP_MAX, or 0 */
} moe_gate_rule;

/*
 * moe_gate -- scores, choice and weights from the logits z of any gate product
 * (moe_route has its own gate product and sigmoid scores only):
 *   s_i = 1 / (1 + exp(-z_i)), or
 *   s_i = exp(z_i - max z) * (1 / sum_k exp(z_k - max z)), the sum rounded once to fp32;
 *   a logit of -infinity or NaN is an expert out of use: s_i = 0;
 *   choice value c_i = s_i + bias_i (one fp32 add), -infinity for an expert out
 *     of use or where the sum is NaN;
 *   a group's score is the sum of its two largest c (its only one where one is
 *     above -infinity), or its largest; the topk_groups best groups are kept,
 *     the c of the others become -infinity;
 *   topk_idx[t] = the topk largest c in decreasing order; every tie goes to the
 *     lower index;
 *   topk_w[t][j] = routed_scale * s_j, with MOE_GATE_RENORM routed_scale *
 *     (s_j / (s_0 + ... + s_{K-1})), the sum from left to right; 0 where
 *     c_j = -infinity (fewer experts in use than slots: such slots hold the
 *     lowest indices left, so that a token's experts stay distinct and
 *     moe_permute takes them) and where the sum is 0.
 * logits [T] rows of n_experts values, ld elements apart (ld >= n_experts);
 * bias [n_experts] fp32 or NULL; scores_out [T][n_experts] fp32 or NULL;
 * topk_idx [T][K] int32; topk_w [T][K] fp32.  All arithmetic is fp32 (the
 * softmax sum fp64).  No workspace.
 */
int moe_gate(const moe_gate_rule *rule, const void *logits, int64_t ld, const float *bias, float *scores_out,
             int32_t *topk_idx, float *topk_w, void *stream);

/*
 * moe_gate_backward -- dL/dz for the choice that moe_gate made (the choice is
 * piecewise constant: it and the bias take no gradient).  With g = dtopk_w,
 * S = routed_scale, D = sum of the chosen s, over the slots whose weight is not 0:
 *   ds_j = S g_j, with MOE_GATE_RENORM S (g_j - sum_k g_k s_k / D) / D,
 *   plus dscores_i at every expert when dscores is given (a loss on scores_out);
 *   sigmoid: dz_i = ds_i s_i (1 - s_i);  softmax: dz_i = s_i (ds_i - sum_k ds_k s_k).
 * An expert out of use gets 0.  s is recomputed from the logits.
 * logits, ld, topk_idx, topk_w as given to and by moe_gate (indices distinct
 * within a token); dtopk_w [T][K] fp32; dscores [T][n_experts] fp32 or NULL;
 * dlogits [T] rows of n_experts values in logits_dtype, dld elements apart,
 * every one of which is written.  Sums run in fp32, in an order that T and n_experts
 * choose; none changes from call to call.
 */
int moe_gate_backward(const moe_gate_rule *rule, const void *logits, int64_t ld, const int32_t *topk_idx,
                      const float *topk_w, const float *dtopk_w, const float *dscores, void *dlogits, int64_t dld,
                      void *stream);

/* ------------------------------------------------------------------------ */
/* MX4: microscaled 4-bit floating point                                    */

/*
 * An MX4 matrix (OCP Microscaling Formats v1.0, element type E2M1, scale type
 * E8M0): blocks of 32 values along a row share a scale 2^(s - 127) held in one
 * byte s; a value is a 4-bit code (sign, then 0, 0.5, 1, 1.5, 2, 3, 4, 6) times
 * its block's scale.  A row of `cols` values takes R = ceil(cols / 128) runs:
 * 64 R code bytes (value 2i in the low half of byte i) and 4 R scale bytes;
 * what lies past the last value is 0 (codes 0; scale 127 in blocks of zeros).
 * With cols % 128 == 0 the rows are thus cols / 2 and cols / 32 dense bytes.
 * Code arrays must be 16-byte aligned and scale arrays 4-byte aligned.
 */

/*
 * moe_quantize_mx4 -- x [rows] rows of cols values (x_dtype MOE_F32 or
 * MOE_BF16), ld elements apart, to codes q [rows][64 R] and scales s [rows][4 R]:
 * s = max(exponent field of the block's largest magnitude - 2, 0), 127 for a
 * block of zeros; code = nearest to x / 2^(s - 127), ties to the even code,
 * magnitudes above 6 to 6 (the largest scaled magnitude lies in [4, 8)).
 * A block that holds an infinity or NaN gets s = 255 (NaN) and codes 0.
 */
int moe_quantize_mx4(int64_t rows, int32_t cols, int32_t x_dtype, const void *x, int64_t ld, uint8_t *q, uint8_t *s,
                     void *stream);

/*
 * moe_dequantize_mx4 -- the values of codes q and scales s as y_dtype (MOE_F32 or
 * MOE_BF16), rows ld elements apart.  Exact in both types; s = 255 gives NaN, and
 * values past the largest number infinity (magnitudes 4 and 6 at s = 253, 2 and up at
 * 254; moe_quantize_mx4 gives no scale above 252 but 255).
 * quantise + dequantise is the rounding of training with MX4 weights: the bf16
 * values go through moe_forward and moe_backward, whose weight gradients are
 * then those of the unrounded weights by the straight-through rule.
 */
int moe_dequantize_mx4(int64_t rows, int32_t cols, const uint8_t *q, const uint8_t *s, int32_t y_dtype, void *y,
                       int64_t ld, void *stream);

/*
 * moe_grouped_ffn_mx4 -- moe_grouped_ffn on MX4 weights and activations:
 *   a = W_gate[e] x_r,  b = W_up[e] x_r,  h = Q(a / (1 + exp(-a)) * b),  y[r] = W_down[e] h
 * for the rows r in [offsets[e], offsets[e+1]) of expert e, x_r = x[gather[r]]
 * (gather NULL: x[r]); Q is moe_quantize_mx4's rounding of the fp32 values;
 * products of codes and scales are summed in fp32; y [max_rows][d] is bf16.
 * Deterministic: no sum's order changes from call to call.  max_rows, n_exp, d, inter,
 * the card's compute units and whether the scales lie at multiples of 16 bytes choose
 * it, so a row among more rows can differ in the last bit of a sum (and, where
 * that meets a rounding boundary, by a code of h).
 * Infinities and NaN go where the formula takes them: a block of scale 255 (NaN) of a row of x makes its y[r]
 * NaN, one of a gate or up row of expert e (or an H that is infinite or NaN) every y[r] whose H it meets, one of
 * a row of W_down[e] that feature of expert e's rows; nothing else changes.
 * n_exp <= 1024 experts; offsets [n_exp+1] int32 on the device, offsets[0] = 0,
 * non-decreasing, offsets[n_exp] <= max_rows.  d and inter are any positive
 * sizes (rows padded to whole runs as above).
 * x codes, x_scales [*]; w = {W_gate, W_up, W_down} codes [n_exp][inter] rows of d,
 * [n_exp][inter] of d, [n_exp][d] rows of inter; w_scales their scales.
 * (The arrays of 3 pointers are host memory, their elements device pointers.)
 * ws: moe_ffn_mx4_workspace_bytes(max_rows, inter).
 */
int moe_grouped_ffn_mx4(int32_t n_exp, const int32_t *offsets, int64_t max_rows, const int32_t *gather, int32_t d,
                        int32_t inter, const uint8_t *x, const uint8_t *x_scales, const uint8_t *const *w,
                        const uint8_t *const *w_scales, void *y, void *ws, size_t ws_bytes, void *stream);

/* Workspace bytes for moe_grouped_ffn_mx4: 68 bytes a row and run of 128 of inter, and less than 1 KB. */
size_t moe_ffn_mx4_workspace_bytes(int64_t max_rows, int32_t inter);

/* ------------------------------------------------------------------------ */
/* products of experts                                                      */

/*
 * One matrix product per expert over ragged rows, for experts of any kind: expert e owns
 * the rows r in [offsets[e], offsets[e+1]) of a batch of max_rows rows.
 *   n_exp <= 1024 experts; offsets [n_exp+1] int32 on the device, offsets[0] = 0,
 *   non-decreasing, offsets[n_exp] <= max_rows < 2^31 (moe_permute gives them).  Rows from
 *   offsets[n_exp] on are neither read nor written; an expert may have none.  gather [max_rows] int32: each a row
 *   of x, which is not checked.  Both 4-byte aligned.
 *   w [n_exp][out][in] dense; in and out any sizes up to 2^20 with in * out <= 2^29.
 *   Rows of the other matrices are *_ld elements apart (*_ld >= the row's values); addresses
 *   and rows at multiples of 16 bytes are the fast case, any other is taken.
 * Products are summed in fp32 (8-bit integers in int32, exactly) and rounded once to the
 * output's type, MOE_BF16 or MOE_F32.  Deterministic: the order of a sum depends on the sizes, the
 * alignment and the card alone, so a row among more rows can differ in a sum's last bit.
 * Infinities and NaN go where the formula takes them, and to no other row or feature.
 * Results share no memory with the other arguments.
 */

/*
 * moe_grouped_product -- y[r] = W[e] x[gather[r]] (gather NULL: x[r]).
 * x bf16 rows of in values, w bf16, y rows of out values in y_dtype.
 */
int moe_grouped_product(int32_t n_exp, const int32_t *offsets, int64_t max_rows, const int32_t *gather, int32_t in,
                        int32_t out, const void *x, int64_t x_ld, const void *w, int32_t y_dtype, void *y, int64_t y_ld,
                        void *stream);

/*
 * moe_grouped_product_dx -- its gradient at the rows of x: dx[r] = W[e]^T dy[r], a row for every row r (a
 * token's rows are added up by moe_combine with weights of 1).
 * dy bf16 rows of out values, w as above, dx rows of in values in dx_dtype.
 */
int moe_grouped_product_dx(int32_t n_exp, const int32_t *offsets, int64_t max_rows, int32_t in, int32_t out,
                           const void *dy, int64_t dy_ld, const void *w, int32_t dx_dtype, void *dx, int64_t dx_ld,
                           void *stream);

/*
 * moe_grouped_product_dw -- its gradient at the weights: dw[e] = sum over r of dy[r] x[gather[r]]^T, with
 * `accumulate` (MOE_F32 only) added to what dw holds.  dw [n_exp][out][in] dense in dw_dtype, every value of
 * which is written: 0 (or kept) for an expert without rows.
 */
int moe_grouped_product_dw(int32_t n_exp, const int32_t *offsets, int64_t max_rows, const int32_t *gather, int32_t in,
                           int32_t out, const void *x, int64_t x_ld, const void *dy, int64_t dy_ld, int32_t dw_dtype,
                           void *dw, int32_t accumulate, void *stream);

/*
 * moe_quantize_int8 -- x [rows] rows of cols values (x_dtype MOE_F32 or MOE_BF16), ld elements apart, to
 * 8-bit integers with a scale a row: with m = max(largest magnitude of the row, 2^-100),
 *   s = m / 127,   code = x * (127 / m) to the nearest whole number, ties to even
 * (fp32 operations, each rounded once; codes lie in -127 .. 127).  A row with an infinity or NaN gets s = NaN and
 * codes 0.  q [rows] rows of ceil(cols / 128) * 128 codes, zeros behind the last, 16-byte aligned; s [rows] fp32.
 * Rows of tokens get a scale a token, rows of weights [n_exp * out] a scale an output channel.
 */
int moe_quantize_int8(int64_t rows, int32_t cols, int32_t x_dtype, const void *x, int64_t ld, int8_t *q, float *s,
                      void *stream);

/*
 * moe_grouped_product_int8 -- y[r][f] = (sum over k of xq[gather[r]][k] wq[e][f][k]) * x_scales[gather[r]] *
 * w_scales[e][f], multiplied from left to right in fp32.  x, w codes and scales of moe_quantize_int8 (w of
 * n_exp * out rows of in values); in <= 131072, so that no sum leaves 32 bits; an expert's codes at most 2^30 bytes.
 */
int moe_grouped_product_int8(int32_t n_exp, const int32_t *offsets, int64_t max_rows, const int32_t *gather, int32_t in,
                             int32_t out, const int8_t *x, const float *x_scales, const int8_t *w, const float *w_scales,
                             int32_t y_dtype, void *y, int64_t y_ld, void *stream);

/* ------------------------------------------------------------------------ */
/* an optimiser's step on the experts' matrices                             */

/*
 * moe_orthogonalize -- brings each of n matrices g [n][rows][cols] (dense, g_dtype MOE_F32 or MOE_BF16) near its
 * nearest orthogonal matrix by Newton-Schulz steps, as the Muon optimiser does with the momentum of a weight's gradient:
 *   X = g / (|g|_F + eps), turned over where rows > cols;
 *   for each step k:  S = X X^T,  X <- a_k X + (b_k S + c_k S S) X;
 *   y = scale * X, turned back, bf16 [n][rows][cols] dense.
 * coeffs (host) holds a_k, b_k, c_k of the steps in turn, 3 * steps floats; 1 <= steps <= 64; eps >= 0.
 * The norm is held in 64 bits.  Operands of products are pairs of bf16, which keep 16 significant bits, with sums in fp32;
 * the X of a_k X has all 24 bits of fp32 as long as the a of the steps left multiply by more than 64, so that rounding stays
 * below a quarter of y's own in matrices of low rank too.
 * A matrix of zeros gives zeros (with eps > 0), one that holds an infinity or NaN gives NaN; other matrices do not
 * change.  Deterministic: sums depend on n, rows, cols and the card alone.  y may be g where g is bf16 (the same address);
 * otherwise they share no memory (a part of X lies in y between the steps).
 * With sides rounded up to multiples of 32: a matrix of at most 2^28 values, n of them below 2^40; the smaller side at
 * most 16384, n at most 65535.
 * ws: moe_orthogonalize_workspace_bytes(n, rows, cols).
 */
int moe_orthogonalize(int64_t n, int32_t rows, int32_t cols, int32_t g_dtype, const void *g, int32_t steps,
                      const float *coeffs, float eps, float scale, void *y, void *ws, size_t ws_bytes, void *stream);

/* Workspace bytes for moe_orthogonalize: 8 r (r + c) a matrix, r and c its smaller and larger side rounded up to
 * multiples of 32, and up to 512 more a matrix and 1024 (0 when rejected). */
size_t moe_orthogonalize_workspace_bytes(int64_t n, int32_t rows, int32_t cols);

/* ------------------------------------------------------------------------ */
/* helpers                                                                  */

enum { MOE_WS_ROUTE = 0, MOE_WS_PERMUTE = 1, MOE_WS_FORWARD = 2 };

/* Workspace bytes for moe_route / moe_permute / moe_forward at this shape,
 * or 0 when the shape is rejected (see moe_last_error). */
size_t moe_workspace_bytes(const moe_shape *shape, int which);

/* Workspace bytes for moe_grouped_ffn with max_rows rows (0 when rejected). */
size_t moe_ffn_workspace_bytes(const moe_shape *shape, int64_t max_rows);

/*
 * moe_bias_update -- one auxiliary-loss-free step (§2.1.2; gamma = 0.001 in
 * §4.2): mean = fp32(T*K) / fp32(N_r);
 *   bias[i] = bias[i] + gamma * sign(mean - counts[i])   (sign(0) = 0)
 * (reading: "overloaded" = load above the mean; an exact tie leaves b_i).
 * counts [N_r] int32, bias [N_r] fp32 updated in place.
 */
int moe_bias_update(const moe_shape *shape, const int32_t *counts, float *bias, float gamma, void *stream);

/*
 * moe_seq_balance -- complementary sequence-wise balance statistic (§2.1.2: a
 * tiny loss alpha * sum_i f_i P_i kept beside the bias rule; §4.2: alpha =
 * 0.0001).  The pages name f_i and P_i without defining them; reading, for a
 * sequence of Ts tokens:
 *   f_i = N_r / (K * Ts) * (slots of the sequence routed to expert i),
 *   P_i = (1/Ts) * sum_t s_{i,t} / sum_k s_{k,t}   (affinity share over all
 *         routed experts, un-biased s).
 * Sequences are consecutive runs of seq_len tokens of the batch (the last one
 * may be shorter): n_seq = ceil(T / seq_len).
 * scores [T][N_r] fp32 (moe_route's scores_out), topk_idx [T][K] int32.
 * loss [n_seq] fp32; counts [n_seq][N_r] int32 and share [n_seq][N_r] fp32
 * (P_i) are optional (NULL).  fp32 sums in a fixed order (deterministic).
 * ws: moe_seq_balance_workspace_bytes(shape, seq_len).
 * Errors: MOE_ERR_INVALID_ARG for seq_len < 1 or a NULL required pointer.
 */
int moe_seq_balance(const moe_shape *shape, const float *scores, const int32_t *topk_idx, int64_t seq_len,
                    float alpha, float *loss, int32_t *counts, float *share, void *ws, size_t ws_bytes,
                    void *stream);

/* Workspace bytes for moe_seq_balance (0 when rejected). */
size_t moe_seq_balance_workspace_bytes(const moe_shape *shape, int64_t seq_len);

/*
 * moe_quantize_1x128 -- Q over 1x128 tiles of each row of x [rows][cols]
 * (x_dtype MOE_F32 or MOE_BF16; cols % 128 == 0): q [rows][cols] e4m3,
 * s [rows][cols/128] fp32 (§3.3 activation tiles).
 */
int moe_quantize_1x128(int64_t rows, int32_t cols, int32_t x_dtype, const void *x, uint8_t *q, float *s,
                       void *stream);

/*
 * moe_quantize_weights_128x128 -- Q over 128x128 blocks of nmat matrices
 * w [nmat][rows][cols] (w_dtype MOE_F32 or MOE_BF16; rows, cols % 128 == 0):
 * q [nmat][rows][cols] e4m3, s [nmat][rows/128][cols/128] fp32 (§3.3 weight
 * blocks).  Weight preparation, not part of the per-step path.
 */
int moe_quantize_weights_128x128(int64_t nmat, int32_t rows, int32_t cols, int32_t w_dtype, const void *w,
                                 uint8_t *q, float *s, void *stream);

/*
 * moe_quantize_128x1 -- Q over 128x1 tiles down the rows of segments, the
 * operands of the FP8 weight-gradient GEMMs.  §3.3 runs Wgrad in FP8 and
 * names 1x128 activation tiles and 128x128 weight blocks, but no tile for a
 * GEMM that reduces over tokens.  Reading (not the page's text): a tile is
 * 128 consecutive elements along the GEMM's reduction, which for a weight
 * gradient runs down the token rows, i.e. 128x1; the tile origin is not
 * stated either, read as runs of 128 list rows from each segment's first row.
 *   n_seg segments; offsets [n_seg+1] (device, int32, offsets[0] >= 0,
 *   nondecreasing, offsets[n_seg] <= max_rows): segment e owns list rows
 *   offsets[e] .. offsets[e+1]-1, cut into runs of 128 rows from its first
 *   row (the last run of a segment may be shorter);
 *   list row r reads x row gather[r] (gather NULL: row r);
 *   x [.][cols] MOE_BF16, or MOE_E4M3 codes with 1x128 fp32 scales
 *   x_s [.][cols/128] (decoded to fp32 before the re-quantisation);
 *   q [offsets[n_seg]][cols] e4m3 codes, rows offsets[0].. written;
 *   s [n_blocks][cols] fp32: one scale per run and column, runs numbered
 *   segment by segment; block_base [n_seg+1] (device, int32, out): the
 *   first run of each segment, block_base[n_seg] = n_blocks
 *   <= max_rows/128 + n_seg.
 * A scale is amax/448 over its run's column (1 for an all-zero column);
 * codes are round-to-nearest-even of clamp(v/scale, -448, 448).
 * Offsets that break the stated order are undefined behaviour.
 * Errors: INVALID_ARG for negative sizes or a NULL buffer; UNSUPPORTED for
 * cols % 128 != 0 or another x_dtype.  n_seg == 0 does nothing.
 */
int moe_quantize_128x1(int32_t n_seg, const int32_t *offsets, int64_t max_rows, int32_t cols, int32_t x_dtype,
                       const void *x, const float *x_s, const int32_t *gather, uint8_t *q, float *s,
                       int32_t *block_base, void *stream);

/* Message for the calling thread's last failed call ("" if none). */
const char *moe_last_error(void);

/* Library version string. */
const char *moe_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H_ */
