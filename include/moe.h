/*
 * moe.h -- C ABI of libmoe.so, a sparse mixture-of-experts layer (forward,
 * and the backward of its training pass) for AMD Instinct MI355X (gfx950).
 *
 * The layer (defined on "Mixture of experts and speculative decoding", section
 * "Opening the hood: the MoE layer precisely", and on "MoE inference: the call
 * centre with 256 specialists ...", section "The bare mechanism"):
 *
 *   r      = x W_r^T (+ logit_bias)                 router scores, fp32
 *   key    = r + select_bias                        selection key (one fp32 add)
 *   TopK   = the k largest keys, ties to the lower expert index,
 *            slot 0 = largest key
 *   g      = softmax over the k kept r (unbiased)   gates, sum to 1
 *   E_e(x) = W_down[e] ( SiLU(W_gate[e] x) * (W_up[e] x) )   SwiGLU expert
 *   y      = sum_{slot} g_slot E_{TopK_slot}(x) + sum_s E_shared_s(x)
 *
 * plus the load-balance statistics of "Keeping the experts busy" (same page)
 * and of the routing-collapse passage of "Mixture of Experts and Guided
 * Decoding": f_e = count_e / (T k), P_e = mean_t softmax(r_t)_e,
 * loss = alpha * N * sum_e f_e P_e.
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every tensor pointer is a DEVICE pointer to a dense row-major array owned
 *    by the caller.  The library never allocates, frees, or synchronises the
 *    device; all work is enqueued on `stream` (a hipStream_t; NULL = the null
 *    stream) and completes asynchronously.
 *  - Arguments are validated on the host before anything is enqueued; on any
 *    error nothing is launched and the status says why.  A HIP launch failure
 *    returns MOE_ERR_HIP.
 *  - Weights use the linear layer's [out, in] layout: W_r [N, d],
 *    W_gate/W_up [N, F, d], W_down [N, d, F]; shared experts [S, F, d] and
 *    [S, d, F].  x and y are [T, d].  The element type of x, y and every weight
 *    is cfg->dtype (expert weights: see moe_weight_format); biases, logits,
 *    gates, scales and statistics are fp32.
 *  - Arithmetic: bf16 inputs are multiplied on the matrix cores with fp32
 *    accumulation; the expert hidden activations and per-expert outputs are
 *    held in the input dtype (bf16 rounding to nearest even); y is rounded once.
 *  - Results are deterministic: the same inputs give bitwise the same outputs.
 *  - Calls are thread-safe; concurrent calls must use distinct workspaces.
 *  - Supported sizes: 1 <= k <= min(N, 16), N <= 512, 0 <= S <= 4, capacity >= 0,
 *    d and F positive multiples of 64, T >= 0 (T = 0 launches nothing and
 *    returns MOE_OK, except that moe_layer_backward writes zero weight
 *    gradients); FP8 expert weights with dtype MOE_BF16 only.  Other sizes
 *    return MOE_ERR_UNSUPPORTED.
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
  MOE_ERR_INVALID_ARG = 1,  /* null required pointer, k > N, negative size ... */
  MOE_ERR_UNSUPPORTED = 2,  /* valid but outside the supported sizes above */
  MOE_ERR_WORKSPACE = 3,    /* workspace NULL or smaller than moe_workspace_size */
  MOE_ERR_HIP = 4           /* a HIP runtime call or kernel launch failed */
} moe_status;

typedef enum { MOE_F32 = 0, MOE_BF16 = 1 } moe_dtype;

/* Storage of the expert weights (routed and shared; W_r always uses dtype).
 * The pages size expert weights at one byte per parameter for FP8 ("MoE
 * inference: the call centre with 256 specialists ...", the weight-memory
 * estimate under "Total memory") but define no format; this library takes
 * OCP FP8 E4M3 codes (bias 7, no infinities, S.1111.111 = NaN, largest
 * finite 448) with one fp32 scale per output channel:
 *   W[e][n][j] = decode(code[e][n][j]) * scale[e][n]
 * (n = row of the [out, in] matrix: F rows of W_gate/W_up, d rows of W_down).
 * Decoded values are exact in bf16; the scale multiplies each fp32 sum in
 * the GEMM epilogue (before SiLU for gate and up).  A NaN code gives NaN. */
typedef enum {
  MOE_WEIGHTS_DTYPE = 0,    /* expert weights in cfg->dtype, like x and y     */
  MOE_WEIGHTS_FP8_E4M3 = 1  /* 1-byte E4M3 codes + fp32 scales (dtype BF16)   */
} moe_weight_format;

/* Layer sizes.  T tokens, d_model, N routed experts, top_k kept per token,
 * d_ff hidden size of every expert (routed and shared), n_shared always-on
 * experts, dtype a moe_dtype.
 *
 * capacity: 0 = dropless.  C > 0 caps every routed expert at C (token, slot)
 * assignments per call ("Mixture of experts and speculative decoding",
 * "Keeping the experts busy": the extras are dropped).  Kept are an expert's
 * first C assignments in token order; a dropped assignment adds nothing to y
 * (the token's other gates are not renormalised).  topk_idx, topk_gate,
 * counts and prob_sum still describe the router's choice before dropping.
 *
 * weight_format: a moe_weight_format (0 = weights in dtype). */
typedef struct {
  int32_t T;
  int32_t d_model;
  int32_t n_experts;
  int32_t top_k;
  int32_t d_ff;
  int32_t n_shared;
  int32_t dtype;
  int32_t capacity;
  int32_t weight_format;
} moe_config;

/* Layer parameters (device pointers, caller-owned, read-only). */
typedef struct {
  const void* w_router;     /* [N, d]                                         */
  const void* w_gate;       /* [N, F, d]   (unused by moe_route)              */
  const void* w_up;         /* [N, F, d]   (unused by moe_route)              */
  const void* w_down;       /* [N, d, F]   (unused by moe_route)              */
  const void* ws_gate;      /* [S, F, d] or NULL when S = 0                   */
  const void* ws_up;        /* [S, F, d] or NULL when S = 0                   */
  const void* ws_down;      /* [S, d, F] or NULL when S = 0                   */
  const float* logit_bias;  /* [N] added to the logits (moves selection,
                               gates and P), or NULL                          */
  const float* select_bias; /* [N] added to the selection key only (the
                               auxiliary-loss-free routing bias of "The bare
                               mechanism"), or NULL                           */
  /* Per-output-channel scales of FP8 expert weights (MOE_WEIGHTS_FP8_E4M3;
     ignored otherwise).  The routed ones are required by moe_layer_forward,
     the shared ones when S > 0.                                              */
  const float* w_gate_scale;  /* [N, F] */
  const float* w_up_scale;    /* [N, F] */
  const float* w_down_scale;  /* [N, d] */
  const float* ws_gate_scale; /* [S, F] */
  const float* ws_up_scale;   /* [S, F] */
  const float* ws_down_scale; /* [S, d] */
} moe_weights;

/* Routing outputs (device pointers, caller-owned, written by the call).  For
 * moe_layer_forward every field is optional (NULL = not wanted); moe_route
 * requires topk_idx and topk_gate.  f, P and aux are the balance statistics
 * moe_balance_stats computes (bitwise the same values), produced inside the
 * call's grouping step instead of a launch of their own. */
typedef struct {
  float* logits;      /* [T, N]  r including logit_bias                       */
  int32_t* topk_idx;  /* [T, k]  chosen experts, slot 0 = largest key          */
  float* topk_gate;   /* [T, k]  softmax over the kept unbiased logits        */
  int32_t* counts;    /* [N]     (token, slot) assignments per routed expert  */
  float* prob_sum;    /* [N]     sum over tokens of softmax(r_t) over all N   */
  float* f;           /* [N]     counts / (T k)                               */
  float* P;           /* [N]     prob_sum / T                                 */
  float* aux;         /* [2]     N sum_e f_e P_e, then balance_alpha times it */
  float balance_alpha;/*         coefficient of aux[1] (not a pointer)        */
} moe_routing;

/* Stage markers for moe_layer_forward_timed. */
enum {
  MOE_STAGE_ROUTE = 0,      /* router GEMM + top-k + gates + block statistics */
  MOE_STAGE_PERMUTE = 1,    /* per-expert offsets, tile lists, token grouping  */
  MOE_STAGE_EXPERT_UP = 2,  /* grouped gate/up GEMM with SiLU(gate)*up         */
  MOE_STAGE_EXPERT_DOWN = 3,/* grouped down GEMM                               */
  MOE_STAGE_COMBINE = 4,    /* gate-weighted combine into y                    */
  MOE_STAGE_COUNT = 5
};

/* Bytes of device workspace moe_layer_forward / moe_route need for `cfg`
 * (a multiple of 256).  Returns 0 for an invalid or unsupported cfg. */
size_t moe_workspace_size(const moe_config* cfg);

/* How moe_layer_forward runs `cfg` on the current device (kernel choices and
 * reduction splits, all decided on the host from cfg and the device's
 * compute-unit count), for tests and profiling.  The kernels and splits do
 * not change the results' definition; they only change where the work runs.
 *   up_kernel / down_kernel: 0 = register-staged tiles (fp32 layers and
 *     batches of few rows per expert), 1 = large-tile kernel (bf16 prefill);
 *   up_tile_rows / down_tile_rows: rows per tile of each grouped GEMM;
 *   route_split: workgroups the router GEMM's reduction is split over
 *     (1 = the router GEMM and the selection run in one kernel);
 *   route_kernel: 0 = the router kernel (64-token tiles), 1 = the router
 *     GEMM on the large-tile expert GEMM kernel (256-token tiles, bf16, 128
 *     to 256 experts, 2048 or more tokens); either way a selection kernel
 *     adds the route_split partial logits in a fixed order when it is > 1;
 *   down_split: pieces every row of the down pass is split into over its
 *     reduction (decode shapes), else 1;
 *   tail_split_cols: column tiles of the down pass when its last row tiles
 *     may be split over the reduction (0 = never);
 *   up_narrow_tails / down_narrow_tails: 1 when an expert's last row tile
 *     of at most 64 rows runs as one tile over two column tiles (the
 *     ping-pong large-tile kernel, an even number of column tiles; the down
 *     pass only with at most 384 rows per expert on average);
 *   compute_units: the device's compute units, as the plan used them;
 *   all_token_pass: 1 when every expert (routed and shared) runs on all T
 *     tokens: batches of at most 32 tokens, at most 64 experts, bf16 or
 *     fp32 expert weights, where one 32-row tile per expert holds the whole
 *     batch and (nearly) every expert is chosen anyway (expected idle
 *     experts N (1 - k/N)^T at most 1/2).
 *     The routing then runs inside the gate/up launch and only the combine
 *     uses it; the result is the same y (each row's arithmetic is unchanged,
 *     rows no slot chose are computed and never read);
 *   split_plan_offset: byte offset in the workspace of the split plan each
 *     forward writes there on the device, int32 [4] = {pieces, first split
 *     row, rows per piece, split row tiles} (pieces = 0: nothing split);
 *   workspace_bytes: moe_workspace_size(cfg).
 * MOE_ERR_INVALID_ARG / MOE_ERR_UNSUPPORTED for a bad cfg or NULL out. */
typedef struct {
  int32_t up_kernel;
  int32_t up_tile_rows;
  int32_t down_kernel;
  int32_t down_tile_rows;
  int32_t route_split;
  int32_t route_kernel;
  int32_t down_split;
  int32_t tail_split_cols;
  int32_t up_narrow_tails;
  int32_t down_narrow_tails;
  int32_t compute_units;
  int32_t all_token_pass;
  uint64_t split_plan_offset;
  uint64_t workspace_bytes;
} moe_plan_info;

moe_status moe_forward_plan(const moe_config* cfg, moe_plan_info* out);

/* Static, human-readable text for a status code (never NULL). */
const char* moe_status_string(int status);

/* Detail of the last MOE_ERR_* returned on the calling thread (static text
 * or a thread-local buffer; never NULL, "" when none). */
const char* moe_last_error(void);

/* Routing only (steps r, key, TopK, g and the statistics' raw sums):
 * x [T, d]; w->w_router, optional w->logit_bias / w->select_bias; writes
 * out->topk_idx and out->topk_gate (required) and out->logits, out->counts,
 * out->prob_sum when non-NULL.  `workspace` must hold moe_workspace_size(cfg)
 * bytes, 256-byte aligned; its contents are scratch.  The logits, selection
 * and statistics are bitwise those moe_layer_forward computes for the same
 * cfg and inputs (a batch that takes the all-token pass is routed here with
 * the same one-workgroup reduction as inside that forward). */
moe_status moe_route(const moe_config* cfg, const void* x, const moe_weights* w,
                     moe_routing* out, void* workspace, size_t ws_bytes,
                     void* stream);

/* Whole layer forward: routing as moe_route, then the SwiGLU experts on the
 * tokens routed to them (experts no token chose are never read, except in
 * the all-token pass of moe_plan_info, which runs every expert on every
 * token of a small batch and combines only the routed rows), the shared
 * experts on every token, and the combine y [T, d] (required).  Optional
 * routing outputs as described at moe_routing. */
moe_status moe_layer_forward(const moe_config* cfg, const void* x,
                             const moe_weights* w, void* y, moe_routing* out,
                             void* workspace, size_t ws_bytes, void* stream);

/* moe_layer_forward that also records stage_events[i] (hipEvent_t, created by
 * the caller) on `stream` before stage i and stage_events[MOE_STAGE_COUNT]
 * after the last one, so the caller can time each stage.  stage_events may be
 * NULL (then identical to moe_layer_forward), and so may any entry (that
 * marker is skipped: a caller timing one stage records only its two). */
moe_status moe_layer_forward_timed(const moe_config* cfg, const void* x,
                                   const moe_weights* w, void* y,
                                   moe_routing* out, void* workspace,
                                   size_t ws_bytes, void* stream,
                                   void* const* stage_events);

/* Bytes of the device array that moe_layer_forward_noalloc uses as its
 * workspace: one array per GPU the library runs on, held until the process
 * ends. */
#define MOE_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/* moe_layer_forward for callers that cannot allocate device memory: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  Same arguments, kernels and results as moe_layer_forward, but
 * no workspace argument: the workspace is a library-owned device array of
 * MOE_NOALLOC_SCRATCH_BYTES on the current GPU, so the call never allocates.
 * A cfg whose workspace (moe_workspace_size) exceeds that returns
 * MOE_ERR_WORKSPACE and launches nothing: decode batches and small prefill
 * batches fit (the Mixtral-shaped layer at 32 tokens needs 4 MB), large
 * prefill batches do not.  Every call on one GPU shares that GPU's array,
 * which keeps the last call's contents (the forward reads nothing from its
 * workspace that it has not written in the same call): calls that overlap
 * on one GPU (concurrent streams, or threads) race and must be serialised
 * by the caller. */
moe_status moe_layer_forward_noalloc(const moe_config* cfg, const void* x,
                                     const moe_weights* w, void* y,
                                     moe_routing* out, void* stream);

/* Balance statistics from the routing sums of T tokens, N experts, top-k:
 * f_out[e] = counts[e] / (T k), P_out[e] = prob_sum[e] / T,
 * aux_out[0] = N * sum_e f_e P_e, aux_out[1] = alpha * aux_out[0]
 * (all fp32 device arrays; T = 0 writes zeros).  Enqueued on `stream`. */
moe_status moe_balance_stats(int32_t T, int32_t N, int32_t k,
                             const int32_t* counts, const float* prob_sum,
                             float alpha, float* f_out, float* P_out,
                             float* aux_out, void* stream);

/* ------------------------------------------------------------- backward
 *
 * Gradients of  L = sum(y * dy) + aux_grad * alpha * N * sum_e f_e P_e  with
 * respect to x and every parameter, through the forward above.  The balance
 * loss reaches the router through P only: f comes from a hard choice and is
 * a constant ("Mixture of Experts and Guided Decoding", routing-collapse
 * passage after the auxiliary-loss equation).  The selection (top-k on the
 * keys) and the capacity mask are held fixed; select_bias gets no gradient.
 *
 *   kept slot j of token t:  d(expert input) = g_tj dy_t,
 *                            dg_tj = <dy_t, E_e(x_t)>
 *   gates (kept softmax):    dr_t[idx_tj] += g_tj (dg_tj - sum_l g_tl dg_tl)
 *   balance loss:            dr_t[e] += p_te (c_e - sum_j c_j p_tj),
 *                            c_e = aux_grad alpha N f_e / T, p_t = softmax(r_t)
 *   router:                  dW_r = dr^T x, dx += dr W_r,
 *                            d logit_bias = sum_t dr_t
 * plus the chain rule through every SwiGLU expert for dx, dW_gate, dW_up and
 * dW_down (shared experts with gate 1).
 *
 * The call recomputes the routing and the gate/up projections from x (it
 * takes no state from a forward call).  Arithmetic: bf16 operands on the
 * matrix cores with fp32 accumulation; the intermediate per-row tensors (gate
 * and up projections, dy W_down, the SwiGLU gradients, each row's dx
 * contribution) are held in dtype; the router gradient and every reduction
 * are fp32; each output is rounded once to its type.  Deterministic.
 * Expert weights must be in dtype (MOE_WEIGHTS_DTYPE): FP8 codes have no
 * gradient, so MOE_ERR_UNSUPPORTED.  T = 0 writes zero weight gradients. */
typedef struct {
  void* dx;           /* [T, d]     dtype, required when T > 0                  */
  void* dw_router;    /* [N, d]     dtype, required                             */
  float* dlogit_bias; /* [N]        fp32, or NULL                               */
  void* dw_gate;      /* [N, F, d]  dtype, required (experts no token chose: 0) */
  void* dw_up;        /* [N, F, d]  dtype, required                             */
  void* dw_down;      /* [N, d, F]  dtype, required                             */
  void* dws_gate;     /* [S, F, d]  dtype, required when S > 0                  */
  void* dws_up;       /* [S, F, d]                                              */
  void* dws_down;     /* [S, d, F]                                              */
} moe_grads;

/* Bytes of device workspace moe_layer_backward needs for `cfg` (a multiple
 * of 256): per-row activations and their K-major segments, plus transposed
 * copies of the expert weights for fp32 layers (bf16 layers whose d_model is
 * a multiple of 128 read the weights as K-rows and hold no copies).  0 for an
 * invalid cfg. */
size_t moe_backward_workspace_size(const moe_config* cfg);

/* Layer backward: x [T, d] and weights as for moe_layer_forward, dy [T, d]
 * the gradient of L with respect to y (dtype), alpha the balance-loss
 * coefficient and aux_grad the weight of that loss in L.  Writes every
 * gradient of `grads` (caller-owned device arrays, 16-byte aligned).
 * `workspace` holds moe_backward_workspace_size(cfg) bytes, 256-byte
 * aligned; its contents are scratch. */
moe_status moe_layer_backward(const moe_config* cfg, const void* x,
                              const moe_weights* w, const void* dy, float alpha,
                              float aux_grad, moe_grads* grads, void* workspace,
                              size_t ws_bytes, void* stream);

/* Stage markers for moe_layer_backward_timed. */
enum {
  MOE_BSTAGE_ROUTE = 0,       /* routing and grouping, recomputed               */
  MOE_BSTAGE_TRANSPOSE_W = 1, /* W_r transposed; W_down, [W_gate | W_up] only where not
                                 read as K-rows (fp32 layers)                       */
  MOE_BSTAGE_RECOMPUTE = 2,   /* gate and up projections of the rows (2 GEMMs)   */
  MOE_BSTAGE_GRAD_H = 3,      /* dy W_down (GEMM), then the SwiGLU backward      */
  MOE_BSTAGE_GRAD_X = 4,      /* [dA dB] [W_gate; W_up] (GEMM), router, dx       */
  MOE_BSTAGE_SEGMENTS = 5,    /* per-expert operands of the weight gradients     */
  MOE_BSTAGE_GRAD_W = 6,      /* dW_down, dW_gate, dW_up (3 grouped GEMMs)       */
  MOE_BSTAGE_GRAD_WR = 7,     /* dW_r                                            */
  MOE_BSTAGE_COUNT = 8
};

/* moe_layer_backward that also records stage_events[i] (hipEvent_t, created
 * by the caller) on `stream` before stage i and stage_events[MOE_BSTAGE_COUNT]
 * after the last; NULL array or NULL entries are skipped, as for
 * moe_layer_forward_timed.  With T = 0 no marker is recorded. */
moe_status moe_layer_backward_timed(const moe_config* cfg, const void* x,
                                    const moe_weights* w, const void* dy,
                                    float alpha, float aux_grad, moe_grads* grads,
                                    void* workspace, size_t ws_bytes, void* stream,
                                    void* const* stage_events);

/* Auxiliary-loss-free balancing ("MoE inference: the call centre with 256
 * specialists ...", "The bare mechanism": a routing bias adjusted during
 * training keeps the experts balanced without a loss term).  The pages give
 * no rule; this library's reading is one step toward the mean load:
 *   select_bias[e] += rate * sign(mean_j counts[j] - counts[e])
 * (fp32 addition; the sign is taken exactly on the integer counts), counts
 * being the (token, slot) assignments per routed expert of a batch
 * (moe_routing.counts).  N <= 512; device arrays; enqueued on `stream`. */
moe_status moe_update_select_bias(int32_t N, const int32_t* counts, float rate,
                                  float* select_bias, void* stream);

/* ------------------------------------------------ experts of one's own
 *
 * The parts of the layer as calls of their own, for experts other than the
 * layer's (another activation, biases, a residual, activations kept between
 * forward and backward):
 *
 *   moe_route            x -> topk_idx, topk_gate
 *   moe_group_rows       topk_idx -> offsets, row_token, slot_row
 *   moe_grouped_linear   rows by expert, any number of times
 *   moe_combine          rows -> tokens
 *
 * and backwards moe_combine_backward, moe_grouped_linear_backward, and
 * moe_combine without gates for the rows read through row_token.  The
 * conventions at the top of this file hold; the calls are deterministic.
 *
 * Grouping.  topk_idx [T, k] (moe_route's, or any int32 indices) to
 *   offsets   [N + 1]  expert e owns rows offsets[e] .. offsets[e + 1] - 1
 *   row_token [T k]    token of every row (entries at or past offsets[N]
 *                      are left as they were)
 *   slot_row  [T, k]   row of every (token, slot), -1 for one without a row
 * The rows of an expert are in the flat order of their (token, slot) pairs.
 * capacity: 0, or the most pairs an expert keeps, its first ones (as in
 * moe_config).  A pair whose index lies outside [0, N) gets no row: -1 marks
 * the slots of padding.  No output may overlap topk_idx.  1 <= N <= 512,
 * k <= 16, T k < 2^30; T = 0 writes offsets only.  workspace:
 * moe_group_workspace_size(T, N, k) bytes, 256-byte aligned (the size is 0 for
 * sizes outside these). */
size_t moe_group_workspace_size(int32_t T, int32_t N, int32_t k);
moe_status moe_group_rows(int32_t T, int32_t N, int32_t k, int32_t capacity,
                          const int32_t* topk_idx, int32_t* offsets, int32_t* row_token,
                          int32_t* slot_row, void* workspace, size_t ws_bytes, void* stream);

/* Activations of moe_grouped_linear.  GELU is z Phi(z) with the normal
 * distribution's CDF; SWIGLU is SiLU(z[:out]) * z[out:], the weights of a
 * group being the gate's rows and then the up projection's. */
typedef enum {
  MOE_ACT_NONE = 0,
  MOE_ACT_RELU = 1,
  MOE_ACT_GELU = 2,
  MOE_ACT_SILU = 3,
  MOE_ACT_SWIGLU = 4
} moe_activation;

/* A linear map for each of `groups` groups of rows.  z_dim = out_dim, or
 * 2 out_dim with MOE_ACT_SWIGLU, is the number of rows of a group's weights.
 * One group is an ordinary dense product.  groups <= 512, in_dim and out_dim
 * multiples of 64 up to 2^20, rows < 2^27, x_rows < 2^30, and
 *   (rows / 128 + groups) max(in_dim, z_dim) / 64 <= 2^23   (rows / 128 rounded down)
 *   groups z_dim in_dim <= 2^39, in a backward that writes dw < 2^36;
 * MOE_WEIGHTS_FP8_E4M3 needs MOE_BF16.  Other sizes are MOE_ERR_UNSUPPORTED. */
typedef struct {
  int32_t rows;          /* rows of y (and of residual, dy, dx, the checkpoint)       */
  int32_t x_rows;        /* rows of x when row_index is given; 0: x has `rows` rows   */
  int32_t groups;
  int32_t in_dim;
  int32_t out_dim;
  int32_t dtype;         /* a moe_dtype                                               */
  int32_t weight_format; /* a moe_weight_format                                       */
  int32_t activation;    /* a moe_activation                                          */
} moe_linear_config;

/* z[r] = x[src(r)] W_e^T + bias[e],  y[r] = act(z[r]) + residual[r]
 * for the rows r of every group e, src(r) = row_index[r] (clamped to x's
 * rows) or r.  Rows of no group (before offsets[0], at or past offsets[groups])
 * are left as they were.
 *
 * offsets is read on the device and has to rise (or stay) from 0 or more to
 * rows or less.  Other values are clamped where they are used: no access goes
 * out of bounds, but the results may be anything.  y may be residual; no output
 * may overlap another input.  With z_codes and z_scale the call also writes the
 * 8-bit checkpoint of z (below), which the backward of an activation reads.  z
 * is held in fp32 until it is rounded to y or coded. */
typedef struct {
  const void* x;            /* [x_rows or rows, in_dim]                               */
  const int32_t* row_index; /* [rows], or NULL when x_rows = 0                        */
  const int32_t* offsets;   /* [groups + 1]                                           */
  const void* w;            /* [groups, z_dim, in_dim]                                */
  const float* w_scale;     /* [groups, z_dim], FP8 weights only                      */
  const float* bias;        /* [groups, z_dim] or NULL                                */
  const void* residual;     /* [rows, out_dim] or NULL                                */
  void* y;                  /* [rows, out_dim]                                        */
  uint8_t* z_codes;         /* [rows, z_dim] or NULL                                  */
  float* z_scale;           /* [rows, z_dim / 64], with z_codes                       */
} moe_linear_args;

/* Bytes of device workspace moe_grouped_linear needs (a multiple of 256);
 * 0 for an invalid or unsupported cfg. */
size_t moe_linear_workspace_size(const moe_linear_config* cfg);
moe_status moe_grouped_linear(const moe_linear_config* cfg, const moe_linear_args* a,
                              void* workspace, size_t ws_bytes, void* stream);

/* Gradients of L with respect to x, W and bias, given dy = dL/dy:
 *   dz[r]    = dy[r] act'(z[r])       z decoded from its 8-bit checkpoint
 *   dx[r]    = dz[r] W_e              one row for every row of y: rows read
 *                                     through row_index are summed over a
 *                                     token's slots by moe_combine
 *   dw[e]    = sum_r dz[r]^T x[src(r)],  dbias[e] = sum_r dz[r]
 * (the residual's gradient is dy).  No output may overlap an input.  Each is
 * optional, one at least is required; groups without rows get zeros; rows of
 * dx of no group are left as they were.  dz is held in dtype as operand of
 * both products, dbias sums it before that rounding.  Weights in dtype only
 * (MOE_WEIGHTS_DTYPE). */
typedef struct {
  const void* x;            /* as in the forward (NULL when dw is)                    */
  const int32_t* row_index;
  const int32_t* offsets;
  const void* w;            /* (NULL when dx is)                                      */
  const void* dy;           /* [rows, out_dim]                                        */
  const uint8_t* z_codes;   /* required unless MOE_ACT_NONE                           */
  const float* z_scale;
  void* dx;                 /* [rows, in_dim] or NULL                                 */
  void* dw;                 /* [groups, z_dim, in_dim] or NULL                        */
  float* dbias;             /* [groups, z_dim] or NULL                                */
} moe_linear_grad_args;

size_t moe_linear_backward_workspace_size(const moe_linear_config* cfg);
moe_status moe_grouped_linear_backward(const moe_linear_config* cfg,
                                       const moe_linear_grad_args* a, void* workspace,
                                       size_t ws_bytes, void* stream);

/* 8-bit activation checkpoints.  x [rows, cols] (dtype a moe_dtype, cols a
 * multiple of 64, rows cols <= 2^35) is held as one OCP E4M3 code for each
 * element and one fp32 scale for each block of 64 columns of a row:
 *   m = max(max |x| over the block, 1e-30),  scale = m / 448,
 *   code = E4M3(x * (448 / m)), to nearest even;  unpack: code * scale,
 * so an element is off by at most 2^-4 of itself, or scale 2^-10 where that
 * is more: one of at most scale 2^-10 becomes 0, where ReLU's slope is 0.  NaN
 * and infinities become the NaN code and do not enter m.  codes [rows, cols],
 * scale [rows, cols / 64].  rows = 0 launches nothing.  No output may overlap
 * an input. */
moe_status moe_checkpoint_pack(int64_t rows, int32_t cols, int32_t dtype, const void* x,
                               uint8_t* codes, float* scale, void* stream);
moe_status moe_checkpoint_unpack(int64_t rows, int32_t cols, int32_t dtype,
                                 const uint8_t* codes, const float* scale, void* x,
                                 void* stream);

/* y[t] = sum_s gate[t, s] rows[slot_row[t, s]] over the slots that have a row
 * (gate NULL: 1), summed in fp32 in slot order.  rows [n_rows, d], slot_row
 * and gate [T, k], y [T, d]; a slot_row outside [0, n_rows) is a slot without
 * a row.  d a multiple of 64, k <= 16, T < 2^23.  y must not overlap rows. */
moe_status moe_combine(int32_t T, int32_t k, int32_t n_rows, int32_t d, int32_t dtype,
                       const void* rows, const int32_t* slot_row, const float* gate, void* y,
                       void* stream);
/* drows[slot_row[t, s]] = gate[t, s] dy[t],  dgate[t, s] = <dy[t], rows[...]>
 * (0 for a slot without a row).  drows and dgate are optional, one at least
 * is required; rows may be NULL when dgate is.  Rows that no slot names are
 * left as they were; no row may be named twice, and no output may overlap an
 * input. */
moe_status moe_combine_backward(int32_t T, int32_t k, int32_t n_rows, int32_t d, int32_t dtype,
                                const void* rows, const int32_t* slot_row, const float* gate,
                                const void* dy, void* drows, float* dgate, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_H_ */
