/*
 * moe_ffn.h -- C ABI of the fused mixture-of-experts FFN layer for GB300
 * (sm_103a), one GPU.
 *
 * The layer is the one named in "ggml-cuda: overlap the MoE shared expert on
 * a separate stream" (ROCm/llama.cpp PR #36, "What this changes"): a router,
 * top-k routed SwiGLU experts and a gated shared expert forked from the same
 * FFN input and joined by add(ffn_moe_out, ffn_shexp), in the small-batch
 * (decode) mat-vec regime.  Here the two branches are one fused operator;
 * nothing is overlapped across CUDA streams.
 *
 * Per token t (x_t is one row of x):
 *   logit[e] = sum_h router_w[e,h] x_t[h]                        (fp32)
 *   ids      = the top_k largest logits, larger first, equal logits ordered
 *              by the lower expert index
 *   p_j      = exp(logit[ids_j] - logit[ids_0]) / sum_i exp(logit[ids_i] - logit[ids_0])
 *              (softmax over all experts followed by renormalisation of the
 *              kept top_k: the same numbers)
 *   s        = sigmoid(sum_h shexp_gate_w[h] x_t[h])
 *   FFN(x)   = down( silu(gate x) * (up x) ),  silu(z) = z / (1 + exp(-z))
 *   out_t    = sum_{j=0..top_k-1} p_j FFN_{ids_j}(x_t)  +  s FFN_shared(x_t)
 * The routed sum runs in rank order and the shared term is added last.  GPU
 * results are bitwise reproducible run to run (no floating-point atomics).
 *
 * The lifecycle follows the prepare / execute / destroy contract of the
 * "ggml operator extensions" page (stable-diffusion.cpp docs/ggml_extensions.md,
 * sections "Kernel selection" and "CUDA kernels can opt into device replay"):
 *   - prepare is host-only: it validates shapes, builds an immutable plan and
 *     reports the workspace size.  It launches nothing and allocates no
 *     device memory.
 *   - execute enqueues device work on the caller's stream only.  It makes no
 *     host decision based on tensor contents and never synchronises, so it
 *     can be captured in a CUDA graph and replayed.  Every counter and flag
 *     in the workspace is initialised by the recorded device work of each
 *     call; workspace contents are not preserved between calls.  An error is
 *     returned, never retried.
 *   - destroy frees the host plan only.
 *
 * Ownership: the caller owns every tensor and the workspace.  The library
 * keeps no pointer beyond a call.  One plan may be executed concurrently on
 * several streams when each call has its own workspace.
 *
 * All functions return MOE_FFN_OK (0) or a negative moe_ffn_status.
 */
#ifndef MOE_FFN_H
#define MOE_FFN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; 0 is the legacy default stream. */
typedef struct CUstream_st* moe_ffn_stream_t;
/* Same type as cudaEvent_t. */
typedef struct CUevent_st* moe_ffn_event_t;

typedef enum {
  MOE_FFN_OK = 0,
  MOE_FFN_ERR_INVALID_ARG = -1, /* null required pointer, null plan, bad enum */
  MOE_FFN_ERR_UNSUPPORTED = -2, /* shapes or dtype outside the supported set (see moe_ffn_prepare) */
  MOE_FFN_ERR_WORKSPACE = -3,   /* workspace_bytes smaller than prepare reported */
  MOE_FFN_ERR_MISALIGNED = -4,  /* a pointer is not 16-byte aligned (workspace: 256-byte) */
  MOE_FFN_ERR_CUDA = -5,        /* a CUDA runtime call or launch failed */
  MOE_FFN_ERR_TIMEOUT = -6,     /* device status only: a bounded in-kernel wait gave up */
  MOE_FFN_ERR_DEVICE = -7       /* the current device is not sm_103 (GB300) or lacks a needed feature */
} moe_ffn_status;

/* T tokens, hidden size H, E experts, top_k kept per token, expert
 * intermediate size I, shared-expert intermediate size Is. */
typedef struct {
  int32_t T, H, E, top_k, I, Is;
} moe_ffn_shapes;

/* MOE_FFN_ACT_F16: the operators around the layer only (not a plan's x). */
typedef enum { MOE_FFN_ACT_F32 = 0, MOE_FFN_ACT_BF16 = 1, MOE_FFN_ACT_F16 = 2 } moe_ffn_act_dtype;

/* Weight format of the routed experts and of the shared expert.  The router
 * and the shared-gate vector are bf16 in both formats. */
typedef enum {
  MOE_FFN_W_BF16 = 0,
  /* 4-bit blocks of 32 along each stored row (H elements for every matrix,
   * see expert_w): one fp16 scale d per block and 4-bit codes n in 0..15
   * with weight = d * (n - 8).
   * Row layout: C/2 bytes of codes (element 2j in the low nibble of byte j,
   * element 2j+1 in the high nibble), then C/32 little-endian fp16 scales;
   * 9*C/16 bytes per row of C elements. */
  MOE_FFN_W_Q4B32 = 1,
  /* int8 rows with one fp32 scale per stored row (the int8 linear,
   * sd.linear_i8.v1, of "ggml operator extensions", section "sd.cpp
   * integration"): weight = s * q, q in -127..127.  Row layout: C int8 codes, the
   * little-endian fp32 scale s, 12 zero bytes; C + 16 bytes per row of C
   * elements.  The activation is quantised per token to int8 in fp32
   * (x_scale = max|x| / 127, q = round-half-away(x / x_scale) clamped to
   * +-127; x_scale = 0 gives q = 0), the gate and up projections are exact
   * int32 dot products, g = float(int32_dot) * x_scale * s in fp32 in that
   * order (likewise u), then SwiGLU; the down projection takes the
   * dequantised rows s * q of the transposed down matrix.  Decode path only
   * (T <= 8), H a multiple of 16. */
  MOE_FFN_W_I8 = 2
} moe_ffn_weight_format;

typedef struct {
  int32_t act;  /* moe_ffn_act_dtype: dtype of x */
  int32_t wfmt; /* moe_ffn_weight_format */
} moe_ffn_dtype;

typedef struct moe_ffn_plan* moe_ffn_plan_t;

/*
 * Validate `shapes` and `dtype`, build a plan and report the workspace size.
 * Host only: no device call, no launch, no device allocation.
 * Supported:
 *   decode path, 1 <= T <= 8: 1 <= E <= 1024, 1 <= top_k <= min(E, 32),
 *     H <= 4096 and a multiple of 8 (bf16 weights), of 256 (4-bit
 *     weights) or of 16 (int8 weights), I, Is >= 1; x fp32 or bf16;
 *   batched path, 9 <= T <= 1024 (routing, expert-sorted gather, grouped
 *     GEMMs on the tcgen05 tensor cores, fixed-order combine): bf16 or 4-bit
 *     weights and bf16 x, E <= 256, top_k <= 32, H a multiple of 256, I and
 *     Is multiples of 128.  With 4-bit weights the GEMM operands are fp16:
 *     each weight is d (code - 8) rounded once to fp16, x and the SwiGLU
 *     output h are carried in fp16 (accumulation fp32), so x and h must lie
 *     within fp16's range (|v| < 65504); the decode path keeps the exact
 *     weights.
 * moe_ffn_query(MOE_FFN_QUERY_PATH) reports the path taken.
 * Returns MOE_FFN_ERR_UNSUPPORTED otherwise, MOE_FFN_ERR_INVALID_ARG for null
 * pointers.  On success *plan is owned by the caller (moe_ffn_destroy).
 */
int moe_ffn_prepare(const moe_ffn_shapes* shapes, moe_ffn_dtype dtype, moe_ffn_plan_t* plan,
                    size_t* workspace_bytes);

/*
 * Enqueue the layer on `stream` (the current device must be a GB300).
 * Device pointers, all caller-owned:
 *   workspace     >= workspace_bytes from prepare, 256-byte aligned, scratch
 *   x             [T,H] fp32 or bf16 (plan dtype), row-major
 *   router_w      bf16 [E,H]
 *   expert_w      E consecutive blocks, block e = gate[I,H] | up[I,H] | downT[I,H]
 *                 in the plan's weight format, each matrix row-major with
 *                 H-element rows: gate and up are [out,in]; downT is the down
 *                 projection stored transposed (row i holds the weights from
 *                 intermediate unit i to all H outputs)
 *                 A caller holding the usual down[H,I] matrix passes its
 *                 transpose; with 4-bit weights it quantises that transpose
 *                 row by row, so down's blocks of 32 run along H.
 *   shexp_w       gate[Is,H] | up[Is,H] | downT[Is,H]
 *   shexp_gate_w  bf16 [H]
 *   out           fp32 [T,H]; may alias x exactly (the layer reads all of x
 *                 before it writes out); any other overlap is undefined.
 * Every pointer must be 16-byte aligned.  Returns without synchronising.
 */
int moe_ffn_execute(moe_ffn_plan_t plan, moe_ffn_stream_t stream, void* workspace, size_t workspace_bytes,
                    const void* x, const void* router_w, const void* expert_w, const void* shexp_w,
                    const void* shexp_gate_w, float* out);

/*
 * moe_ffn_execute, and also write the routing: topk_ids int32 [T,top_k] and
 * topk_w fp32 [T,top_k] in rank order (either may be NULL).
 */
int moe_ffn_execute_ex(moe_ffn_plan_t plan, moe_ffn_stream_t stream, void* workspace, size_t workspace_bytes,
                       const void* x, const void* router_w, const void* expert_w, const void* shexp_w,
                       const void* shexp_gate_w, float* out, int32_t* topk_ids, float* topk_w);

/*
 * Pre-norm transformer-block form (one layer of a decode stack):
 *   xn = bf16( x_res / sqrt(mean(x_res^2) + eps) )      (RMSNorm, weight 1)
 *   x_res <- x_res + layer(xn)
 * with the layer output and the residual add rounded to fp32 separately.
 * x_res is fp32 [T,H], read and updated in place.  The plan must have been
 * prepared with act = MOE_FFN_ACT_BF16 (the layer sees the bf16 xn) and
 * T <= 8.  topk_ids / topk_w as in moe_ffn_execute_ex (may be NULL).  Other
 * arguments as moe_ffn_execute; eps >= 0 or MOE_FFN_ERR_INVALID_ARG.
 */
int moe_ffn_execute_block(moe_ffn_plan_t plan, moe_ffn_stream_t stream, void* workspace, size_t workspace_bytes,
                          float* x_res, const void* router_w, const void* expert_w, const void* shexp_w,
                          const void* shexp_gate_w, float eps, int32_t* topk_ids, float* topk_w);

/*
 * Test/debug: synchronise `stream`, then copy the device status word of the
 * last execute that used `workspace` (MOE_FFN_OK or MOE_FFN_ERR_TIMEOUT) to
 * *device_status.  Returns a host-side status.
 */
int moe_ffn_read_status(moe_ffn_plan_t plan, const void* workspace, moe_ffn_stream_t stream,
                        int32_t* device_status);

/*
 * Test/debug: synchronise `stream`, then copy the token -> expert bucketing
 * of the last execute that used `workspace` to host arrays:
 *   counts [E]      tokens routed to each expert
 *   offsets [E+1]   exclusive prefix sum of counts
 *   perm [T*top_k]  flat (t*top_k + j) indices grouped by ascending expert,
 *                   token-major inside a group (a stable counting sort)
 *   active [E]      experts with counts > 0, ascending; *num_active of them
 */
int moe_ffn_read_routing(moe_ffn_plan_t plan, const void* workspace, moe_ffn_stream_t stream, int32_t* counts,
                         int32_t* offsets, int32_t* perm, int32_t* active, int32_t* num_active);

/*
 * Allocation-free variant of moe_ffn_execute, for callers that cannot
 * allocate device memory: for example a library embedded in a runtime that
 * has already handed all free device memory to its own pool (an inference
 * server that reserves the memory for its caches at start-up), or a plugin
 * given no allocator and no workspace.  This entry point has no counterpart
 * on the pages the layer is built from; it is an addition of this library.
 *
 * The scratch lives in one file-scope __device__ array of
 * MOE_FFN_STATIC_SCRATCH_BYTES bytes inside the library, which every GPU that
 * loads the library holds until the process exits.  The caller still passes
 * inputs and output exactly as for moe_ffn_execute.  Plans whose workspace is
 * larger than the array are rejected with MOE_FFN_ERR_WORKSPACE (the decode
 * shapes of one token batch, e.g. T <= 8, H = 2048, E = 128, top_k = 8,
 * I = 768, fit).  No cudaMalloc, cudaFree or other allocating call is made.
 *
 * The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current) and caches it; make that
 * first call before any stream capture.  Every call on a device shares the
 * one array and the kernels re-initialise what they read in each call, but
 * calls whose work overlaps on the GPU (other streams, or graphs replayed
 * concurrently) race on the array and give undefined results: serialise them.
 */
#define MOE_FFN_STATIC_SCRATCH_BYTES (1 << 24)
int moe_ffn_execute_static_scratch(moe_ffn_plan_t plan, moe_ffn_stream_t stream, const void* x, const void* router_w,
                                   const void* expert_w, const void* shexp_w, const void* shexp_gate_w, float* out);

/*
 * Test: the in-kernel failure path, without a fault.  Enqueues on `stream` one
 * small kernel that waits, with the bounded waits the layer's kernels use, on
 * a condition that nothing ever satisfies: which = 0 an mbarrier phase that
 * never completes (the wait of a shared-memory copy that never lands), which
 * = 1 a workspace flag that never receives the value waited for (the decode
 * kernel's grid-wide barriers), which = 2 a tagged workspace word that never
 * carries the tag waited for (the decode kernel's poll of the partial
 * outputs, T = 1).  The wait gives up after its iteration cap, records
 * MOE_FFN_ERR_TIMEOUT in the workspace status word (read it with
 * moe_ffn_read_status) and the kernel returns; the CUDA context stays usable
 * and the next execute on the workspace clears the word.  Returns a host-side
 * status (MOE_FFN_ERR_INVALID_ARG for a bad `which` or null pointers,
 * MOE_FFN_ERR_WORKSPACE if workspace_bytes is below the plan's size).
 */
int moe_ffn_probe_timeout(moe_ffn_plan_t plan, moe_ffn_stream_t stream, void* workspace, size_t workspace_bytes,
                          int32_t which);

/*
 * The layer in the form of "ggml-cuda: overlap the MoE shared expert on a
 * separate stream" (ROCm/llama.cpp PR #36, "What this changes"): the routed
 * branch (router, top-k, routed experts: ffn_moe_out) runs on `stream`, the
 * gated shared expert (ffn_shexp) on `aux_stream`, forked after everything
 * enqueued on `stream` before this call (fork_event recorded on `stream`,
 * waited by `aux_stream`) and joined back (join_event recorded on
 * `aux_stream`, waited by `stream`); then out = ffn_moe_out + ffn_shexp on
 * `stream`, the add of the page's diamond.  Decode plans (T <= 8) only, like
 * the page's batch gate; MOE_FFN_ERR_UNSUPPORTED otherwise.  The two
 * branches split the SMs in proportion to the bytes they stream.  When
 * aux_stream equals `stream` or an event is NULL, the same kernels run one
 * after the other on `stream` (the sequential form); both forms give
 * bit-identical results.  The fused moe_ffn_execute overlaps the shared
 * expert inside one kernel instead; its results agree with these within
 * the layer's tolerance (the sums are formed in another order).
 * Arguments as moe_ffn_execute, except that the workspace must hold
 * moe_ffn_query(MOE_FFN_QUERY_TWO_STREAM_WORKSPACE) bytes.  The events are
 * caller-owned (cudaEventCreateWithFlags with cudaEventDisableTiming is
 * enough); the call records and waits on them and keeps no reference.
 */
int moe_ffn_execute_two_stream(moe_ffn_plan_t plan, moe_ffn_stream_t stream, moe_ffn_stream_t aux_stream,
                               moe_ffn_event_t fork_event, moe_ffn_event_t join_event, void* workspace,
                               size_t workspace_bytes, const void* x, const void* router_w, const void* expert_w,
                               const void* shexp_w, const void* shexp_gate_w, float* out);

/*
 * moe_ffn_execute for a routing that the caller brings (another router's, or
 * moe_ffn_route's) instead of the layer's own:
 *   out_t = sum_{j=0..top_k-1} w[t,j] FFN_{ids[t,j]}(x_t)  +  s FFN_shared(x_t)
 *   ids  int32 [T,top_k]; an id outside 0..E-1 (-1 by convention) drops the
 *        choice, whatever its weight; an expert named twice by a token counts
 *        once with the sum of its weights
 *   w    fp32 [T,top_k], used as they stand
 * shexp_gate_w NULL: the shared expert is not gated (s = 1).  shexp_w NULL: no
 * shared term (shexp_gate_w is then ignored, and so is the plan's Is).  A token
 * whose choices are all dropped gets the shared term alone (0 without one).
 * Results are bitwise reproducible.  Other arguments, plans and paths as
 * moe_ffn_execute; ids and w 4-byte aligned.  out may alias x exactly.
 * moe_ffn_read_routing reports the buckets of the kept choices: offsets[E]
 * entries of perm.
 */
int moe_ffn_execute_routed(moe_ffn_plan_t plan, moe_ffn_stream_t stream, void* workspace, size_t workspace_bytes,
                           const void* x, const int32_t* ids, const float* w, const void* expert_w,
                           const void* shexp_w, const void* shexp_gate_w, float* out);

/* ---------------------------------------------------------------------------
 * Operators around the layer.  They need no plan: a call checks its argument
 * block on the host, enqueues on `stream` and returns without synchronising;
 * each can be captured in a CUDA graph, allocates nothing and is bitwise
 * reproducible.  Row strides are in elements and at least the row's width.
 * Tensors need the alignment of their element type only (16-byte aligned rows
 * are faster), unless stated.  T = 0 is a call that does nothing.
 */

/*
 * Routing: scores, selection and weights from router logits.
 *   l_te  logit (fp32, bf16 or fp16); -inf and NaN mask expert e for token t,
 *         +inf counts as the largest fp32 number
 *   s_te  = exp(l_te) / sum_i exp(l_ti)  (MOE_FFN_SCORE_SOFTMAX, over the
 *           experts that are not masked), or 1 / (1 + exp(-l_te))
 *           (MOE_FFN_SCORE_SIGMOID)
 *   c_te  = s_te + bias_e   (bias for balance, fp32; used for the choice alone.
 *           -inf and NaN mask the expert for every token, +inf counts as the
 *           largest fp32 number).  bias NULL: c_te = s_te
 *   groups: the experts form `groups` groups of E / groups neighbours; a group's
 *           value is its largest c (MOE_FFN_GROUP_MAX) or the sum of its two
 *           largest (MOE_FFN_GROUP_TOP2; of one, where only one is left); the
 *           top_groups groups of the largest values keep their experts, equal
 *           values going to the lower group
 *   ids   = the top_k largest c of the kept experts, larger first, equal c
 *           ordered by the larger logit, then by the lower expert index
 *   w_tj  = scale s_{t,ids_j}, divided by sum_i s_{t,ids_i} when renorm != 0
 * Where fewer than top_k experts are left the last ids are -1 and their
 * weights 0 (a wholly masked token: all of them); moe_ffn_execute_routed drops
 * such choices.  The choice is that of c to the resolution of fp64: scores
 * closer than fp32 can tell apart are compared in fp64.
 * 1 <= E <= 1024, 1 <= top_k <= min(E, 32), groups <= 32 and a divisor of E,
 * 1 <= top_groups <= groups, top_k <= top_groups E / groups.
 */
typedef enum { MOE_FFN_SCORE_SOFTMAX = 0, MOE_FFN_SCORE_SIGMOID = 1 } moe_ffn_score;
typedef enum { MOE_FFN_GROUP_MAX = 0, MOE_FFN_GROUP_TOP2 = 1 } moe_ffn_group_score;
typedef struct {
  int32_t T, E, top_k;
  int32_t score;               /* moe_ffn_score */
  int32_t groups, top_groups;  /* 1, 1: no groups */
  int32_t group_score;         /* moe_ffn_group_score */
  int32_t renorm;
  int32_t dtype;               /* moe_ffn_act_dtype of the logits */
  float scale;                 /* finite */
  int64_t row_stride;          /* of the logits */
} moe_ffn_route_args;
/* logits [T,E], bias [E] or NULL, ids int32 [T,top_k], w fp32 [T,top_k]. */
int moe_ffn_route(const moe_ffn_route_args* args, moe_ffn_stream_t stream, const void* logits, const float* bias,
                  int32_t* ids, float* w);

/*
 * The norms after one block and before the next, with the block's gate and
 * the residual scale between them.  Per token:
 *   z      = y rsqrt(mean(y^2) + eps) (w_offset + w_post)  if post_norm, else y
 *   r'     = alpha r + beta a(gate) z        a(g) = g or 1 / (1 + exp(-g));
 *            gate NULL: a = 1.  y NULL: r' = alpha r
 *   normed = r' rsqrt(mean(r'^2) + eps) (w_offset + w_pre)
 * All in fp32; r' enters the second norm unrounded; res_out and normed are
 * rounded once.  w_post, w_pre fp32 or bf16 [H] (NULL: w_offset + w = 1).
 * gate: [H] (MOE_FFN_GATE_CHANNEL), [T] (MOE_FFN_GATE_TOKEN, gate_stride apart)
 * or [T,H] (MOE_FFN_GATE_FULL).  res_out may be res (same dtype and stride),
 * normed may be y (same); either may be NULL, not both.  Any other overlap is
 * undefined.  1 <= H <= 32768.
 */
typedef enum { MOE_FFN_GATE_CHANNEL = 0, MOE_FFN_GATE_TOKEN = 1, MOE_FFN_GATE_FULL = 2 } moe_ffn_gate_layout;
typedef struct {
  int32_t T, H;
  int32_t y_dtype, res_dtype, normed_dtype, gate_dtype;  /* moe_ffn_act_dtype; res_dtype: res and res_out */
  int32_t w_post_dtype, w_pre_dtype;                     /* MOE_FFN_ACT_F32 or MOE_FFN_ACT_BF16 */
  int32_t post_norm;
  int32_t gate_layout;   /* moe_ffn_gate_layout */
  int32_t gate_sigmoid;  /* a(g): 0 linear, 1 sigmoid */
  float alpha, beta, w_offset, eps;  /* finite, eps >= 0 */
  int64_t y_stride, res_stride, res_out_stride, normed_stride, gate_stride;
} moe_ffn_norm_args;
int moe_ffn_norm_residual(const moe_ffn_norm_args* args, moe_ffn_stream_t stream, const void* res, const void* y,
                          const void* w_post, const void* gate, const void* w_pre, void* res_out, void* normed);

/*
 * Low-rank adapters of many requests beside a projection (or the layer) that
 * they share.  Per token t with adapter a = adapter_ids[t]:
 *   out_t = y_t + scales_a B_a (A_a x_t)
 * A [n_adapters,R,K] and B [n_adapters,N,R] bf16 or fp16 as x, contiguous and
 * 16-byte aligned; x [T,K] 16-byte aligned, its stride a multiple of 8; y and
 * out [T,N] of one dtype.  out may be y (same stride).
 * adapter_ids int32 [T]; outside 0..n_adapters-1 (-1 by convention): out_t =
 * y_t.  ranks int32 [n_adapters] or NULL (all R): only the first ranks_a rows
 * of A_a and columns of B_a count (clamped to 0..R; what the others hold does
 * not matter).  scales fp32 [n_adapters] or NULL (1).
 * Sums are in fp32.  A_a x_t enters the second product as the sum of numbers of
 * x's type: 22 bits of each element and more where y is fp32, else 16 bits and
 * more (fp16: of elements from 2^-28 of the token's largest on; smaller ones are
 * off by at most 2^-50 of it).
 * T <= 16777216, 1 <= R <= 128, 8 <= K <= 65536 a multiple of 8, 1 <= N <=
 * 1048576.
 * The workspace (256-byte aligned, scratch) holds what
 * moe_ffn_adapters_workspace reports for the argument block.
 */
typedef struct {
  int32_t T, K, N, R, n_adapters;
  int32_t x_dtype;  /* MOE_FFN_ACT_BF16 or MOE_FFN_ACT_F16: x, A and B */
  int32_t y_dtype;  /* moe_ffn_act_dtype: y and out */
  int64_t x_stride, y_stride, out_stride;
} moe_ffn_adapters_args;
int moe_ffn_adapters_workspace(const moe_ffn_adapters_args* args, size_t* bytes);
int moe_ffn_add_adapters(const moe_ffn_adapters_args* args, moe_ffn_stream_t stream, void* workspace,
                         size_t workspace_bytes, const void* x, const int32_t* adapter_ids, const void* A,
                         const void* B, const int32_t* ranks, const float* scales, const void* y, void* out);

/* ---------------------------------------------------------------------------
 * The attention half of a block, as calls of their own like those above:
 * products with 4-bit weights, the append of keys and values to a paged cache
 * and attention over that cache, for decode steps with drafted tokens.
 */

/*
 * Product of few tokens with 4-bit weights:
 *   y_tn = sum_k W_nk x_tk + bias_n,    W_nk = d_n,g(k) (c_nk - 8)
 * Rows of W are those of MOE_FFN_W_Q4B32 with groups of `group` weights: K/2
 * bytes of codes (element 2j in the low nibble of byte j), then K/group fp16
 * scales; with group = 32 any stored matrix of the layer's 4-bit format is
 * such a W.  Rows are w_stride bytes apart.
 * x [T,K] bf16 or fp16, y [T,N] of any type, bias fp32 [N] or NULL.  Codes and
 * x enter the products exactly; sums, scales and bias are in fp32, y is rounded
 * once.  y overlaps no other tensor.
 * x 16-byte aligned, its stride a multiple of 8; w 16-byte aligned, w_stride a
 * multiple of 16 below 2^40.  T <= 1024, group 32, 64 or 128, K <= 65536 a multiple of
 * group, 1 <= N <= 16777216.
 */
typedef struct {
  int32_t T, K, N, group;
  int32_t x_dtype;  /* MOE_FFN_ACT_BF16 or MOE_FFN_ACT_F16 */
  int32_t y_dtype;  /* moe_ffn_act_dtype */
  int64_t x_stride, y_stride;
  int64_t w_stride; /* bytes */
} moe_ffn_project_args;
int moe_ffn_project(const moe_ffn_project_args* args, moe_ffn_stream_t stream, const void* x, const void* w,
                    const float* bias, void* y);

/*
 * Keys and values of new tokens into a paged cache, rotated by their position
 * on the way; the tokens' queries, rotated, beside them.  Per token t and head,
 * with the angle th_i = positions_t inv_freq_i of pair i < rot / 2:
 *   a' = scale (a cos th_i - b sin th_i),  b' = scale (a sin th_i + b cos th_i)
 * (a, b) = elements (i, i + rot/2) of the head, or (2i, 2i + 1) if interleaved.
 * Elements from rot on, and values, are taken as they are.  In fp32, rounded
 * once; the angle is reduced exactly (positions over all of int32, inv_freq
 * fp32 with |inv_freq| < 256; others give NaN).
 * k, v [T,kv_heads,D] and q [T,q_heads,D] of x_dtype, q NULL: none.
 * Caches: element (page, slot, head, d) of k at k_cache + page kc_page_stride +
 * slot kc_slot_stride + head kc_head_stride + d, page < pages, slot <
 * page_size; v likewise.
 * slots int32 [T]: the token goes to page slots_t / page_size, slot slots_t %
 * page_size.  A token whose slot is outside 0..pages page_size - 1 (-1 by
 * convention) is padding: nothing is written for it, q_out neither.  Tokens of
 * one call have different slots (where two have the same, either's elements may
 * remain).
 * q_out may be q (same dtype and strides); nothing else overlaps.
 * T <= 16777216, 1 <= D <= 512, rot even, 0 <= rot <= D, at most 4096 heads each, pages
 * page_size < 2^31.  Head strides are at least D.
 */
typedef struct {
  int32_t T, q_heads, kv_heads, D, rot;
  int32_t interleaved;
  int32_t x_dtype, q_out_dtype, cache_dtype;  /* moe_ffn_act_dtype */
  int32_t page_size, pages;
  float scale;                                /* finite */
  int64_t q_stride, q_head_stride, k_stride, k_head_stride, v_stride, v_head_stride;
  int64_t q_out_stride, q_out_head_stride;
  int64_t kc_page_stride, kc_slot_stride, kc_head_stride, vc_page_stride, vc_slot_stride, vc_head_stride;
} moe_ffn_append_args;
int moe_ffn_append_kv(const moe_ffn_append_args* args, moe_ffn_stream_t stream, const void* q, const void* k,
                      const void* v, const int32_t* positions, const int32_t* slots, const float* inv_freq,
                      void* q_out, void* k_cache, void* v_cache);

/*
 * Attention of B sequences' newest tokens over the paged cache that holds them:
 * one token each, a tree of drafted tokens, or the end of a prompt.
 * Sequence b has the rows t = q_start_b .. q_start_{b+1} - 1 of q, n of them;
 * its cache holds lens_b tokens, the last n of which are these rows' own (row
 * q_start_b + j is cached token lens_b - n + j).  Cached token i lies in page
 * page_table[b][i / page_size], slot i % page_size.
 *   s_ti   = scale q_t k_i;  softcap > 0: softcap tanh(s_ti / softcap)
 *   out_t  = sum_i exp(s_ti) v_i / sum_i exp(s_ti),   lse_t = log sum_i exp(s_ti)
 * over the tokens i that row t sees: all before the sequence's own n, and of
 * those the j-th where bit j % 32 of mask[t][j / 32] is set; mask NULL: those up
 * to the row's own.  Query head h reads key head h / (q_heads / kv_heads).
 * A row that sees nothing, or only scores of -inf, gets out = 0 and lse = -inf.
 * What a row does not see has no effect on it, infinities and NaN included.  A value
 * that it sees counts however small its weight: an infinity makes that element of out
 * the same infinity, NaN or infinities of both signs make it NaN.  Tokens of pages
 * outside 0..pages - 1 are not seen.  lens is taken within 0..max_pages page_size,
 * q_start within 0..T; rows of no sequence (padding behind the last) are left as
 * they are, those of several get any of the results.  out and lse overlap no other
 * tensor.
 * q [T,q_heads,D] and the caches are bf16 or fp16 (dtype), out any type, lse
 * fp32 [T,q_heads] or NULL.  Scores, statistics and sums are in fp32; weights
 * enter the second product as the sum of two numbers of the cache's type (bf16
 * with fp32 out: three).  Weights are held up to 2^8 (fp16: 2^15) before they are
 * divided by their sum: bf16 values from 2^119 / lens on may overflow.  Caches as in
 * moe_ffn_append_kv, 16-byte aligned with strides that are multiples of 8.
 * T <= 1048576, B <= 65536, q_heads a multiple of kv_heads and at most 128 kv_heads, kv_heads <= 4096,
 * D a multiple of 8 up to 256, pages page_size < 2^31, max_pages page_size <= 2^30.
 * The workspace (256-byte aligned, scratch) holds what
 * moe_ffn_attend_workspace reports for these heads and for T and B or any larger
 * ones; calls that overlap on the GPU need one each.
 */
typedef struct {
  int32_t T, B, q_heads, kv_heads, D;
  int32_t dtype;      /* MOE_FFN_ACT_BF16 or MOE_FFN_ACT_F16: q and the caches */
  int32_t out_dtype;  /* moe_ffn_act_dtype */
  int32_t page_size, pages, max_pages;
  int32_t mask_words; /* int32 words a row of the mask */
  float scale, softcap; /* finite, softcap >= 0 (0: no cap) */
  int64_t q_stride, q_head_stride, out_stride, out_head_stride;
  int64_t kc_page_stride, kc_slot_stride, kc_head_stride, vc_page_stride, vc_slot_stride, vc_head_stride;
  int64_t table_stride, mask_stride;
} moe_ffn_attend_args;
int moe_ffn_attend_workspace(const moe_ffn_attend_args* args, size_t* bytes);
int moe_ffn_attend(const moe_ffn_attend_args* args, moe_ffn_stream_t stream, void* workspace, size_t workspace_bytes,
                   const void* q, const void* k_cache, const void* v_cache, const int32_t* page_table,
                   const int32_t* lens, const int32_t* q_start, const int32_t* mask, void* out, float* lse);

/* Queries on a plan. */
typedef enum {
  MOE_FFN_QUERY_PATH = 0,                 /* 0 = decode, 1 = grouped GEMM */
  MOE_FFN_QUERY_LAUNCHES_PER_EXECUTE = 1, /* kernels one execute launches */
  MOE_FFN_QUERY_TWO_STREAM_WORKSPACE = 2  /* workspace bytes of moe_ffn_execute_two_stream (decode plans) */
} moe_ffn_query_t;
int moe_ffn_query(moe_ffn_plan_t plan, int32_t what, int64_t* value);

/* Free a plan (host memory only).  NULL is ignored. */
void moe_ffn_destroy(moe_ffn_plan_t plan);

/* Static text for a status code. */
const char* moe_ffn_strerror(int status);

/* Text of the CUDA runtime error behind the last MOE_FFN_ERR_CUDA returned to
 * the calling host thread ("" if none).  The pointer stays valid until that
 * thread's next call into the library. */
const char* moe_ffn_last_cuda_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FFN_H */
