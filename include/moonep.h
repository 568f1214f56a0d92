/*
 * moonep.h -- C ABI of the GB300 (sm_103a) balanced expert-parallel hot path.
 *
 * One process, one GPU.  The R expert-parallel ranks of the method are R
 * logical partitions of this device's HBM: rank j's dispatched rows are rows
 * [j*NvS, (j+1)*NvS) of one [R*NvS, H] buffer, so a "remote" write of the
 * method is an ordinary scatter inside one allocation.
 *
 * Sources (page title, section):
 *   [API]    "MoonEP Public API Visual Guide": Notation; Buffer(...);
 *            Buffer.dispatch(...); Buffer.prefetch_weight(...);
 *            Buffer.combine(...); Buffer.reduce_grad(...);
 *            Buffer.hidden_nvsh_buffer_view; Buffer.router_weight_buffer_view;
 *            Buffer.destroy(); MoonEPCommPlan and MoonEPCommPlan.clone().
 *   [README] "MoonshotAI/MoonEP" README: items 1-3; "Weight buffer";
 *            "How to set B".
 *   [vLLM]   "vllm ... prepare_finalize.moonep": prepare() and finalize().
 *
 * Conventions shared by every entry point
 *   - Arrays are dense, row-major, and live in device memory unless stated.
 *     bf16 tensors travel as uint16_t bit patterns.
 *   - Every device pointer must be 16-byte aligned; H % 8 == 0 and, for the
 *     weight entry points, HHp % 8 == 0 (16-byte rows).  moonep_prefetch_rows
 *     takes any alignment and row size (other than 16-byte multiples on a
 *     16-byte aligned base, rows move byte by byte).
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Every call
 *     is stream-ordered and asynchronous: nothing synchronises with the host
 *     except moonep_get_status, moonep_ctx_destroy and moonep_plan_destroy
 *     (fixed shapes need no per-layer host synchronisation [README item 3]).
 *   - Return value: MOONEP_OK (0) or a negative MOONEP_ERR_*.  Errors found on
 *     the host (bad argument, destroyed context, CUDA launch failure) return
 *     at once and launch nothing.  Errors found by a kernel (bad expert id,
 *     histogram mismatch, too many slots, corrupted plan) are latched in the
 *     context's device status word and read with moonep_get_status; outputs of
 *     the failing call and of calls that use its plan are then unspecified but
 *     every kernel stays inside the buffers it was given.
 *   - Outputs do not overlap inputs, except where a call says "in place".
 *   - The caller owns every tensor argument.  The library owns the context's
 *     scratch and status word, the plan's arrays and the optional zero-copy
 *     buffers behind moonep_hidden_view / moonep_weight_view.
 *   - One context plans one batch at a time: its planner scratch (counters,
 *     per-rank totals) is shared by its moonep_plan calls, and its router
 *     scratch by its moonep_route and moonep_route_select calls, so two plans,
 *     or two routes, must not
 *     overlap on the GPU (issue them on one stream, or order the streams); use
 *     one context per concurrent stream.  A plan and a route may overlap.  The
 *     other entry points keep no state between calls and may overlap freely.
 *   - Kernels are launched with programmatic dependent launch: each waits
 *     for the previous kernel on its stream before touching memory, so
 *     stream order is kept as with plain launches.
 */
#ifndef MOONEP_H
#define MOONEP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOONEP_OK 0
#define MOONEP_ERR_INVALID_ARG (-1)   /* bad argument or configuration (host) */
#define MOONEP_ERR_BAD_EXPERT (-2)    /* a top-k id outside [0, E) (device) */
#define MOONEP_ERR_HIST_MISMATCH (-3) /* tokens_per_expert != recount of topk (device) */
#define MOONEP_ERR_SLOTS (-4)         /* a rank needs more than B slots (device) */
#define MOONEP_ERR_CUDA (-5)          /* a CUDA call failed (host) */
#define MOONEP_ERR_DESTROYED (-6)     /* context already destroyed (host) */
#define MOONEP_ERR_PLAN (-7)          /* plan row outside [0, R*NvS) (device) */
#define MOONEP_ERR_NOMEM (-8)         /* device allocation failed (host) */
#define MOONEP_ERR_TIMEOUT (-9)       /* a planner block gave up waiting (device) */

/* Constructor controls [API, Buffer(...)]: E % R == 0; B prefetch slots per
 * rank (B = E/R is what training needs [README, How to set B]; smaller B is
 * allowed and reported as MOONEP_ERR_SLOTS when a plan needs more);
 * token_padding = row alignment of every non-empty segment; num_sms caps the
 * SMs that the copy kernels, the router and the expert stage use (<= 0: the
 * MOONEP_NUM_SMS environment variable when set to a positive count, else every
 * SM): a launch has no more blocks than that many SMs hold.  At the least, the
 * router, moonep_quantize_mx and moonep_gated_act launch one block per rank,
 * the router's sums one cluster of eight blocks and moonep_expert_product one
 * pair of SMs. */
typedef struct moonep_config {
  int R;             /* expert-parallel ranks (logical partitions), >= 1 */
  int E;             /* experts, multiple of R */
  int K;             /* routes per token, 1..32 */
  int S;             /* tokens per rank, >= 0 */
  int H;             /* hidden size, multiple of 8 */
  int B;             /* prefetch slots per rank, >= 0 */
  int token_padding; /* >= 1 */
  int num_sms;       /* <= 0: MOONEP_NUM_SMS, else all SMs */
} moonep_config;

typedef struct moonep_ctx moonep_ctx;

/* Plan flags */
#define MOONEP_PLAN_DUP_RECORDS 1 /* also build dup_groups / dup_loffs */

/* A communication plan [API, MoonEPCommPlan].  All pointers are device
 * arrays owned by the plan (moonep_plan_create / _clone / _destroy).
 *   dst[R, S*K]              encoded global row of every route i = s*K + k of
 *                            source rank r: g = j*NvS + w for the first route
 *                            of the token that lands on rank j, -(g+1) for a
 *                            later route of that token on the same rank
 *                            [API, Buffer.combine: positive/negative encoding]
 *   experts_to_copy[R, B]    expert held by each prefetch slot, -1 = unused
 *   cu_seqlens[R, E+B]       inclusive padded end offset of every segment,
 *                            rank-local rows, no leading 0 [API,
 *                            Buffer.dispatch; vLLM prepare: diff(cu_seqlens)]
 *   zero_fill_ranges[R,E+B,2] [start, end) padding rows of every segment
 *   remote_stats[R, 2]       {routes received from a remote home group,
 *                            prefetch slots used}
 *   dup_counts[R, 2]         {local duplicate routes, duplicate groups}
 *   dup_groups[R, NvS, 3]    (primary row, first index into dup_loffs, number
 *                            of duplicates), ascending primary row; valid
 *                            prefix dup_counts[j][1]; NULL unless the plan was
 *                            created with MOONEP_PLAN_DUP_RECORDS
 *   dup_loffs[R, NvS]        duplicate rows, grouped as dup_groups says; valid
 *                            prefix dup_counts[j][0]
 *   internal                 library-private tables (do not touch)
 * Segments of rank j: x = e for its home experts e in [j*E/R, (j+1)*E/R),
 * x = E + b for prefetch slot b; other segments are empty.  Rows
 * [cu_seqlens[j][E+B-1], NvS) of a rank (the tail) are never written. */
typedef struct moonep_comm_plan {
  int32_t *dst;
  int32_t *experts_to_copy;
  int32_t *cu_seqlens;
  int32_t *zero_fill_ranges;
  int32_t *remote_stats;
  int32_t *dup_counts;
  int32_t *dup_groups;
  int32_t *dup_loffs;
  int32_t *internal;
  int N;          /* routes per rank, S*K */
  int R, E, B, K, S;
  int NvS;        /* dispatched-row capacity per rank */
  int NvS_padded; /* row stride between ranks (== NvS) */
  int flags;
  size_t internal_bytes;
} moonep_comm_plan;

/* Sizes for a configuration: NvS = roundup(S*K + (E/R + B)*(tp-1), tp) and the
 * context's device scratch in bytes.  Any output pointer may be NULL. */
int moonep_query_sizes(const moonep_config *cfg, int *NvS, int *NvS_padded,
                       size_t *scratch_bytes);

/* Create a context on the current CUDA device [API, Buffer(...)]: validates
 * the configuration, allocates planner scratch and the status word, and, when
 * alloc_views != 0, the persistent [R*NvS, H] bf16 hidden buffer and [R*NvS]
 * fp32 weight buffer behind the zero-copy views.  *out is set on success. */
int moonep_ctx_create(const moonep_config *cfg, int alloc_views,
                      moonep_ctx **out);

/* Synchronise the device, free everything the context owns, mark it
 * destroyed [API, Buffer.destroy()].  Idempotent; NULL is accepted.  The
 * handle itself stays allocated so that later calls on it return
 * MOONEP_ERR_DESTROYED; moonep_ctx_free releases it. */
int moonep_ctx_destroy(moonep_ctx *ctx);
void moonep_ctx_free(moonep_ctx *ctx);
/* 1 once moonep_ctx_destroy has completed [API, Buffer.destroyed]. */
int moonep_ctx_destroyed(const moonep_ctx *ctx);

/* Allocate a plan's device arrays for the context's configuration.  flags:
 * MOONEP_PLAN_DUP_RECORDS. */
int moonep_plan_create(moonep_ctx *ctx, int flags, moonep_comm_plan *plan);
/* Free a plan's arrays (synchronises the device first); idempotent. */
int moonep_plan_destroy(moonep_comm_plan *plan);
/* Deep copy of every array and scalar [API, MoonEPCommPlan.clone()]: dst
 * must be a plan created for the same configuration and flags. */
int moonep_plan_clone(const moonep_comm_plan *src, moonep_comm_plan *dst, void *stream);

/* Online planner [API, Buffer.dispatch(...): the planning step that turns
 * every rank's S*K routes into the dst map; README items 1-2].
 *   topk  [R, S, K] int32 expert ids, each in [0, E)
 *   tpe   [R, E] int32 per-rank histogram, or NULL; when given it is checked
 *         against a recount of topk: a mismatch latches
 *         MOONEP_ERR_HIST_MISMATCH, and the plan is built from the recount
 * Fills every array of `plan`.  Deterministic: the same inputs give the same
 * plan, bit for bit.  Every rank receives exactly S*K routes; the experts a
 * rank prefetches come from one remote home group, at most B of them. */
int moonep_plan(moonep_ctx *ctx, const int32_t *topk, const int32_t *tpe,
                moonep_comm_plan *plan, void *stream);

/* Rank-local planner: the per-rank form of moonep_plan when each of the R
 * ranks is its own GPU [API, Buffer.dispatch(...): planning is collective,
 * every rank plans from the cross-rank statistics (MoonEPCommPlan
 * remote_stats); README, "How to set B"].  The one exchange step is an
 * all-gather of every rank's [E] tokens_per_expert into hist_all; each rank
 * then derives the same balance tables from hist_all and assigns only its own
 * routes, so no other routing data crosses between ranks.
 *   rank      source rank r of this call, 0 <= r < R
 *   topk_r    [S, K] int32 expert ids of rank r only
 *   hist_all  [R, E] int32 gathered per-rank histograms; row r is checked
 *             against a recount of topk_r (a mismatch latches
 *             MOONEP_ERR_HIST_MISMATCH; the tables stay those of hist_all,
 *             which every rank shares, and rank r's rows are unspecified)
 * Writes rank r's row of dst ([S*K] at plan->dst + r*S*K; other rows are not
 * touched), and experts_to_copy, cu_seqlens, zero_fill_ranges, remote_stats
 * and the plan's internal tables for every rank, equal to moonep_plan's.
 * dup_counts[j] is written with rank r's share: {duplicate routes of rank
 * r's tokens landing on rank j, their groups}; summed over the R calls (an
 * all-reduce across GPUs) it equals moonep_plan's.  The R calls together
 * give moonep_plan's plan, bit for bit.  Plans with MOONEP_PLAN_DUP_RECORDS,
 * and configurations whose planner tables do not fit in shared memory, are
 * refused (MOONEP_ERR_INVALID_ARG).  Rank-local calls of one context must
 * not overlap on the GPU (they share its scratch, as moonep_plan calls do). */
int moonep_plan_rank(moonep_ctx *ctx, int rank, const int32_t *topk_r,
                     const int32_t *hist_all, moonep_comm_plan *plan, void *stream);

/* Rank-local dispatch [API, Buffer.dispatch(...): tokens written straight
 * into the receiving ranks' buffers; README item 3]: rank r's tokens go to
 * their K destination rows in R rank windows, each its own allocation (on R
 * GPUs, peer pointers), and rank r zero-fills the padding rows of its own
 * window.  The R calls together give moonep_dispatch's rows.
 *   hidden_r   [S, H] bf16 rows of rank r
 *   w_r        [S, K] fp32 route weights of rank r, or NULL
 *   windows    HOST array of R device pointers: windows[j] = rank j's
 *              [NvS, H] bf16 rows (16-byte aligned)
 *   w_windows  HOST array of R device pointers to [NvS] fp32, or NULL
 *              (given exactly when w_r is)
 * Uses the plan's dst row r and its tables (moonep_plan or moonep_plan_rank). */
int moonep_dispatch_rank(moonep_ctx *ctx, const moonep_comm_plan *plan, int rank,
                         const uint16_t *hidden_r, const float *w_r,
                         uint16_t *const *windows, float *const *w_windows, void *stream);

/* Rank-local combine [API, Buffer.combine(...): the owner gathers its
 * tokens' K rows and reduces them; vLLM finalize(): an unweighted K-sum]:
 * out_r[s,:] = bf16_rne(fp32 sum over k = 0..K-1, in k order, of the row
 * |dst(r,s,k)| read from the rank window that holds it).
 *   y_windows  HOST array of R device pointers: rank j's [NvS, H] bf16 rows
 *   w_windows  HOST array of R device pointers to [NvS] fp32, or NULL
 *   out_r      [S, H] bf16 out
 *   w_out_r    [S, K] fp32 out (bit copies of the routes' weights), given
 *              exactly when w_windows is */
int moonep_combine_rank(moonep_ctx *ctx, const moonep_comm_plan *plan, int rank,
                        const uint16_t *const *y_windows, const float *const *w_windows,
                        uint16_t *out_r, float *w_out_r, void *stream);

/* Planner for callers that cannot allocate device memory.  The pages have no
 * counterpart: it exists for callers that must not call cudaMalloc, such as a
 * framework whose caching allocator owns (and accounts for) all device memory,
 * or a host path that cannot absorb cudaMalloc's implicit synchronisation.
 * It needs no context and no plan object and allocates nothing.
 *   cfg          as for moonep_ctx_create (H and num_sms are not used)
 *   topk, tpe    as for moonep_plan
 *   dst[R,S*K], experts_to_copy[R,B], cu_seqlens[R,E+B],
 *   zero_fill_ranges[R,E+B,2], remote_stats[R,2], dup_counts[R,2]
 *                caller-allocated device outputs, same contents as the
 *                fields of the same name that moonep_plan writes
 *   status       caller-allocated device int32: cleared by the call, then set
 *                to the first MOONEP_ERR_* a kernel meets (0 if none)
 * The planner's intermediate tables live in one file-scope device array of
 * 4 MiB (1 << 20 int32 words) that every GPU loading the library keeps until
 * the process exits; configurations whose tables do not fit (roughly
 * E*R*ceil(S*K/2048) + R*S*K + a few tables of E+B words) are rejected with
 * MOONEP_ERR_INVALID_ARG.  The first call on a device looks up that array's
 * device address, and the first call for each new (R, E, B) raises the
 * planner kernels' shared-memory limits, so make those calls before any
 * stream capture.  All calls share the array and a call overwrites what the last
 * one left there: calls that overlap on the GPU (on different streams, or
 * from several host threads without ordering) race and give wrong plans.
 * The plan it produces feeds no other entry point (they take a
 * moonep_comm_plan). */
int moonep_plan_noalloc(const moonep_config *cfg, const int32_t *topk,
                        const int32_t *tpe, int32_t *dst,
                        int32_t *experts_to_copy, int32_t *cu_seqlens,
                        int32_t *zero_fill_ranges, int32_t *remote_stats,
                        int32_t *dup_counts, int32_t *status, void *stream);

/* Fused-permute dispatch [API, Buffer.dispatch; README item 3].
 *   hidden      [R, S, H] bf16 source rows
 *   w_sk        [R, S, K] fp32 route weights, or NULL
 *   hidden_nvsh [R*NvS, H] bf16 out: row |dst| of every route = its token's
 *               row; padding rows zero; tail rows untouched
 *   w_nvs       [R*NvS] fp32 out, or NULL: route weight per row, 0 on padding
 *               (w_sk and w_nvs are both given or both NULL, else
 *               MOONEP_ERR_INVALID_ARG; an empty batch, R*S = 0, takes
 *               either without complaint)
 * Passing a saved plan again is the plan-reuse path (combine-backward
 * dispatch of an [R, S, H] gradient, weights NULL) [API, Buffer.dispatch:
 * a saved plan skips planning and ignores the routing inputs]. */
int moonep_dispatch(moonep_ctx *ctx, const moonep_comm_plan *plan,
                    const uint16_t *hidden, const float *w_sk,
                    uint16_t *hidden_nvsh, float *w_nvs, void *stream);

/* Combine [API, Buffer.combine; vLLM finalize: the K-sum is unweighted].
 *   y_nvsh   [R*NvS, H] bf16 expert outputs in dispatched order
 *   w_nvs    [R*NvS] fp32 or NULL
 *   out_sh   [R, S, H] bf16 out: out[r,s,:] = bf16_rne(fp32 sum over
 *            k = 0..K-1, in k order, of y[|dst(r,s,k)|,:])
 *   w_sk_out [R, S, K] fp32 out or NULL: w_nvs[|dst|] (bit copy); given
 *            together with w_nvs or not at all (any pair for an empty batch)
 * Reads only rows that dst names (never padding or tail rows). */
int moonep_combine(moonep_ctx *ctx, const moonep_comm_plan *plan,
                   const uint16_t *y_nvsh, const float *w_nvs,
                   uint16_t *out_sh, float *w_sk_out, void *stream);

/* Deduplicated dispatch [API, Buffer.dispatch: a token routed to several
 * experts on one rank is transferred once and expanded locally in an
 * epilogue].  Same arguments and results as moonep_dispatch, bit for bit,
 * in two launches: the copy writes the primary rows (dst >= 0) and every
 * route weight, then the expand epilogue copies each primary row to the
 * duplicate rows that plan->dup_groups / dup_loffs list for it.  Requires a
 * plan created with MOONEP_PLAN_DUP_RECORDS (else MOONEP_ERR_INVALID_ARG).
 * A record that points outside its rank sets MOONEP_ERR_PLAN in the status
 * word and is skipped. */
int moonep_dispatch_dedup(moonep_ctx *ctx, const moonep_comm_plan *plan,
                          const uint16_t *hidden, const float *w_sk,
                          uint16_t *hidden_nvsh, float *w_nvs, void *stream);

/* Deduplicated combine [API, Buffer.combine: duplicate rows are accumulated
 * into their primaries in fp32 before the gather].  Two launches:
 *   1. fold prologue, IN PLACE on y_nvsh: for every group of rank j,
 *      y[primary] = bf16_rne(fp32 y[primary] + y[dup_1] + ... ) in k order;
 *      the duplicate rows are left as they were;
 *   2. out[r,s,:] = bf16_rne(fp32 sum, in k order, over the token's primary
 *      routes only (dst >= 0; route 0 always is)); w_sk_out as moonep_combine.
 * The result can differ from moonep_combine by the fold's extra rounding
 * (at most 2^-7 * sum |y| per element).  Requires MOONEP_PLAN_DUP_RECORDS.
 * y_nvsh is written: a second call on the same buffer folds twice. */
int moonep_combine_dedup(moonep_ctx *ctx, const moonep_comm_plan *plan,
                         uint16_t *y_nvsh, const float *w_nvs,
                         uint16_t *out_sh, float *w_sk_out, void *stream);

/* Redundant-expert weight prefetch [API, Buffer.prefetch_weight; README,
 * Weight buffer].  W[p] (p < n_proj <= 4) is a device pointer to one
 * [E + R*B, HHp] bf16 tensor: rows [0, E) are the experts, rows E + j*B + b
 * are rank j's slots.  For every slot with experts_to_copy[j][b] = e >= 0:
 * row E + j*B + b = row e (bit copy).  Unused slots are not touched.
 * `W` itself is a host array of n_proj device pointers. */
int moonep_prefetch_weight(moonep_ctx *ctx, const moonep_comm_plan *plan,
                           int n_proj, uint16_t *const *W, int64_t HHp,
                           void *stream);

/* Weight prefetch of any row format [API, Buffer.prefetch_weight: packed
 * MXFP4 weights are uint8; optional block-scale tensors follow the same
 * leading E + B row convention and come as a complete gate/up/down set].
 * tensors[t] (t < n_tensors <= 8) is a device pointer to an [E + R*B] array
 * of rows of row_bytes[t] bytes each (packed MXFP4 [H, H'/2] bytes, E8M0
 * block scales [H, H'/32] bytes, bf16 [H, H'] as 2*H*H' bytes, ...).  For
 * every slot with experts_to_copy[j][b] = e >= 0 and every tensor: row
 * E + j*B + b = row e, byte for byte.  Unused slots are not touched.  A
 * tensor whose rows are 16-byte multiples on a 16-byte aligned base moves
 * 16-byte vectors, any other single bytes (correct, slower).  Pass the whole
 * set in one call: one launch covers every tensor.  `tensors` and
 * `row_bytes` are host arrays; a tensor with row_bytes 0 is skipped (its
 * pointer may be NULL). */
int moonep_prefetch_rows(moonep_ctx *ctx, const moonep_comm_plan *plan,
                         int n_tensors, void *const *tensors,
                         const int64_t *row_bytes, void *stream);

/* Decode-path preparation [vLLM, MoonEPPrepareAndFinalize: prepare() and
 * _pad_to_capacity]: the step's batch is padded to the context's static
 * capacity S, and invalid (negative) expert ids become expert 0 with zero
 * route weight (the planner has no sentinel for them), in place:
 *   num_tokens  HOST array [R]: valid tokens of each rank, 0 <= n <= S
 *               (NULL: S for every rank, only invalid ids are mapped)
 *   hidden      [R, S, H] bf16 or NULL, 16-byte aligned: rows s >= n of rank
 *               r are set to 0
 *   topk        [R, S, K] int32: ids < 0, and every id of rows s >= n, set
 *               to 0; ids >= E are left for the planner to report
 *   w_sk        [R, S, K] fp32 or NULL: the weights of those routes set to 0
 *   tokens_per_expert  [R, E] int32 out or NULL: per-rank counts of the
 *               prepared ids below E (the planner's tokens_per_expert)
 * Only padding rows and invalid routes are written. */
int moonep_prepare(moonep_ctx *ctx, const int32_t *num_tokens, uint16_t *hidden,
                   int32_t *topk, float *w_sk, int32_t *tokens_per_expert,
                   void *stream);

/* Gradient reduce of the redundant experts [API, Buffer.reduce_grad; README,
 * Weight buffer].  Gh[p] -> [E, HHp] fp32 home-expert gradients, Gs[p] ->
 * [R*B, HHp] fp32 slot gradients (the [R, B, H, H'] reduce buffer).  For
 * every expert e held by at least one slot:
 *   Gh[e] = Gh[e] + Gs[slot_1] + Gs[slot_2] + ...   (fp32, slots in
 *           ascending (rank, slot) order)
 * then every used slot is set to 0; unused slots are not touched.  `Gh` and
 * `Gs` are host arrays of n_proj (<= 4) device pointers. */
int moonep_reduce_redundant_grad(moonep_ctx *ctx, const moonep_comm_plan *plan,
                                 int n_proj, float *const *Gh,
                                 float *const *Gs, int64_t HHp, void *stream);

/* The router.  logits [R, S, E] (fp32, or bf16 when logits_bf16) -> for every
 * valid token (s < num_tokens[r]; num_tokens is a HOST array [R], NULL = S):
 *   scores  softmax: s_e = exp(z_e - max z), sigmoid: s_e = 1/(1+exp(-z_e));
 *           p_e = s_e / sum s
 *   topk [R, S, K]  the K largest logits, largest first, equal ones by lowest
 *           index (a NaN logit ranks first)
 *   w_sk [R, S, K]  p of the picks over their sum (0 when every score is 0;
 *           a score below 2^-126, a sigmoid of less than about -87, counts
 *           as 0)
 * Rows past num_tokens get id 0 and weight 0, as moonep_prepare leaves them.
 *   tokens_per_expert [R, E]  counts of the written ids (moonep_plan's)
 * and, when loss is given, the balance loss over the valid tokens' picks
 * c[r, e] and probability sums P[r, e]:
 *   MOONEP_SCOPE_RANK    a/R' sum_r sum_e (E c[r,e]/(K n_r)) (P[r,e]/n_r), R'
 *                        the ranks that hold a token
 *   MOONEP_SCOPE_GLOBAL  a sum_e (E c[e]/(K T)) (P[e]/T), summed over ranks
 *   loss [1] fp32, coef [R, E] fp32: the factor of P[r, e] in the loss, which
 *           moonep_route_backward reads (both given, or both NULL)
 * Needs K <= E.  Uses the context's router scratch: two moonep_route calls of
 * one context must not overlap.  Results do not depend on scheduling (sums in a
 * fixed order). */
#define MOONEP_SCORE_SOFTMAX 0
#define MOONEP_SCORE_SIGMOID 1
#define MOONEP_SCOPE_RANK 0
#define MOONEP_SCOPE_GLOBAL 1
int moonep_route(moonep_ctx *ctx, const void *logits, int logits_bf16,
                 int scoring, float balance, int scope,
                 const int32_t *num_tokens, int32_t *topk, float *w_sk,
                 int32_t *tokens_per_expert, float *coef, float *loss,
                 void *stream);

/* Gradient of the logits, in their type, from moonep_route's topk, w_sk and
 * coef (NULL: no balance loss), d_w_sk [R, S, K] fp32 (NULL: zero) and d_loss
 * [1] fp32 in device memory (NULL: 1).  The counts are constants of the loss.
 *   g_e = d_loss p_e (coef_e - sum_j p_j coef_j)
 *         + [e picked] w_e (d_w_e - sum_k w_k d_w_k)
 *   d_logits_e = g_e (softmax), g_e (1 - s_e) (sigmoid)
 * Rows past num_tokens get 0. */
int moonep_route_backward(moonep_ctx *ctx, const void *logits, int logits_bf16,
                          int scoring, const int32_t *num_tokens,
                          const int32_t *topk, const float *w_sk,
                          const float *d_w_sk, const float *coef,
                          const float *d_loss, void *d_logits, void *stream);

/* The router with a bias that balances the experts' loads, and with expert
 * groups.  Scores and shares as moonep_route's; a_e = p_e (softmax) or s_e
 * (sigmoid), and in place of the logits
 *   c_e = a_e + bias[e]
 * selects: the E/groups neighbouring experts of a group score the largest c
 * (MOONEP_GROUP_MAX) or the sum of the two largest (MOONEP_GROUP_TOP2; the one
 * of a group of one), and the picks are the K largest c within the top_groups
 * best groups; equal values by lowest index, a NaN first.  The order is that
 * of c in 64 bits; without a bias that of the logits, of experts and of groups by
 * their largest (sums of two are those of c).
 *   w_sk   scale a of the picks over their sum (renormalize; 0 when that is 0),
 *          or scale a; the bias weighs nothing
 * Everything else as moonep_route.  bias: [E] fp32 in device memory or NULL; -inf
 * shuts an expert out (a large finite one does too, at the cost of the fast way);
 * E % groups == 0, 1 <= top_groups <= groups, K <= top_groups * (E / groups). */
#define MOONEP_GROUP_MAX 0
#define MOONEP_GROUP_TOP2 1
typedef struct moonep_route_selection {
  const float *bias;
  int groups;      /* 1: no groups */
  int top_groups;
  int group_score;
  int renormalize;
  float scale;     /* finite, 0 or at least 2^-126 in size */
} moonep_route_selection;
int moonep_route_select(moonep_ctx *ctx, const void *logits, int logits_bf16,
                        int scoring, const moonep_route_selection *selection,
                        float balance, int scope, const int32_t *num_tokens,
                        int32_t *topk, float *w_sk, int32_t *tokens_per_expert,
                        float *coef, float *loss, void *stream);

/* moonep_route_backward for moonep_route_select's weights (selection's
 * renormalize and scale; picks, bias and groups have no gradient):
 *   g_e = d_loss p_e (coef_e - sum_j p_j coef_j) + [e picked] t_e - u p_e
 *   renormalize   t_e = w_e (d_w_e - sum_k w_k d_w_k / scale), u = 0
 *   otherwise     t_e = w_e d_w_e, u = sum_k w_k d_w_k (softmax) or 0 (sigmoid) */
int moonep_route_select_backward(moonep_ctx *ctx, const void *logits,
                                 int logits_bf16, int scoring,
                                 const moonep_route_selection *selection,
                                 const int32_t *num_tokens,
                                 const int32_t *topk, const float *w_sk,
                                 const float *d_w_sk, const float *coef,
                                 const float *d_loss, void *d_logits,
                                 void *stream);

/* One step of the bias, in place: bias[e] += rate sign(mean load - load_e), the
 * load of an expert its picks among the valid tokens of all ranks
 * (tokens_per_expert [R, E] as the router wrote it, num_tokens as given to it);
 * a load equal to the mean leaves the bias as it is.  Counts are compared as
 * whole numbers. */
int moonep_update_route_bias(moonep_ctx *ctx, const int32_t *tokens_per_expert,
                             const int32_t *num_tokens, float rate,
                             float *bias, void *stream);

/* Microscaled 4-bit quantisation (OCP MX v1.0, MXFP4) of x [rows, cols] (bf16,
 * or fp32 when x_fp32), cols % 32 == 0: every 32 values of a row share the
 * scale 2^(s - 127), s = floor(log2(largest magnitude)) - 2 + 127 (at least
 * 0), and become E2M1 codes, rounded to nearest even, saturating at 6.
 *   packed [rows, cols/2] uint8, value 2i in the low four bits of byte i
 *   scales [rows, cols/32] uint8 (E8M0)
 * A block with a NaN or an infinity gets scale 255 (NaN).  With cu_seqlens
 * (device [R, E+B]), rows must be R*NvS, and only rows that belong to a
 * segment are read and written. */
int moonep_quantize_mx(moonep_ctx *ctx, const void *x, int x_fp32, int64_t rows,
                       int64_t cols, const int32_t *cu_seqlens,
                       uint8_t *packed, uint8_t *scales, void *stream);

/* The values that codes and scales stand for, y [rows, cols] bf16 (fp32 when
 * y_fp32). */
int moonep_dequantize_mx(moonep_ctx *ctx, const uint8_t *packed,
                         const uint8_t *scales, int y_fp32, int64_t rows,
                         int64_t cols, void *y, void *stream);

/* The experts' product over the dispatched layout, both sides MXFP4:
 *   out[row, n] = sum_k A[row, k] W[g, n, k]
 * for every row of every segment, g the weight row of its segment (home
 * expert e: e; slot b of rank j: E + j*B + b, as moonep_prefetch_rows fills
 * them); fp32 accumulation, one rounding to bf16 (none when out_fp32).
 *   cu_seqlens   device [R, E+B]: the plan's; segments outside [0, NvS) are
 *                skipped and latch MOONEP_ERR_PLAN
 *   a            R*NvS rows of Kd/2 packed bytes, row_bytes apart (a multiple
 *                of 16, at least Kd/2), 16-byte aligned
 *   a_scales     R*NvS rows of Kd/32 bytes, scale_row_bytes apart
 *   w, w_scales  dense [E + R*B, N, Kd/2] (16-byte aligned), [E + R*B, N, Kd/32]
 *   out          [R*NvS, N], 16-byte aligned; other rows are not written
 *                (their codes may be read, as part of a tile, and never count)
 * N % 8 == 0, Kd % 32 == 0.  Runs on pairs of SMs: at least one pair, however
 * few SMs the context may use. */
int moonep_expert_product(moonep_ctx *ctx, const int32_t *cu_seqlens,
                          const uint8_t *a, int64_t row_bytes,
                          const uint8_t *a_scales, int64_t scale_row_bytes,
                          const uint8_t *w, const uint8_t *w_scales, int N,
                          int Kd, int out_fp32, void *out, void *stream);

/* The experts' weight gradients over the dispatched layout: for every segment,
 * with g its weight row,
 *   G[n, k] = sum over its rows of d[row, n] x[row, k]
 * x the rows that a product with weights [N, Kd] read, d the gradient of what it
 * gave.  bf16 in, fp32 sums.
 *   cu_seqlens   device [R, E+B]: the plan's; segments outside [0, NvS) are taken
 *                as empty and latch MOONEP_ERR_PLAN
 *   x, d         R*NvS rows of Kd and N bf16 values, x_row_bytes and d_row_bytes
 *                apart (multiples of 16), 16-byte aligned; rows outside every
 *                segment may be read and never count, whatever they hold
 *   grad         [E, N, Kd] fp32: home experts'; all written, zeros for one
 *                without rows
 *   slots        [R, B, N, Kd] fp32 (may be NULL when B = 0): the slots', those
 *                without rows are not touched (moonep_reduce_redundant_grad's Gs)
 *   workspace    moonep_expert_weight_grad_workspace(ctx, N, Kd) bytes of device
 *                memory, 16-byte aligned, the call's own until it has run (0: NULL
 *                will do): few small gradients are computed in shares of their rows
 * accumulate: both are added to instead (one addition per element).  Sums are in a
 * fixed order.  N % 8 == 0, Kd % 8 == 0, each at most 2^20.  Runs on pairs of SMs: at least one pair,
 * however few SMs the context may use. */
size_t moonep_expert_weight_grad_workspace(const moonep_ctx *ctx, int N,
                                           int Kd);
int moonep_expert_weight_grad(moonep_ctx *ctx, const int32_t *cu_seqlens,
                              const uint16_t *x, int64_t x_row_bytes,
                              const uint16_t *d, int64_t d_row_bytes, int N,
                              int Kd, int accumulate, float *grad,
                              float *slots, void *workspace, void *stream);

/* The experts' gated activation over the dispatched layout, times the route
 * weight (combine sums unweighted):
 *   act[row, f] = w[row] * gate * sigmoid(gate) * up
 * gate, up, act [R*NvS, F] bf16, F % 32 == 0, w_nvs [R*NvS] fp32 or NULL (1);
 * fp32 inside, one rounding.  With a checkpoint (all four given, or all
 * NULL): gate and up as E4M3 codes [R*NvS, F] uint8 with E8M0 scales
 * [R*NvS, F/32] (largest exponent 8, saturating at 448; otherwise as
 * moonep_quantize_mx).  Only rows that belong to a segment are read and
 * written. */
int moonep_gated_act(moonep_ctx *ctx, const int32_t *cu_seqlens,
                     const uint16_t *gate, const uint16_t *up,
                     const float *w_nvs, int F, uint16_t *act, uint8_t *gate8,
                     uint8_t *up8, uint8_t *gate_scales, uint8_t *up_scales,
                     void *stream);

/* Backward pass from the checkpoint: the formula's gradient at the gate and
 * up values that the checkpoint stands for.  d_act [R*NvS, F] bf16 ->
 * d_gate, d_up [R*NvS, F] bf16 and, when given, d_w_nvs [R*NvS] fp32 (sum
 * over f in a fixed order), which moonep_combine gathers back to [R, S, K]. */
int moonep_gated_act_backward(moonep_ctx *ctx, const int32_t *cu_seqlens,
                              const uint8_t *gate8, const uint8_t *up8,
                              const uint8_t *gate_scales,
                              const uint8_t *up_scales, const uint16_t *d_act,
                              const float *w_nvs, int F, uint16_t *d_gate,
                              uint16_t *d_up, float *d_w_nvs, void *stream);

/* The norm of many gradients: norm[0] = sqrt(sum over all tensors of g^2), fp32
 * in device memory.  g is a host array of n_tensors device pointers (fp32, or
 * bf16 when g_bf16; any element alignment), sizes their elements.  Squares are
 * taken in fp32 (below 2^-126 they lose bits, from 2^128 on they are
 * infinite), sums of eight in fp32 and the rest in 45 bits or more, in a fixed
 * order.
 * workspace: moonep_grad_norm_workspace(ctx) bytes of device memory, 8-byte
 * aligned, the call's own until it has run. */
size_t moonep_grad_norm_workspace(const moonep_ctx *ctx);
int moonep_grad_norm(moonep_ctx *ctx, int n_tensors, const void *const *g,
                     const int64_t *sizes, int g_bf16, void *workspace,
                     float *norm, void *stream);

/* One AdamW step over many tensors, in place:
 *   g' = g min(1, max_norm / norm[0])        (g without a norm)
 *   m = beta1 m + (1 - beta1) g'    v = beta2 v + (1 - beta2) g'^2
 *   p = p (1 - lr wd) - lr / (1 - beta1^step) m /
 *                       (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * in fp32, subnormals kept (a g'^2 (1 - beta2) below 2^-150 is 0).  When norm[0] is
 * not finite the call changes nothing.  No two tensors overlap.
 *   p, g     n_tensors host arrays of device pointers, fp32 or bf16 (one type
 *            per call each), any element alignment; sizes: elements, >= 0
 *   m, v     bits 32: fp32; bits 8: codes, uint8, with ms, vs their scales;
 *            16-byte aligned.  Of a tensor of n elements they hold n rounded up
 *            to a multiple of 32 (8 bits: a scale byte for every 32), the ones
 *            past n zero; a new state is all zero
 *   w        NULL, or per tensor NULL or a bf16 tensor that receives p rounded
 *            to nearest even (fp32 p only)
 * Moments in 8 bits: every 32 values share the power 2^(s - 127), the smallest
 * (s >= 0) under which none saturates; m is E4M3, v code c stands for c/8
 * (c < 8) or (1 + (c & 7)/8) 2^(c/8 - 1).  A block with a NaN or an infinity gets
 * the scale 255 and reads back as NaN.  Values round to nearest even; when
 * seeded, up with the probability that makes them right on average, and so does
 * a bf16 p, by 16 bits of a hash of (seed, step, tensor's place, element).  A v
 * above zero keeps at least code 1.
 *   lr_dev, step_dev   device scalars used in place of lr and step when given
 *            (a captured step then goes on from replay to replay); a step below
 *            1 there counts as 1
 * 0 <= beta < 1, 2^-126 <= eps <= 2^125, step >= 1, and max_norm > 0 with a norm. */
typedef struct moonep_adamw_config {
  double lr, beta1, beta2, eps, weight_decay;
  const float *lr_dev;
  const int32_t *step_dev;
  const float *norm;
  float max_norm;
  int32_t step;
  uint32_t seed;
  int seeded;
  int bits;   /* 32 or 8 */
  int p_bf16, g_bf16;
} moonep_adamw_config;
int moonep_adamw(moonep_ctx *ctx, const moonep_adamw_config *config,
                 int n_tensors, const int64_t *sizes, void *const *p,
                 const void *const *g, void *const *m, void *const *v,
                 uint8_t *const *ms, uint8_t *const *vs, uint16_t *const *w,
                 void *stream);

/* The values of n (a multiple of 32) moments in 8 bits, bf16 (fp32 when fp32);
 * every pointer 16-byte aligned but the scales'. */
int moonep_adamw_moments(moonep_ctx *ctx, int64_t n, const uint8_t *m8,
                         const uint8_t *ms, const uint8_t *v8,
                         const uint8_t *vs, int fp32, void *m, void *v,
                         void *stream);

/* Zero-copy aliases [API, Buffer.hidden_nvsh_buffer_view and
 * router_weight_buffer_view]: device address of rank `rank`'s [NvS, H] bf16
 * window (row rank*NvS of the context's hidden buffer) and of its [NvS] fp32
 * weight window.  NULL if the context was created without views or the rank
 * is out of range.  Later calls overwrite what they hold. */
void *moonep_hidden_view(moonep_ctx *ctx, int rank);
void *moonep_weight_view(moonep_ctx *ctx, int rank);

/* Synchronise `stream`, return the first error any kernel latched since the
 * last call in *device_status (0 if none) and clear it.  After
 * MOONEP_ERR_TIMEOUT it also clears the planner's cross-block counters and
 * accumulators (a wait that ran out may leave them out of step), so the
 * context plans correctly again; re-plan before reusing a plan from that
 * call.  The return value is the host-side status of the query itself. */
int moonep_get_status(moonep_ctx *ctx, int *device_status, void *stream);

/* Static text for a status code. */
const char *moonep_strerror(int code);

/* Number of SMs the copy kernels use for this context. */
int moonep_num_sms(const moonep_ctx *ctx);

#ifdef __cplusplus
}
#endif
#endif /* MOONEP_H */
