/*
 * ep.h -- C ABI of the MI355X (gfx950) MoE expert-parallel dispatch / combine
 * library (libep.so).
 *
 * The operations are the expert-parallel hot path of the page
 * "[Not ready] MSCCLPP EP implementation #852" (microsoft/mscclpp pull 852):
 *   - get_dispatch_layout (PR body, "Scope / Intranode" and "Internode HT"),
 *   - dispatch and combine over the x[T,H] bf16 / topk_idx[T,k] int64 /
 *     topk_weights[T,k] fp32 tensor ABI (same section),
 *   - the low-latency dispatch with per-token FP8 casting and one scale per
 *     128 channels (low-latency port commit, dispatch<kUseFP8,...>),
 *   - combine consuming the receiver-side layout produced by dispatch (commit
 *     fixing internode HT combine: receiver-side prefix sums),
 * and, around that path, routing, the experts' products with 4-bit weights and
 * the gradients of routing and combine.
 * On one GPU every destination "rank" is a contiguous range of one receive
 * buffer in this GPU's HBM: experts are split into num_ranks contiguous
 * blocks of num_experts/num_ranks, and rank r's rows are
 * [recv_rank_offset[r], recv_rank_offset[r+1]).
 *
 * Conventions shared by every entry point
 * ----------------------------------------
 * Pointers.  Every array argument is a DEVICE pointer (HBM of the current HIP
 * device), row-major and densely packed, owned by the caller; the library
 * keeps no reference after the call returns and allocates nothing at run
 * time (ep_dispatch_noalloc's fixed scratch is part of the loaded code).  The
 * workspace is caller-owned device memory of at least the size reported by
 * the matching *_workspace_bytes() call, 4-byte aligned (the kernels keep
 * 32-bit counters there; EP_ERR_INVALID_ARGUMENT otherwise); its contents on
 * entry do not matter and on exit are unspecified.
 *
 * bf16 data is passed as raw 16-bit patterns (void*).
 *
 * Streams.  `stream` is a hipStream_t (NULL = the default stream).  Every call
 * only validates its arguments on the host and enqueues kernels on `stream`;
 * it never synchronises.  Outputs are valid once the stream reaches that
 * point.  Calls on different streams touching disjoint buffers may run
 * concurrently; the library holds no mutable global state apart from the
 * fixed device scratch of ep_dispatch_noalloc (below) and the per-device
 * cache of its address, filled once under a lock.
 *
 * Routing slots.  Slot (t, j) is valid iff 0 <= topk_idx[t*k + j] <
 * num_experts.  Any other value (conventionally -1) is an empty slot: it gets
 * no receive row, no count, and token_row = -1.  The same expert may appear
 * twice in a token; each slot then gets its own row.
 *
 * Receive order.  Rows are grouped by expert (ascending), so every rank's
 * experts are one contiguous range; inside an expert, rows follow (t, j)
 * ascending.  This order is unique, so every index output is deterministic
 * and bit-reproducible.  Receive buffers are sized at capacity
 * num_tokens * num_topk rows; the filled row count is
 * recv_expert_offset[num_experts]; rows beyond it are not written.
 *
 * Errors.  Every entry point returns an ep_status_t (as int).  Invalid
 * arguments are detected on the host before anything is enqueued and leave
 * all outputs untouched.  EP_ERR_HIP reports a failed launch
 * (hipGetLastError).  ep_last_error() returns a thread-local description of
 * the last failure on the calling thread.  No C++ exception crosses the ABI.
 */
#ifndef EP_MI355X_EP_H
#define EP_MI355X_EP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    EP_OK = 0,
    EP_ERR_INVALID_ARGUMENT = 1,   /* null pointer, bad size, misalignment, ... */
    EP_ERR_UNSUPPORTED = 2,        /* valid but beyond the library's limits     */
    EP_ERR_WORKSPACE_TOO_SMALL = 3,
    EP_ERR_HIP = 4                 /* a HIP runtime call or launch failed        */
} ep_status_t;

/* Limits of the library (EP_ERR_UNSUPPORTED beyond them). */
#define EP_MAX_TOPK 64          /* num_topk                                   */
#define EP_MAX_RANKS 64         /* num_ranks                                  */
#define EP_MAX_EXPERTS 2048     /* num_experts                                */
/* The bf16 copies (ep_dispatch, ep_dispatch_cached, ep_dispatch_ht,
 * ep_dispatch_ll) run in one
 * launch of T * ceil(H / 1024) blocks of 64 * min(fanout, 8) threads, where
 * fanout is num_topk (num_ranks for ep_dispatch_ht); a launch holds at most
 * 2^32 - 1 threads, and larger shapes return EP_ERR_UNSUPPORTED before any
 * work is enqueued (e.g. T = 2^20 tokens of H = 8192 at fanout 8). */

/* Static description of a status code; never NULL. */
const char* ep_status_string(int status);

/* Thread-local text of the last non-EP_OK status returned on this thread. */
const char* ep_last_error(void);

/* Library version string, e.g. "ep-mi355x 0.1 gfx950". */
const char* ep_version(void);

/* ---------------------------------------------------------------------------
 * ep_get_dispatch_layout -- routing histogram of one batch (get_dispatch_layout
 * of the page's "Scope / Intranode"; the per-group count is the per-RDMA-rank
 * count of "Scope / Internode HT", a group being ranks_per_group consecutive
 * ranks).
 *
 *   topk_idx              [T, k] int64   routing (see "Routing slots")
 *   num_tokens_per_rank   [R]    int32   out: tokens with >= 1 valid slot on r
 *   num_tokens_per_group  [R/P]  int32   out: tokens touching any rank of group
 *                                        g (may be NULL)
 *   num_tokens_per_expert [E]    int32   out: valid slots routed to e
 *   is_token_in_rank      [T, R] uint8   out: 1 iff token t has a valid slot on
 *                                        rank r, else 0
 *
 * Requires T >= 0, 1 <= k <= EP_MAX_TOPK, 1 <= R <= EP_MAX_RANKS,
 * E % R == 0, E <= EP_MAX_EXPERTS, 1 <= P, R % P == 0.  T == 0 writes zero
 * counts.  Workspace: ep_layout_workspace_bytes(T, E, R, P).
 * ------------------------------------------------------------------------- */
size_t ep_layout_workspace_bytes(int64_t num_tokens, int num_experts, int num_ranks,
                                 int ranks_per_group);

int ep_get_dispatch_layout(const int64_t* topk_idx, int64_t num_tokens, int num_topk,
                           int num_experts, int num_ranks, int ranks_per_group,
                           int32_t* num_tokens_per_rank, int32_t* num_tokens_per_group,
                           int32_t* num_tokens_per_expert, uint8_t* is_token_in_rank,
                           void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * ep_dispatch -- permute each token's hidden vector into the contiguous
 * per-rank / per-expert receive buffer (intranode dispatch of "Scope /
 * Intranode"), and emit the receiver-side maps that combine consumes.
 *
 *   x                  [T, H]  bf16  in: token activations (16-byte aligned)
 *   topk_idx           [T, k]  int64 in
 *   topk_weights       [T, k]  fp32  in (may be NULL)
 *   recv_x             [T*k, H] bf16 out: recv_x[token_row[t,j]] = x[t], bit
 *                                    for bit (16-byte aligned)
 *   recv_src_idx       [T*k]   int32 out: source token of each filled row
 *   recv_topk_weights  [T*k]   fp32  out: topk_weights[t,j] of each filled row
 *                                    (may be NULL; ignored if topk_weights is)
 *   recv_expert_offset [E+1]   int32 out: first row of each expert; [E] = rows
 *   recv_rank_offset   [R+1]   int32 out: recv_expert_offset[r*E/R] (may be NULL)
 *   token_row          [T, k]  int32 out: row of slot (t,j), -1 if empty
 *
 * Requires H % 8 == 0 (rows are whole 16-byte vectors), T*k < 2^31, the
 * layout limits above and (bf16) the copy-launch limit.
 * Workspace: ep_dispatch_workspace_bytes(T, k, E).
 * The offsets are computed from topk_idx itself, so no earlier call's output
 * is trusted and every write stays inside the buffers described above.
 * ------------------------------------------------------------------------- */
size_t ep_dispatch_workspace_bytes(int64_t num_tokens, int num_topk, int num_experts);

int ep_dispatch(const void* x, const int64_t* topk_idx, const float* topk_weights,
                int64_t num_tokens, int hidden, int num_topk, int num_experts, int num_ranks,
                void* recv_x, int32_t* recv_src_idx, float* recv_topk_weights,
                int32_t* recv_expert_offset, int32_t* recv_rank_offset, int32_t* token_row,
                void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * ep_dispatch_noalloc -- ep_dispatch for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid allocation): the same operation, kernels and outputs as ep_dispatch,
 * with no workspace argument.  The receive-order scratch is a fixed device
 * array inside the library, EP_NOALLOC_SCRATCH_BYTES per GPU, held until the
 * process ends; the call itself allocates nothing.
 *
 * Arguments and outputs as ep_dispatch.  The stream must belong to the
 * current HIP device.  A batch whose scratch need,
 * ep_dispatch_workspace_bytes(T, k, E), exceeds EP_NOALLOC_SCRATCH_BYTES
 * returns EP_ERR_UNSUPPORTED before anything is enqueued (e.g. 32768 tokens
 * at top-8 need 64 KiB + 256 B over 256 experts, 512 KiB + 256 B over 2048).
 * All calls on one GPU share that GPU's array: calls that overlap on one GPU
 * (two streams, two threads) race and must be serialised by the caller.
 * ------------------------------------------------------------------------- */
#define EP_NOALLOC_SCRATCH_BYTES (1u << 20)

int ep_dispatch_noalloc(const void* x, const int64_t* topk_idx, const float* topk_weights,
                        int64_t num_tokens, int hidden, int num_topk, int num_experts,
                        int num_ranks, void* recv_x, int32_t* recv_src_idx,
                        float* recv_topk_weights, int32_t* recv_expert_offset,
                        int32_t* recv_rank_offset, int32_t* token_row, void* stream);

/* ---------------------------------------------------------------------------
 * ep_dispatch_fp8 -- ep_dispatch with the low-latency FP8 cast (low-latency
 * port commit, dispatch<kUseFP8,...>).  For token t and 128-channel block c:
 *   a = max |x[t, 128c .. 128c+127]|,  s = a / 448 (IEEE fp32 division),
 *   code = E4M3(x / s) (OCP E4M3FN, round to nearest even, saturating at
 *   +-448), or 0x00 for every channel when s == 0.
 * Every row of the token receives the same codes and scales:
 *   recv_x_fp8  [T*k, H]     uint8 out: E4M3FN codes (16-byte aligned)
 *   recv_scales [T*k, H/128] fp32  out: s per 128-channel block
 * All other arguments as ep_dispatch.  Requires H % 128 == 0.
 * Workspace: ep_dispatch_workspace_bytes(T, k, E).
 * ------------------------------------------------------------------------- */
int ep_dispatch_fp8(const void* x, const int64_t* topk_idx, const float* topk_weights,
                    int64_t num_tokens, int hidden, int num_topk, int num_experts,
                    int num_ranks, uint8_t* recv_x_fp8, float* recv_scales,
                    int32_t* recv_src_idx, float* recv_topk_weights,
                    int32_t* recv_expert_offset, int32_t* recv_rank_offset,
                    int32_t* token_row, void* workspace, size_t workspace_bytes,
                    void* stream);

/* ---------------------------------------------------------------------------
 * ep_dispatch_cached / ep_dispatch_fp8_cached -- repeat dispatch that reuses
 * the receive map of an earlier ep_dispatch / ep_dispatch_fp8 with the same
 * routing (the cached_notify of page #852, "Scope / Internode HT": a repeat
 * dispatch skips the layout and count exchange).  No receive-order work is
 * done: for every slot (t, j) whose row r = token_row[t, j] lies in
 * [0, recv_rows), row r receives x[t] (bf16, bit for bit) or its FP8 cast
 * (codes and scales exactly as ep_dispatch_fp8 computes them).  Slots with
 * any other row, including -1, are skipped, so no map can make the kernel
 * write outside the recv_rows rows given.  Other rows are not written.
 *
 *   x           [T, H]          bf16  in (16-byte aligned)
 *   token_row   [T, k]          int32 in (an earlier dispatch's output)
 *   recv_x      [recv_rows, H]  bf16  out (16-byte aligned)
 *   recv_x_fp8  [recv_rows, H]  uint8 out (16-byte aligned), recv_scales
 *               [recv_rows, H/128] fp32 out (FP8 variant)
 * Requires H % 8 == 0 (bf16) or H % 128 == 0 (FP8), 1 <= k <= EP_MAX_TOPK
 * and (bf16) the copy-launch limit.
 * No workspace.  T == 0 or recv_rows == 0 enqueues nothing.
 * ------------------------------------------------------------------------- */
int ep_dispatch_cached(const void* x, const int32_t* token_row, int64_t num_tokens, int hidden,
                       int num_topk, void* recv_x, int64_t recv_rows, void* stream);

int ep_dispatch_fp8_cached(const void* x, const int32_t* token_row, int64_t num_tokens,
                           int hidden, int num_topk, uint8_t* recv_x_fp8, float* recv_scales,
                           int64_t recv_rows, void* stream);

/* ---------------------------------------------------------------------------
 * ep_dispatch_ht -- rank-deduplicated ("high-throughput") dispatch: the
 * intranode dispatch of page #852, "Scope / Intranode", which sends each
 * token once to every rank hosting at least one of its experts, the receiver
 * seeing the token's top-k ids remapped to its local experts.  One receive
 * row per (token t, rank r) with t routed to r (is_token_in_rank[t, r] = 1),
 * ordered by rank, then token:
 *
 *   recv_x            [T*R, H]  bf16  out: row = x[t], bit for bit (capacity
 *                                     T*R rows; recv_rank_offset[R] filled)
 *   recv_src_idx      [T*R]     int32 out: source token of each filled row
 *   recv_topk_idx     [T*R, k]  int64 out: topk_idx[t, j] - r*E/R when that
 *                                     expert is on rank r, else -1
 *   recv_topk_weights [T*R, k]  fp32  out: topk_weights[t, j] on the same
 *                                     condition, else 0 (may be NULL)
 *   recv_rank_offset  [R+1]     int32 out: first row of each rank; [R] = rows
 *   token_rank_row    [T, R]    int32 out: row of (t, r), or -1
 *
 * The matching combine is ep_combine(expert_out, rows, token_rank_row, NULL,
 * T, H, R, out): out[t] = bf16(sum over ranks, in rank order, of the rank's
 * row for t), each row holding that rank's already weighted partial result.
 * Requires H % 8 == 0, T*R < 2^31, the routing limits above and the
 * copy-launch limit with fanout R.
 * Workspace: ep_dispatch_ht_workspace_bytes(T, R).
 * ------------------------------------------------------------------------- */
size_t ep_dispatch_ht_workspace_bytes(int64_t num_tokens, int num_ranks);

int ep_dispatch_ht(const void* x, const int64_t* topk_idx, const float* topk_weights,
                   int64_t num_tokens, int hidden, int num_topk, int num_experts, int num_ranks,
                   void* recv_x, int32_t* recv_src_idx, int64_t* recv_topk_idx,
                   float* recv_topk_weights, int32_t* recv_rank_offset, int32_t* token_rank_row,
                   void* workspace, size_t workspace_bytes, void* stream);

/* ---------------------------------------------------------------------------
 * ep_dispatch_ll / ep_dispatch_ll_fp8 -- padded expert-major ("low-latency")
 * dispatch.  Page #852: the LL benchmark's receive buffer is one fixed-size
 * region per expert (the commit that stops cloning that buffer inside the
 * timed loop), and the low-latency runtime is tested at capacities 1 and 2.
 * With one source the receive buffer is [E, capacity, H]; expert e owns rows
 * e*capacity .. e*capacity + capacity - 1, filled in (token, slot) order, and
 * a slot that finds its region full is dropped:
 *
 *   recv_x            [E, capacity, H]  bf16 out: slot = x[t], bit for bit
 *     (ep_dispatch_ll_fp8: recv_x_fp8 [E, capacity, H] E4M3FN codes and
 *      recv_scales [E, capacity, H/128] fp32, the cast of ep_dispatch_fp8)
 *   recv_count        [E]          int32 out: min(slots routed to e, capacity)
 *   recv_src_idx      [E, capacity] int32 out: source token of each filled slot
 *   recv_topk_weights [E, capacity] fp32  out: topk_weights[t, j] of each
 *                                     filled slot (may be NULL; ignored if
 *                                     topk_weights is NULL)
 *   token_slot        [T, k]       int32 out: e*capacity + position of (t, j),
 *                                     or -1 (empty slot, or dropped)
 *
 * Rows recv_count[e] .. capacity-1 of each expert are not written.  Combine:
 * ep_combine(expert_out [E*capacity, H], E*capacity, token_slot, weights, ...);
 * a dropped slot then contributes nothing.  capacity = T never drops.
 * Requires 1 <= capacity, E*capacity < 2^31, H % 8 == 0 (bf16) or
 * H % 128 == 0 (FP8), the routing limits above (ranks are not involved) and
 * (bf16) the copy-launch limit.  Workspace: ep_dispatch_ll_workspace_bytes.
 * ------------------------------------------------------------------------- */
size_t ep_dispatch_ll_workspace_bytes(int64_t num_tokens, int num_topk, int num_experts);

int ep_dispatch_ll(const void* x, const int64_t* topk_idx, const float* topk_weights,
                   int64_t num_tokens, int hidden, int num_topk, int num_experts, int capacity,
                   void* recv_x, int32_t* recv_count, int32_t* recv_src_idx,
                   float* recv_topk_weights, int32_t* token_slot, void* workspace,
                   size_t workspace_bytes, void* stream);

int ep_dispatch_ll_fp8(const void* x, const int64_t* topk_idx, const float* topk_weights,
                       int64_t num_tokens, int hidden, int num_topk, int num_experts,
                       int capacity, uint8_t* recv_x_fp8, float* recv_scales,
                       int32_t* recv_count, int32_t* recv_src_idx, float* recv_topk_weights,
                       int32_t* token_slot, void* workspace, size_t workspace_bytes,
                       void* stream);

/* ---------------------------------------------------------------------------
 * ep_combine -- gather each token's expert outputs back and sum them weighted
 * by topk_weights (intranode combine of "Scope / Intranode", consuming the
 * receiver-side map token_row that dispatch produced).  For every t, h:
 *   acc = +0.0f;  for j = 0 .. k-1 in this order, if 0 <= token_row[t,j] < num_rows:
 *       acc = fmaf(topk_weights[t,j], expert_out[token_row[t,j], h], acc);
 *   combined_x[t, h] = bf16(acc), rounded to nearest even.
 * topk_weights may be NULL: every weight is then 1 (a plain fp32 sum in j
 * order), which is the combine of ep_dispatch_ht's per-rank rows.
 *
 *   expert_out   [num_rows, H] bf16 in (16-byte aligned)
 *   token_row    [T, k]        int32 in (from ep_dispatch; a slot whose row
 *                              lies outside [0, num_rows) contributes nothing.
 *                              For small batches the kernel still issues a
 *                              load for such a slot -- of row 0 of expert_out,
 *                              or, when num_rows == 0, of the token's own
 *                              combined_x segment before writing it -- and
 *                              discards the value; nothing outside the
 *                              buffers described here is read)
 *   topk_weights [T, k]        fp32  in (NULL: all weights 1)
 *   combined_x   [T, H]        bf16  out (16-byte aligned)
 * Requires H % 8 == 0, 1 <= k <= EP_MAX_TOPK, num_rows >= 0.  No workspace.
 * ------------------------------------------------------------------------- */
int ep_combine(const void* expert_out, int64_t num_rows, const int32_t* token_row,
               const float* topk_weights, int64_t num_tokens, int hidden, int num_topk,
               void* combined_x, void* stream);

/* ---------------------------------------------------------------------------
 * ep_route -- router logits to the topk_idx / topk_weights that every dispatch
 * entry point takes.  For each token t:
 *   score   s[e] = softmax over all E logits, or sigmoid of each logit.
 *   choice  c[e] = fl32(s[e]) + bias[e] in fp32, where fl32 rounds the score
 *           from 64 bits.  With bias NULL and either one group or
 *           group_top == 1 experts are ranked by the logits themselves: the
 *           order of the exact scores, free of their rounding.
 *   An expert whose logit or choice is -inf or NaN is unavailable: it is never
 *   chosen.  A logit of -inf or NaN also has a softmax term of 0.  A bias steers
 *   the choice only: an expert that it makes unavailable keeps its score, which
 *   counts in the sum over all E logits (mask the logit to leave it out).
 *   groups  num_groups contiguous blocks of E / num_groups experts.  A group's
 *           score is the fp32 sum of its group_top (1 or 2) largest available
 *           choices; only the experts of the topk_groups best groups stay.
 *   topk_idx[t]  the k largest choices that stay, in descending order.
 *   topk_weights[t, j] = scale * s[topk_idx[t, j]], divided by the sum of the
 *           chosen scores if renormalize is not 0.  (The bias only steers the
 *           choice.)  The division happens before any underflow: scores too
 *           small for fp32 still renormalise to weights that add to scale.
 * Ties go to the lowest expert (or group) index.  Where fewer than k experts
 * are available the remaining slots are empty: topk_idx -1, topk_weights 0 (a
 * token whose logits are all -inf gets k empty slots, so padding tokens are
 * dispatched nowhere).  Infinite logits: sigmoid is 1; softmax shares the
 * whole score equally among a token's +inf logits.
 *
 *   logits        [T, E] in, of type logits_type (EP_TYPE_*), aligned to its
 *                        element
 *   bias          [E]    fp32  in (may be NULL)
 *   topk_idx      [T, k] int64 out
 *   topk_weights  [T, k] fp32  out
 * Requires T >= 0, 1 <= E <= EP_MAX_EXPERTS, 1 <= k <= EP_MAX_TOPK,
 * T*k < 2^31, 1 <= num_groups <= EP_MAX_GROUPS, E % num_groups == 0,
 * 1 <= topk_groups <= num_groups, k <= topk_groups * E / num_groups, a finite
 * scale.  Outputs must not overlap inputs.  No workspace.
 *
 * ep_route_backward -- gradient of topk_weights with respect to the logits
 * (the choice itself has none, nor has the bias).  With g = grad_weights[t],
 * s as above and p[j] the renormalised weight (before scale) of slot j:
 *   softmax, renormalize: d logit += scale * p[j] * (g[j] - sum_i g[i] p[i])
 *   sigmoid, renormalize: the same times (1 - s)
 *   sigmoid:              d logit += scale * g[j] * s * (1 - s)
 *   softmax:              d logit[e] = scale * s[e] * (sum of g[j] over the
 *                         slots that chose e - sum_i g[i] s[topk_idx[i]])
 * each added at the expert of slot j, in slot order and in fp32, and rounded
 * once to the logits' type; every other element is 0.  Empty slots (ids
 * outside [0, E)) and unavailable logits contribute nothing.
 *
 *   topk_idx      [T, k] int64 in (of ep_route; an id may appear twice)
 *   grad_weights  [T, k] fp32  in
 *   grad_logits   [T, E] out, of type logits_type
 * Limits, alignment and overlap as ep_route; no workspace.
 * ------------------------------------------------------------------------- */
#define EP_TYPE_F32 0
#define EP_TYPE_BF16 1
#define EP_TYPE_F16 2
#define EP_SCORE_SOFTMAX 0
#define EP_SCORE_SIGMOID 1
#define EP_MAX_GROUPS 64        /* num_groups of ep_route                     */

int ep_route(const void* logits, int logits_type, const float* bias, int64_t num_tokens,
             int num_experts, int num_topk, int score, int num_groups, int topk_groups,
             int group_top, int renormalize, float scale, int64_t* topk_idx,
             float* topk_weights, void* stream);

int ep_route_backward(const void* logits, int logits_type, const int64_t* topk_idx,
                      const float* grad_weights, int64_t num_tokens, int num_experts,
                      int num_topk, int score, int renormalize, float scale, void* grad_logits,
                      void* stream);

/* ---------------------------------------------------------------------------
 * ep_combine_backward -- gradient of ep_combine.  With g = grad_out[t], for
 * every slot (t, j) whose row r = token_row[t, j] lies in [0, num_rows):
 *   grad_expert_out[r, h]   = bf16(topk_weights[t, j] * g[h])
 *   grad_topk_weights[t, j] = sum over h of g[h] * expert_out[r, h], in fp32
 * and grad_topk_weights[t, j] = 0 for every other slot.  Rows that no slot
 * maps to are not written.  Rows have to be distinct, as every dispatch makes
 * them: what is written to a row of grad_expert_out that two slots name is
 * unspecified (grad_topk_weights is as above).
 * (The gradient of ep_dispatch with respect to x is ep_combine over the same
 * token_row with topk_weights NULL.)
 *
 *   grad_out          [T, H]        bf16 in (16-byte aligned)
 *   expert_out        [num_rows, H] bf16 in (16-byte aligned; may be NULL if
 *                                   grad_topk_weights is)
 *   token_row         [T, k]        int32 in
 *   topk_weights      [T, k]        fp32 in (NULL: all weights 1)
 *   grad_expert_out   [num_rows, H] bf16 out (16-byte aligned; may be NULL)
 *   grad_topk_weights [T, k]        fp32 out (may be NULL, but not both)
 * Requires H % 8 == 0, 1 <= k <= EP_MAX_TOPK, T*k < 2^31, num_rows >= 0.
 * Outputs must not overlap inputs.  No workspace.
 * ------------------------------------------------------------------------- */
int ep_combine_backward(const void* grad_out, const void* expert_out, int64_t num_rows,
                        const int32_t* token_row, const float* topk_weights, int64_t num_tokens,
                        int hidden, int num_topk, void* grad_expert_out,
                        float* grad_topk_weights, void* stream);

/* ---------------------------------------------------------------------------
 * ep_expert_linear_w4 -- the experts' products over dispatched rows, with
 * 4-bit weights: y[r, n] = sum over i of x[r, i] * W[e, n, i] for every row r
 * of expert e, accumulated in fp32 and rounded once to bf16.
 * A weight is an OCP E2M1 code (sign, 2 exponent bits, 1 mantissa bit: 0, 0.5,
 * 1, 1.5, 2, 3, 4, 6 and their negatives) times the scale 2^(b - 127) of its
 * group of 32 consecutive inputs (E8M0 byte b; 255 is NaN).  A weight of 2^128
 * or more (codes 4 and 6 at b >= 253, 2 and 3 too at b = 254) is infinite.
 *
 * Rows.  capacity == 0: the packed receive order of ep_dispatch, expert_rows
 * being recv_expert_offset [E+1] (rows expert_rows[e] .. expert_rows[e+1]-1).
 * capacity > 0: the padded layout of ep_dispatch_ll, expert_rows being
 * recv_count [E] (rows e*capacity .. e*capacity + expert_rows[e] - 1) and
 * num_rows = E*capacity.  Offsets are limited to [0, num_rows] and counts to
 * [0, capacity], and of offsets out of order an expert takes only rows that no
 * expert before it has, so no map can make the kernel touch rows outside x and
 * y or do more than num_rows rows' work.  Rows of no expert are neither read
 * for a result nor written.
 *
 * Epilogue.  EP_EPILOGUE_NONE: W has out_features rows.
 * EP_EPILOGUE_SILU_MUL: W has 2*out_features rows, first the gate's, then the
 * up projection's, and y = bf16(silu(gate) * up) with gate and up kept in
 * fp32; silu(v) = v / (1 + exp(-v)).
 *
 *   x           [num_rows, in_features]     bf16  in (16-byte aligned)
 *   expert_rows [E+1] or [E]                int32 in
 *   w_codes     [E, W rows, in_features/2]  uint8 in (16-byte aligned), two
 *               codes a byte, the even input in the low four bits
 *   w_scales    [E, W rows, in_features/32] uint8 in (4-byte aligned)
 *   y           [num_rows, out_features]    bf16  out (16-byte aligned)
 * Requires in_features % 128 == 0, out_features % 8 == 0, both positive,
 * in_features <= EP_MAX_IN_FEATURES,
 * 1 <= E <= EP_MAX_EXPERTS, 0 <= num_rows < 2^31, capacity >= 0.  y must not
 * overlap the inputs.  No workspace.
 * ------------------------------------------------------------------------- */
#define EP_EPILOGUE_NONE 0
#define EP_EPILOGUE_SILU_MUL 1
#define EP_MAX_IN_FEATURES (1 << 22)

int ep_expert_linear_w4(const void* x, int64_t num_rows, const int32_t* expert_rows, int capacity,
                        const uint8_t* w_codes, const uint8_t* w_scales, int num_experts,
                        int in_features, int out_features, int epilogue, void* y, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* EP_MI355X_EP_H */
