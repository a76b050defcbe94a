/*
 * moe_dispatch.h -- C ABI of the MI355X (gfx950) MoE token dispatch / combine
 * library (libmoe_dispatch.so).
 *
 * The three entry points are the local (one-device) stages of the pair of
 * operators documented on the torch_npu API reference page for
 * npu_moe_distribute_combine (Ascend): the dispatch side lays token rows out
 * expert-contiguously and returns expand_idx and the send counts in
 * prefix-sum form; the combine side retraces that path back to token order
 * and forms the weighted sum of the formula in that page's 计算公式 (formula)
 * section.
 * With one device the page's ReduceScatterV (tensor-parallel) and AlltoAllv
 * (expert-parallel) exchanges are identities: the whole expert set is the one
 * expert-parallel rank's share.
 *
 * Conventions for every call:
 *  - Tensor pointers are DEVICE pointers owned by the caller (for example
 *    allocated by PyTorch).  The library allocates nothing, keeps no state
 *    between calls (apart from the per-thread timing events of
 *    moe_time_next_launches in moe_probe.h, a measurement aid) and is safe
 *    to call from several host threads.
 *  - `stream` is a hipStream_t passed as void* (NULL = the null stream).  A
 *    call validates its arguments on the host, enqueues its kernels on
 *    `stream` and returns; it never synchronises.  Buffers must stay alive
 *    and unmodified until the stream has finished the call (the page on the
 *    DeepSeek Ascend toolchain, troubleshooting step 5: reuse or free buffers
 *    only after the asynchronous work is done).
 *  - Row strides are counted in elements of the row's own type.
 *  - A failed argument check returns a non-zero moe_status and enqueues
 *    nothing.  Problems that only the device can see (ids out of range,
 *    repeated ids, a slot beyond the buffer) set bits of the optional
 *    device-side `status` word and the offending pair is skipped; no write
 *    ever leaves the caller's buffers (the DeepEP compensation PR, Kernel /
 *    host section: fail-safe bounds guards on the scatter writes).
 *  - No call waits on another device (same toolchain page, single-card
 *    compute section: a local operator never holds a cross-rank wait).
 */
#ifndef MOE_DISPATCH_H
#define MOE_DISPATCH_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
enum moe_status {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,   /* a shape, range, pointer or alignment rule failed */
    MOE_ERR_WORKSPACE = 2,     /* workspace_bytes below the call's workspace size */
    MOE_ERR_UNSUPPORTED = 3,   /* unknown dtype */
    MOE_ERR_HIP = 4,           /* the HIP runtime refused a launch */
    MOE_ERR_SCRATCH = 5        /* batch too large for moe_dispatch_fused_noalloc's scratch */
};

/* Element type of the dispatched buffer. */
enum moe_dtype {
    MOE_BF16 = 0,              /* bfloat16 bit copy of the token row */
    MOE_FP8_E4M3 = 1,          /* OCP e4m3fn (max 448) + one fp32 scale per 128 channels */
    MOE_FP32 = 2               /* float: norm weights and logits only */
};

/* Expert scores of moe_route, and how it ranks groups of experts. */
enum moe_score { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 };
enum moe_group_score {
    MOE_GROUP_TOP2 = 0,        /* the sum of a group's two largest scores (with the bias) */
    MOE_GROUP_MAX = 1          /* a group's largest key */
};

/* Bits of the device-side status word. */
enum moe_flag {
    MOE_FLAG_ID_RANGE = 1,     /* some expert_ids value lies outside [0, num_experts) */
    MOE_FLAG_DUP_ID = 2,       /* some row of expert_ids repeats an expert */
    MOE_FLAG_GUARD = 4,        /* some slot fell outside [0, capacity_rows): pair skipped */
    MOE_FLAG_REPLICA = 8       /* a replica table gave an expert no replica for some draw */
};

/* Version of this interface (incremented on any change of a signature or of
 * a caller's obligations; 2: the layout workspace must start zero-filled). */
int moe_abi_version(void);

/* Human-readable text of a moe_status value (static storage). */
const char* moe_status_string(int status);

/*
 * Rows of the expert-contiguous buffer that always hold the padded layout,
 * whatever the routing: with n = bs*k pairs, each expert's segment is rounded
 * up to a multiple of `align`, so the total is at most
 *   align * floor((n + (align-1) * min(num_experts, n)) / align).
 * This is the padded form of the page's rule that A, the number of rows a
 * card receives, be at least BS * min(local_expert_num, K) per source card
 * (npu_moe_distribute_combine, constraint notes on A).  Returns -1 when the
 * arguments break the rules of moe_dispatch_layout.
 */
int64_t moe_dispatch_capacity(int32_t bs, int32_t k, int32_t num_experts, int32_t align);

/* Bytes of device workspace moe_dispatch_layout (and the fused and
 * replica-aware calls) need for this shape: 0 when the whole layout fits one
 * workgroup (bs*k <= 2048; then `workspace` may be NULL).  Returns 0 for
 * invalid arguments as well; the layout call reports those.
 * The workspace must be zero-filled before its first use (for example with
 * hipMemset, or a fill kernel where a memset node is unwanted, as under
 * graph capture).  Its first word is an arrival counter that tells a ranking
 * workgroup it is the last to finish; every call leaves that word zero
 * again, so one workspace serves any number of calls of any shapes that fit
 * it, one call at a time.  The rest (the ranking workgroups' histograms,
 * which the last workgroup scans, their flags and ranks) needs no initial
 * contents. */
size_t moe_dispatch_layout_workspace_size(int32_t bs, int32_t k, int32_t num_experts);

/*
 * Layout: routing -> per-expert counts, padded prefix sum, stable ranks.
 *
 * Follows the parameters expert_ids, expand_idx and ep_send_counts of the
 * npu_moe_distribute_combine page (which are the paired dispatch operator's
 * outputs) and the 128-row M-tile padding of the grouped GEMM in the TEMPO
 * summary (section 1, padded compute).
 *
 *  expert_ids     in  int32 [bs, k], row-major, contiguous.  Values must lie in
 *                     [0, num_experts) and be distinct within a row (page rule).
 *  bs             in  tokens, >= 0 (0 is an empty batch: counts and offsets 0).
 *  k              in  experts per token, 1 <= k <= min(16, num_experts).
 *  num_experts    in  1 <= num_experts <= 512.
 *  align          in  segment alignment in rows, a power of two in [1, 1024];
 *                     128 matches the grouped GEMM's M-tile.
 *  expert_counts  out int32 [num_experts]: c_e = number of pairs routed to e.
 *  ep_send_counts out int32 [num_experts + 1]: exclusive prefix of the padded
 *                     counts ceil(c_e/align)*align; entry num_experts is the
 *                     padded total M_pad.  Every entry is a multiple of align.
 *  expand_idx     out int32 [bs * k]: for pair (t, j), the number of pairs
 *                     (t', j') before it in row-major order routed to the same
 *                     expert (the within-expert rank), or -1 if its id is out
 *                     of range.  Pair (t, j) lives in row
 *                     ep_send_counts[expert_ids[t,j]] + expand_idx[t*k+j].
 *  status         out int32 [1] or NULL: OR of MOE_FLAG_ID_RANGE and
 *                     MOE_FLAG_DUP_ID, overwritten (not accumulated).
 *                     Out-of-range pairs are excluded from the counts;
 *                     repeated ids are laid out like distinct ones.
 *  workspace      in/out device scratch of workspace_bytes >=
 *                     moe_dispatch_layout_workspace_size(bs, k, num_experts),
 *                     16-byte aligned, zero-filled before its first use (see
 *                     moe_dispatch_layout_workspace_size); calls that share a
 *                     workspace must not overlap.
 * The result is deterministic (no atomics decide any position).  Batches of
 * more than 2048 pairs take two launches: ranking workgroups of whole tokens
 * (at most 256, each walking chunks of at most 2048 pairs) write their
 * ranks and per-expert histograms, and the last of them to finish turns the
 * histograms into each expert's exclusive prefix over workgroups (a
 * device-wide scan in which every histogram entry is read and written once)
 * and writes the counts and ep_send_counts; a second launch adds each
 * workgroup's prefix to its ranks.  Work grows linearly with bs*k.
 */
int moe_dispatch_layout(const int32_t* expert_ids, int32_t bs, int32_t k, int32_t num_experts,
                        int32_t align, int32_t* expert_counts, int32_t* ep_send_counts,
                        int32_t* expand_idx, int32_t* status, void* workspace,
                        size_t workspace_bytes, void* stream);

/*
 * Rank-partitioned layout: moe_dispatch_layout plus the per-destination-rank
 * send offsets an expert-parallel all-to-all(v) needs.  The combine page's
 * A3-series ep_send_counts has ep_world_size * local_expert_num entries and
 * its expert count must divide evenly over the expert ranks: expert e lives
 * on rank e / L with L = num_experts / ep_world_size, so the expert-major
 * layout is already rank-major and rank r's rows are
 *   [rank_offsets[r], rank_offsets[r+1]),  rank_offsets[r] = ep_send_counts[r*L],
 * rank_offsets[ep_world_size] = the padded total.  With align = 1 the send
 * buffer carries no padding rows.
 *
 *  ep_world_size  in  1 <= ep_world_size <= num_experts, dividing num_experts.
 *  rank_offsets   out int32 [ep_world_size + 1].
 * Other arguments and outputs as for moe_dispatch_layout.
 */
int moe_dispatch_layout_ep(const int32_t* expert_ids, int32_t bs, int32_t k, int32_t num_experts,
                           int32_t ep_world_size, int32_t align, int32_t* expert_counts,
                           int32_t* ep_send_counts, int32_t* rank_offsets, int32_t* expand_idx,
                           int32_t* status, void* workspace, size_t workspace_bytes,
                           void* stream);

/*
 * Replica-aware layout: the in-graph probabilistic dispatch with count
 * gathering of the TEMPO summary (section 2, system integration), where hot
 * experts have several physical replicas and each (token, k) pair is sent to
 * one of them.  Replicas of logical expert e are the physical ids
 * [replica_offsets[e], replica_offsets[e+1]), contiguous and disjoint.  Pair
 * i = t*k + j draws u = the upper 32 bits of draw i of the SplitMix64 stream
 * seeded with `seed` (Steele, Lea and Flood, OOPSLA 2014: the state
 * seed + (i+1)*0x9E3779B97F4A7C15 through the variant-13 finaliser), and
 * goes to the first replica r of its expert with u <= replica_thresholds[r]
 * (thresholds are cumulative within an expert; the last should be
 * 0xFFFFFFFF).  Then the layout of moe_dispatch_layout runs over the
 * num_replicas physical replicas: replica_counts[r] is the token count N_r
 * gathered per replica, ep_send_counts its 128-padded exclusive prefix (so
 * replica r spans ceil(N_r/128) M-tiles), expand_idx the stable rank.
 * Dispatch and combine then take replica_ids as their expert_ids with
 * num_experts = num_replicas.
 *
 *  expert_ids          in  int32 [bs, k] logical experts in [0, num_experts).
 *  replica_offsets     in  int32 [num_experts + 1], non-decreasing, last =
 *                          num_replicas (device memory).
 *  replica_thresholds  in  uint32 [num_replicas] (device memory).
 *  num_replicas        in  1 <= num_replicas <= 512, k <= num_replicas.
 *  replica_ids         out int32 [bs, k]: chosen replica, -1 if the logical id
 *                          is out of range (MOE_FLAG_ID_RANGE) or the table
 *                          gives none (MOE_FLAG_REPLICA); such pairs are
 *                          dropped like out-of-range ids.
 *  workspace           as for moe_dispatch_layout, sized with num_replicas.
 * Other arguments as for moe_dispatch_layout.  Deterministic for a fixed seed.
 */
int moe_dispatch_layout_replicated(const int32_t* expert_ids, int32_t bs, int32_t k,
                                   int32_t num_experts, const int32_t* replica_offsets,
                                   const uint32_t* replica_thresholds, int32_t num_replicas,
                                   uint64_t seed, int32_t align, int32_t* replica_ids,
                                   int32_t* replica_counts, int32_t* ep_send_counts,
                                   int32_t* expand_idx, int32_t* status, void* workspace,
                                   size_t workspace_bytes, void* stream);

/*
 * Dispatch: scatter token rows into the expert-contiguous buffer.
 *
 * The inverse path of the combine on the npu_moe_distribute_combine page
 * (function description: combine retraces the dispatch path); expand_x is
 * that page's (max(tp,1)*A, H) input, here [capacity_rows, hidden].  With
 * out_dtype MOE_FP8_E4M3 the rows are quantised on the way, the page's
 * comm_quant_mode option for a quantised transfer (its dtype is unreadable
 * on the page; e4m3fn with per-128-channel scales is this library's
 * reading).
 *
 *  x              in  bf16 [bs, hidden], row stride x_stride (>= hidden);
 *                     base 16-byte aligned, x_stride*2 a multiple of 16.
 *  hidden         in  > 0, a multiple of 32 (page rule on H), <= 65536;
 *                     a multiple of 128 for MOE_FP8_E4M3; bs*hidden/8 < 2^31.
 *  expert_ids, expand_idx, ep_send_counts
 *                 in  the layout call's input and outputs, unchanged.
 *  expand_x       out [capacity_rows, hidden] of out_dtype, row stride
 *                     expand_x_stride (>= hidden); 16-byte aligned, stride in
 *                     bytes a multiple of 16.  Row slot(t,j) receives token t
 *                     for every pair j.  Padding rows are NOT written.
 *  capacity_rows  in  rows of expand_x (size it with moe_dispatch_capacity).
 *                     A smaller value is accepted (a caller that knows the
 *                     padded total may size the buffer to it), but a pair
 *                     whose row lies at or beyond capacity_rows is DROPPED:
 *                     its row is not written and MOE_FLAG_GUARD is set in
 *                     `status`, which such a caller must read.  With 0 rows
 *                     every pair is guarded and nothing is written; expand_x
 *                     and quant_scales may then be NULL.
 *  quant_scales   out fp32 [capacity_rows, hidden/128] row-major when
 *                     out_dtype is MOE_FP8_E4M3 (else ignored, may be NULL):
 *                     s = amax/448 over the 128 channels of the block;
 *                     the code is e4m3(x/s) rounded to nearest even and
 *                     saturated to +-448 (all-zero block: s = 0, codes 0).
 *                     Dequantise as e4m3_value * s.
 *  status         in/out int32 [1] or NULL: MOE_FLAG_GUARD is OR-ed in when a
 *                     slot falls outside [0, capacity_rows); never cleared.
 *
 * Launches: one scatter; for bf16 output, when x is contiguous (x_stride ==
 * hidden) and its rows total 32 MB to 240 MB, a launch that reads them into
 * the 256 MB Infinity Cache goes first, so that the scatter writes from
 * cache-resident rows instead of interleaving row reads from HBM with its
 * writes.
 */
int moe_dispatch(const void* x, int64_t x_stride, int32_t bs, int32_t hidden,
                 const int32_t* expert_ids, const int32_t* expand_idx,
                 const int32_t* ep_send_counts, int32_t k, int32_t num_experts, void* expand_x,
                 int64_t expand_x_stride, int64_t capacity_rows, int32_t out_dtype,
                 float* quant_scales, int32_t* status, void* stream);

/*
 * Layout and dispatch in one call: the results of moe_dispatch_layout
 * followed by moe_dispatch on the same stream, bit for bit (outputs, padding
 * rows left unwritten, e4m3 codes and scales, status bits).  For
 * decode-sized batches (bs*k <= 2048) it is a single kernel launch: every
 * scatter workgroup derives the whole layout from the ids in on-chip memory,
 * so no separate layout launch or wait precedes the scatter (the TEMPO
 * summary, section 2, folds count gathering into the dispatch kernel; here
 * the counts, offsets and ranks are folded in).  Larger batches take two
 * launches: the layout's ranking launch (its last workgroup scans the
 * histograms, as in moe_dispatch_layout), then the scatter, which adds each
 * token's workgroup prefix to the ranks and writes expand_idx itself, so no
 * finalize launch sits between them.  The ranking launch, which is latency
 * bound, also reads the token rows x ahead (ordinary loads, x contiguous:
 * all rows up to 240 MB, else the first 128 MB) so that the scatter finds
 * them in the 256 MB Infinity Cache instead of interleaving row reads from
 * HBM with its writes.  When every row was read ahead, the bf16 scatter
 * runs with fewer waves in flight (at most 7 workgroups of 64 threads per
 * compute unit), which narrows the window of destination rows being
 * written at once.
 *
 *  x, x_stride, bs, hidden                   as for moe_dispatch.
 *  expert_ids, k, num_experts, align         as for moe_dispatch_layout.
 *  expert_counts, ep_send_counts, expand_idx out, as for moe_dispatch_layout.
 *  expand_x, expand_x_stride, capacity_rows, out_dtype, quant_scales
 *                                            as for moe_dispatch.
 *  status         out int32 [1] or NULL: MOE_FLAG_ID_RANGE | MOE_FLAG_DUP_ID |
 *                     MOE_FLAG_GUARD of this call, overwritten.
 *  workspace      as for moe_dispatch_layout (unused, may be NULL, when the
 *                     single launch applies).
 */
int moe_dispatch_fused(const void* x, int64_t x_stride, int32_t bs, int32_t hidden,
                       const int32_t* expert_ids, int32_t k, int32_t num_experts, int32_t align,
                       int32_t* expert_counts, int32_t* ep_send_counts, int32_t* expand_idx,
                       void* expand_x, int64_t expand_x_stride, int64_t capacity_rows,
                       int32_t out_dtype, float* quant_scales, int32_t* status, void* workspace,
                       size_t workspace_bytes, void* stream);

/*
 * moe_dispatch_fused without a workspace argument, for callers that cannot
 * allocate device memory: code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc.  It allocates nothing; the layout's
 * workspace is a static device array of moe_noalloc_scratch_bytes() bytes
 * (5 MiB) that each GPU the library runs on holds until the process ends,
 * its address looked up once per device on the first call there.  Every
 * batch of at most 2^20 pairs fits (more with fewer experts: the rule is
 * moe_dispatch_layout_workspace_size(bs, k, num_experts) <=
 * moe_noalloc_scratch_bytes()); a larger one returns MOE_ERR_SCRATCH and
 * enqueues nothing.  All calls on one GPU share its array: calls that
 * overlap on one GPU (from other streams or threads) race and must be
 * serialised by the caller.  Arguments, outputs and results are those of
 * moe_dispatch_fused, bit for bit.
 */
int moe_dispatch_fused_noalloc(const void* x, int64_t x_stride, int32_t bs, int32_t hidden,
                               const int32_t* expert_ids, int32_t k, int32_t num_experts,
                               int32_t align, int32_t* expert_counts, int32_t* ep_send_counts,
                               int32_t* expand_idx, void* expand_x, int64_t expand_x_stride,
                               int64_t capacity_rows, int32_t out_dtype, float* quant_scales,
                               int32_t* status, void* stream);

/* Bytes of the static per-GPU scratch moe_dispatch_fused_noalloc uses. */
size_t moe_noalloc_scratch_bytes(void);

/*
 * Combine: gather each token's K expert-output rows back and form
 *   x_out[t,:] = sum_j expert_scales[t,j] * expand_x[slot(t,j), :] + shared_expert_x[t,:]
 * (the formula of the npu_moe_distribute_combine page, with the shared expert
 * added without a weight as its expert_scales parameter note states).
 *
 * Arithmetic: fp32, a fused multiply-add chain over j = 0..k-1 in order,
 * starting from +0; then the shared row is added; then one round to nearest
 * even into bf16.  Pairs with expand_idx < 0 or an out-of-range id contribute
 * nothing.
 *
 *  expand_x       in  bf16 expert outputs [capacity_rows, hidden], row stride
 *                     expand_x_stride; 16-byte aligned, stride*2 % 16 == 0.
 *  expert_ids, expand_idx, ep_send_counts
 *                 in  the same layout outputs the dispatch used.
 *  expert_scales  in  fp32 [bs, k] row-major, contiguous.
 *  shared_expert_x in bf16 [bs, hidden], row stride shared_stride, or NULL.
 *  bs, hidden     in  as for moe_dispatch (bs*hidden/8 < 2^31).
 *  x_out          out bf16 [bs, hidden], contiguous (the page requires a
 *                     contiguous output), 16-byte aligned.
 *  status         in/out int32 [1] or NULL: MOE_FLAG_GUARD is OR-ed in when a
 *                     pair's row lies at or beyond capacity_rows; that pair
 *                     contributes nothing to its token's sum.
 */
int moe_combine(const void* expand_x, int64_t expand_x_stride, int64_t capacity_rows,
                const int32_t* expert_ids, const int32_t* expand_idx,
                const int32_t* ep_send_counts, const float* expert_scales,
                const void* shared_expert_x, int64_t shared_stride, int32_t bs, int32_t hidden,
                int32_t k, int32_t num_experts, void* x_out, int32_t* status, void* stream);

/*
 * Quantised-transfer combine: the same weighted gather-sum as moe_combine,
 * with the expert outputs in the e4m3 format that moe_dispatch emits (the
 * combine page's comm_quant_mode names a quantised transfer on this path;
 * its dtype is unreadable there, and this library reads it as that format).
 *
 *   x_out[t,h] = bf16( fma-chain_j( expert_scales[t,j],
 *                         e4m3(expand_x[slot(t,j), h]) * quant_scales[slot(t,j), h/128] )
 *                      + shared_expert_x[t,h] )
 *
 * Each term is dequantised with one fp32 multiply before the fused
 * multiply-add chain over j ascending from +0; then the shared row is added
 * and the sum rounded to nearest even into bf16.
 *
 *  expand_x       in  e4m3fn codes [capacity_rows, hidden], row stride
 *                     expand_x_stride bytes (>= hidden, multiple of 16),
 *                     16-byte aligned.
 *  quant_scales   in  fp32 [capacity_rows, hidden/128] row-major.
 *  hidden         in  a multiple of 128, <= 65536, bs*hidden/8 < 2^31.
 *  other arguments as for moe_combine.
 */
int moe_combine_fp8(const void* expand_x, int64_t expand_x_stride, int64_t capacity_rows,
                    const float* quant_scales, const int32_t* expert_ids,
                    const int32_t* expand_idx, const int32_t* ep_send_counts,
                    const float* expert_scales, const void* shared_expert_x,
                    int64_t shared_stride, int32_t bs, int32_t hidden, int32_t k,
                    int32_t num_experts, void* x_out, int32_t* status, void* stream);

/*
 * The replica-aware layout and the dispatch over replicas in one call: the
 * results of moe_dispatch_layout_replicated followed by moe_dispatch with
 * expert_ids = replica_ids and num_experts = num_replicas, on the same
 * stream, bit for bit (replica ids, counts, offsets, ranks, dispatched rows,
 * padding rows left unwritten, e4m3 codes and scales, status bits).  As in
 * moe_dispatch_fused, batches of more than 2048 pairs take the ranking
 * launch, which also reads the token rows ahead into the Infinity Cache (x
 * contiguous; all rows up to 240 MB, else the first 128 MB), and the
 * scatter, which completes expand_idx; a bf16 scatter of rows that were all
 * read ahead runs with fewer waves in flight.  Batches of at most 2048
 * pairs take one layout launch and the scatter launch.
 *
 *  x, x_stride, hidden, expand_x, expand_x_stride, capacity_rows, out_dtype,
 *  quant_scales               as for moe_dispatch (over num_replicas).
 *  expert_ids, bs, k, num_experts, replica_offsets, replica_thresholds,
 *  num_replicas, seed, align, replica_ids, replica_counts, ep_send_counts,
 *  expand_idx, workspace      as for moe_dispatch_layout_replicated.
 *  status         out int32 [1] or NULL: MOE_FLAG_ID_RANGE | MOE_FLAG_DUP_ID |
 *                     MOE_FLAG_REPLICA | MOE_FLAG_GUARD of this call,
 *                     overwritten.
 * Returns the first error of the two calls' argument rules (nothing is
 * enqueued), MOE_ERR_WORKSPACE, MOE_ERR_HIP if a launch fails, else 0.
 */
int moe_dispatch_fused_replicated(const void* x, int64_t x_stride, int32_t bs, int32_t hidden,
                                  const int32_t* expert_ids, int32_t k, int32_t num_experts,
                                  const int32_t* replica_offsets,
                                  const uint32_t* replica_thresholds, int32_t num_replicas,
                                  uint64_t seed, int32_t align, int32_t* replica_ids,
                                  int32_t* replica_counts, int32_t* ep_send_counts,
                                  int32_t* expand_idx, void* expand_x, int64_t expand_x_stride,
                                  int64_t capacity_rows, int32_t out_dtype, float* quant_scales,
                                  int32_t* status, void* workspace, size_t workspace_bytes,
                                  void* stream);

/*
 * The experts' product over dispatched rows, in e4m3 with block scales: the
 * grouped GEMM that the 128-row tiles of the layout are made for (TEMPO
 * summary, section 1).  For the rows r of expert e, that is
 * ep_send_counts[e] <= r < ep_send_counts[e] + expert_counts[e]:
 *
 *   out[r, n] = bf16( sum_b quant_scales[r, b] * weight_scales[e, n/128, b]
 *                       * sum_{c in block b} expand_x[r, c] * weight[e, n, c] )
 *
 * over the 128-channel blocks b of a row, ascending (with in_features a
 * multiple of 4096, from a block that follows n/256 on, and round).
 * Products of codes are exact and the running sum is fp32 (a fused
 * multiply-add per block).  A
 * block's own sum is the e4m3 matrix instruction's: it aligns each group of
 * 8 products to the largest and keeps 13 bits below that one's leading bit,
 * then adds in fp32 (measured on N(0,1) rows: 1.3e-5 of the result, against
 * 2e-3 for its one rounding to bf16, to nearest even, at the end, so that 2 %
 * of the outputs are the bf16 value next to the nearest; where terms cancel,
 * what is lost is below 7 * 2^-13 of each group's largest product).  Rows of no expert (padding,
 * and rows behind the last segment) are neither read nor written.  The
 * result of a row does not depend on the other rows or on expected_rows.
 * Scales and codes are taken as they are: a NaN code or a non-finite scale
 * reaches every output that uses it.  The gradient of expand_x is the same
 * call with the weights transposed (128 x 128 blocks transpose with them).
 *
 *  expand_x       in  e4m3fn codes [capacity_rows, in_features], row stride
 *                     expand_x_stride bytes (>= in_features, a multiple of
 *                     16, at most 2^23), 16-byte aligned: moe_dispatch's
 *                     e4m3 output.
 *  capacity_rows  in  rows of expand_x and out, >= 0, at most 2^30 and at
 *                     most 2^40 / out_features.
 *  quant_scales   in  fp32 [capacity_rows, in_features/128] row-major.
 *  weight         in  e4m3fn codes [num_experts, out_features, in_features],
 *                     contiguous, 16-byte aligned.
 *  weight_scales  in  fp32 [num_experts, ceil(out_features/128),
 *                     in_features/128]: one per 128 x 128 block of weight.
 *  expert_counts, ep_send_counts
 *                 in  the layout's outputs (any align).  Both NULL: one
 *                     group of all capacity_rows rows (num_experts must be
 *                     1), the dense product of a shared expert.
 *  num_experts    in  1 <= num_experts <= 512.
 *  in_features    in  a positive multiple of 128, at most 65536.
 *  out_features   in  a positive multiple of 32, at most 65536.
 *  expected_rows  in  about how many rows the experts have together (BS*K of
 *                     the batch; 0: unknown, capacity_rows is taken).  It
 *                     chooses launch and tile shapes, never the result.
 *  out            out bf16 [capacity_rows, out_features], row stride
 *                     out_stride elements, 16-byte aligned, stride*2 % 16 ==
 *                     0; a buffer that overlaps an input is refused (columns
 *                     of one wider buffer, at one stride, may lie side by
 *                     side).
 *  status         in/out int32 [1] or NULL: MOE_FLAG_GUARD is OR-ed in when
 *                     a segment leaves [0, capacity_rows) (the rows outside
 *                     are skipped) or two segments share a row of the buffer
 *                     (then nothing is written).
 */
int moe_grouped_gemm_fp8(const void* expand_x, int64_t expand_x_stride, int64_t capacity_rows,
                         const float* quant_scales, const void* weight,
                         const float* weight_scales, const int32_t* expert_counts,
                         const int32_t* ep_send_counts, int32_t num_experts,
                         int32_t in_features, int32_t out_features, int64_t expected_rows,
                         void* out, int64_t out_stride, int32_t* status, void* stream);

/*
 * The experts' first product with its gated activation and the quantisation
 * for the second product in one launch.  With z the product of
 * moe_grouped_gemm_fp8 over weight rows [0, 2*inter_features), gate rows
 * first, all of its sums in full fp32 (the codes are widened to fp16 for the
 * matrix unit, since out_scales is an fp32 result) and not rounded:
 *
 *   h[r, c] = z[r, c] / (1 + exp(-z[r, c])) * z[r, inter_features + c]
 *   out_scales[r, b] = max_{c in block b} |h[r, c]| / 448
 *   out[r, c] = e4m3( h[r, c] / out_scales[r, b] ), nearest even, saturated
 *
 * (a gate below -87 may give h = 0: its factor is under 2^-125) over
 * 128-channel blocks b: the format moe_dispatch emits, so out and
 * out_scales are the next product's expand_x and quant_scales.  A block
 * whose scale is 0 has codes 0; a block that holds an infinity or a NaN has
 * that as its scale and NaN codes.
 *
 *  weight         in  e4m3fn codes [num_experts, 2*inter_features,
 *                     in_features]; weight_scales fp32 [num_experts,
 *                     2*inter_features/128, in_features/128].
 *  inter_features in  a positive multiple of 128, at most 32768.
 *  out            out e4m3fn codes [capacity_rows, inter_features], row
 *                     stride out_stride bytes, a multiple of 16; 16-byte
 *                     aligned.
 *  out_scales     out fp32 [capacity_rows, inter_features/128] row-major.
 *                     Neither output may overlap the other or an input
 *                     (quant_scales among them): such calls are refused.
 *  other arguments as for moe_grouped_gemm_fp8.
 */
int moe_grouped_gemm_silu_fp8(const void* expand_x, int64_t expand_x_stride,
                              int64_t capacity_rows, const float* quant_scales,
                              const void* weight, const float* weight_scales,
                              const int32_t* expert_counts, const int32_t* ep_send_counts,
                              int32_t num_experts, int32_t in_features, int32_t inter_features,
                              int64_t expected_rows, void* out, int64_t out_stride,
                              float* out_scales, int32_t* status, void* stream);

/*
 * Gradient of moe_combine.  With g = grad_out (dL/dx_out):
 *
 *   grad_expand_x[slot(t,j), :] = bf16( expert_scales[t,j] * g[t, :] )
 *   grad_expert_scales[t,j]     = sum_h g[t,h] * expand_x[slot(t,j), h]   (fp32)
 *
 * The gradient of shared_expert_x is g itself.  A pair that the combine
 * skipped (id out of range, expand_idx < 0, slot beyond capacity_rows) has
 * grad_expert_scales 0 and no row; rows of no pair are not written.  The
 * sums' order follows bs, k and hidden alone, so results repeat bit for bit.
 *
 *  grad_out       in  bf16 [bs, hidden], row stride grad_out_stride; 16-byte
 *                     aligned, stride*2 % 16 == 0 (as every row buffer here).
 *  expand_x       in  the combine's input (read for grad_expert_scales only;
 *                     may be NULL without it).
 *  expert_ids, expand_idx, ep_send_counts, expert_scales, bs, hidden, k,
 *  num_experts, capacity_rows
 *                 in  as for moe_combine (expert_scales is read for
 *                     grad_expand_x only).
 *  grad_expand_x  out bf16 [capacity_rows, hidden], or NULL: not wanted.  May
 *                     be expand_x itself (same address and stride): each
 *                     element is read before it is overwritten.
 *  grad_expert_scales
 *                 out fp32 [bs, k] row-major, or NULL: not wanted.  May be
 *                     expert_scales itself.  One of the two outputs must be
 *                     given (unless capacity_rows is 0).  An output that
 *                     overlaps the other or what is read, except as named
 *                     here, is refused.
 *  status         in/out int32 [1] or NULL, as for moe_combine.
 */
int moe_combine_backward(const void* grad_out, int64_t grad_out_stride, const void* expand_x,
                         int64_t expand_x_stride, int64_t capacity_rows,
                         const int32_t* expert_ids, const int32_t* expand_idx,
                         const int32_t* ep_send_counts, const float* expert_scales, int32_t bs,
                         int32_t hidden, int32_t k, int32_t num_experts, void* grad_expand_x,
                         int64_t grad_expand_x_stride, float* grad_expert_scales,
                         int32_t* status, void* stream);

/*
 * Gradient of moe_dispatch with respect to the token rows: every row a token
 * was sent to gives its gradient back, plus what reaches the token on other
 * paths (its shared expert, the residual):
 *
 *   grad_x[t, :] = bf16( sum_j grad_expand_x[slot(t,j), :] + grad_x_add[t, :] )
 *
 * in fp32 over j ascending, then grad_x_add, then one round to nearest even.
 * Dropped pairs contribute nothing; a token with none left gets grad_x_add,
 * or 0.  (e4m3 dispatch: the quantisation counts as the identity.)
 *
 *  grad_expand_x  in  bf16 [capacity_rows, hidden].
 *  grad_x_add     in  bf16 [bs, hidden], row stride grad_x_add_stride, or NULL.
 *  grad_x         out bf16 [bs, hidden], contiguous; one that overlaps an
 *                     input is refused.
 *  other arguments as for moe_combine.
 */
int moe_dispatch_backward(const void* grad_expand_x, int64_t grad_expand_x_stride,
                          int64_t capacity_rows, const int32_t* expert_ids,
                          const int32_t* expand_idx, const int32_t* ep_send_counts,
                          const void* grad_x_add, int64_t grad_x_add_stride, int32_t bs,
                          int32_t hidden, int32_t k, int32_t num_experts, void* grad_x,
                          int32_t* status, void* stream);

/*
 * The norm before a block, with the residual's addition and the rows in the
 * formats that the next products take.  Per row:
 *
 *   z = bf16( x + residual )         (x itself without residual)
 *   r = 1 / sqrt( sum_c z[c]^2 / hidden + eps )
 *   y = z * r * weight               (fp32)
 *   residual_out = z,  out = bf16( y ),
 *   scales[t, b] = max_{c in block b} |y[c]| / 448,
 *   codes[c] = e4m3( y[c] / scales[t, b] ), nearest even, saturated
 *
 * over 128-channel blocks b: the e4m3 rows of moe_grouped_gemm_silu_fp8 (a
 * shared expert's), quantised from y before its rounding to bf16.  All sums
 * are fp32.  A block whose scale is 0 has codes 0; one that holds an infinity
 * or a NaN has that as its scale and NaN codes.  A row whose sum of squares
 * leaves fp32 (values above 1e19) gives zeros, as r is then 0.
 *
 *  x, residual    in  bf16 [bs, hidden], row strides in elements; 16-byte
 *                     aligned, stride*2 % 16 == 0.  residual may be NULL.
 *  weight         in  [hidden], bf16 or fp32 (weight_dtype MOE_BF16 or
 *                     MOE_FP32), 16-byte aligned.
 *  hidden         in  a positive multiple of 32 (of 128 with codes), at most
 *                     65536; bs * hidden / 8 < 2^31.
 *  eps            in  > 0, finite.
 *  residual_out   out bf16 [bs, hidden] or NULL (it needs residual).
 *  out            out bf16 [bs, hidden] or NULL.
 *  codes, scales  out e4m3fn [bs, hidden] (row stride codes_stride bytes) and
 *                     fp32 [bs, hidden/128] row-major, or both NULL.  One of
 *                     out and codes must be given.
 * residual_out and out may each be x or residual itself (same address and
 * stride); any other overlap of an output with an input or an output is
 * refused.
 */
int moe_rms_norm(const void* x, int64_t x_stride, const void* residual, int64_t residual_stride,
                 const void* weight, int32_t weight_dtype, int32_t bs, int32_t hidden, float eps,
                 void* residual_out, int64_t residual_out_stride, void* out, int64_t out_stride,
                 void* codes, int64_t codes_stride, float* scales, void* stream);

/*
 * Gradient of moe_rms_norm.  With x the rows that were normalised (its
 * residual_out, or its x without a residual), g = grad_out * weight and r as
 * above:
 *
 *   grad_x[t]   = bf16( r * (g - x * r^2 * sum_c(g*x) / hidden) + grad_x_add[t] )
 *   grad_weight = sum_t grad_out[t] * x[t] * r        (fp32)
 *
 * grad_x is the gradient of x and of residual alike; grad_x_add is what
 * reaches residual_out on other paths.  (The e4m3 quantisation counts as the
 * identity.)  Sums are fp32 in an order that follows bs and hidden alone, so
 * results repeat bit for bit.
 *
 *  grad_x         out bf16 [bs, hidden] or NULL: not wanted.  May be
 *                     grad_out, x or grad_x_add itself (same address and
 *                     stride).
 *  grad_weight    out fp32 [hidden], 16-byte aligned, or NULL: not wanted.
 *                     With bs = 0 it becomes 0.
 *  grad_x_add     in  bf16 [bs, hidden] or NULL.
 *  workspace      16-byte aligned, moe_rms_norm_backward_workspace_size bytes
 *                     (grad_weight only); no initial contents.  Calls that
 *                     may run at the same time need one each.
 */
size_t moe_rms_norm_backward_workspace_size(int32_t bs, int32_t hidden);
int moe_rms_norm_backward(const void* grad_out, int64_t grad_out_stride, const void* x,
                          int64_t x_stride, const void* weight, int32_t weight_dtype, int32_t bs,
                          int32_t hidden, float eps, const void* grad_x_add,
                          int64_t grad_x_add_stride, void* grad_x, int64_t grad_x_stride,
                          float* grad_weight, void* workspace, size_t workspace_bytes,
                          void* stream);

/*
 * The router's product:
 *
 *   logits[t, e] = sum_h x[t, h] * weight[e, h]        (fp32)
 *
 * Products of bf16 values are exact in fp32 and so are the sums' terms; the
 * sums' order follows bs, hidden and num_experts alone, so results repeat bit
 * for bit.
 *
 *  x              in  bf16 [bs, hidden], as for moe_rms_norm.
 *  weight         in  bf16 [num_experts, hidden], contiguous, 16-byte aligned.
 *  num_experts    in  1 <= num_experts <= 512.
 *  hidden         in  a positive multiple of 32, at most 65536; bs * hidden / 8
 *                     < 2^31.
 *  logits         out fp32 [bs, num_experts], row stride logits_stride; an
 *                     overlap with an input is refused.
 *  workspace      16-byte aligned, moe_router_logits_workspace_size bytes (may
 *                     be 0); no initial contents.  Calls that may run at the
 *                     same time need one each.
 */
size_t moe_router_logits_workspace_size(int32_t bs, int32_t hidden, int32_t num_experts);
int moe_router_logits(const void* x, int64_t x_stride, const void* weight, int32_t bs,
                      int32_t hidden, int32_t num_experts, float* logits, int64_t logits_stride,
                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradient of moe_router_logits:
 *
 *   grad_x[t, h]      = bf16( sum_e grad_logits[t, e] * weight[e, h] + grad_x_add[t, h] )
 *   grad_weight[e, h] = sum_t grad_logits[t, e] * x[t, h]       (fp32)
 *
 * grad_x_add is what reaches the token on other paths (moe_dispatch_backward's
 * grad_x).  Sums are fp32.  grad_logits enter grad_weight with all of their 24
 * bits (down to 2^-133) and grad_x, which is rounded to 8 itself, with 16: a
 * term of grad_x is off by at most 2^-16 of its magnitude, also where the terms
 * cancel.  They enter in parts, so where the formula makes an infinity of one
 * in weight or x and a finite grad_logits, the result may be a NaN.
 *
 *  grad_logits    in  fp32 [bs, num_experts], row stride grad_logits_stride.
 *  x              in  as for moe_router_logits (read for grad_weight only).
 *  weight         in  likewise (read for grad_x only).
 *  grad_x_add     in  bf16 [bs, hidden] or NULL.
 *  grad_x         out bf16 [bs, hidden] or NULL: not wanted.  May be
 *                     grad_x_add itself (same address and stride).
 *  grad_weight    out fp32 [num_experts, hidden] contiguous, 16-byte aligned,
 *                     or NULL: not wanted.  With bs = 0 it becomes 0.
 *  workspace      16-byte aligned, moe_router_logits_backward_workspace_size
 *                     bytes (for grad_weight: 0 without it); no initial
 *                     contents.  Calls that may run at the same time need one
 *                     each.
 */
size_t moe_router_logits_backward_workspace_size(int32_t bs, int32_t hidden,
                                                 int32_t num_experts);
int moe_router_logits_backward(const float* grad_logits, int64_t grad_logits_stride,
                               const void* x, int64_t x_stride, const void* weight,
                               const void* grad_x_add, int64_t grad_x_add_stride, int32_t bs,
                               int32_t hidden, int32_t num_experts, void* grad_x,
                               int64_t grad_x_stride, float* grad_weight, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * Routing: each token's k experts and their weights, the expert_ids and
 * expert_scales of the calls above.  With scores
 *
 *   s[e] = exp(l[e]) / sum_f exp(l[f])   (MOE_SCORE_SOFTMAX), or
 *   s[e] = 1 / (1 + exp(-l[e]))          (MOE_SCORE_SIGMOID)
 *
 * of a row l of logits, an expert's key is l[e], or s[e] + bias[e] with a
 * bias.  Of `groups` groups of num_experts/groups neighbouring experts the
 * top_groups best stay, by their largest key (MOE_GROUP_MAX) or by the sum of
 * their two largest s[e] (+ bias[e]) (MOE_GROUP_TOP2; one alone counts as the
 * sum).  Of what stays the k largest keys are taken, in descending order,
 * equal ones by the lower index (groups too):
 *
 *   expert_scales[t, j] = scale * s[id_j]                       or, renormalize:
 *   expert_scales[t, j] = scale * s[id_j] / sum_i s[id_i]
 *
 * Keys are compared as 64-bit values, so a choice does not depend on the
 * rounding of fp32 scores.  An expert whose logit is -inf or NaN, or whose
 * bias is -inf or NaN, is never chosen (without renormalize, a softmax's sum
 * still counts an expert that only its bias excludes); +inf counts as the
 * largest finite value.  expert_scales are made in 64 bits and rounded once;
 * without renormalize a softmax divides by a sum of fp32 exponentials, off by
 * less than 2^-19 of itself.  Where fewer than k experts are left, the remaining
 * expert_ids are -1 and their expert_scales 0: pairs that every call drops.
 *
 *  logits         in  [bs, num_experts], fp32 or bf16 (logits_dtype MOE_FP32
 *                     or MOE_BF16), row stride logits_stride elements.
 *  bias           in  fp32 [num_experts] or NULL.
 *  k              in  1 <= k <= min(16, num_experts/groups * top_groups).
 *  groups         in  1 .. 64, dividing num_experts (1: no groups);
 *                     1 <= top_groups <= groups.
 *  scale          in  finite.
 *  expert_ids     out int32 [bs, k] row-major.
 *  expert_scales  out fp32 [bs, k] row-major.  Outputs that overlap an input
 *                     or each other are refused.
 */
int moe_route(const void* logits, int32_t logits_dtype, int64_t logits_stride,
              const float* bias, int32_t bs, int32_t num_experts, int32_t k, int32_t score,
              int32_t groups, int32_t top_groups, int32_t group_score, int32_t renormalize,
              float scale, int32_t* expert_ids, float* expert_scales, void* stream);

/*
 * Gradient of moe_route's expert_scales with respect to the logits (the choice
 * has none, nor has the bias), from the logits and the expert_ids it chose:
 * with g = grad_expert_scales, q = expert_scales / scale and G = sum_j g_j q_j,
 *
 *   softmax                   scale * s[e] * (sum_{j: id_j = e} g_j - G), every e
 *   softmax, renormalize      scale * q_j * (g_j - G)              at e = id_j
 *   sigmoid                   scale * s_j * (1 - s_j) * g_j        at e = id_j
 *   sigmoid, renormalize      scale * q_j * (1 - s_j) * (g_j - G)  at e = id_j
 *
 * and 0 elsewhere.  What is there at e = id_j is made in 64 bits and rounded
 * once to fp32; the first line's other terms are products of fp32 exponentials
 * (a few 2^-24 of a term beside the rounding of l[e] - max l).  Rounded to bf16
 * if the logits are.  Ids outside
 * [0, num_experts), or of an expert whose logit is -inf or NaN, count as
 * none; an id that occurs twice counts twice.
 *
 *  grad_logits    out [bs, num_experts] in the logits' type; may be logits
 *                     itself (same address and stride).
 */
int moe_route_backward(const float* grad_expert_scales, const void* logits,
                       int32_t logits_dtype, int64_t logits_stride, const int32_t* expert_ids,
                       int32_t bs, int32_t num_experts, int32_t k, int32_t score,
                       int32_t renormalize, float scale, void* grad_logits,
                       int64_t grad_logits_stride, void* stream);

/*
 * Compensation planner (host code, host pointers; no GPU involved).  The
 * DeepEP compensation PR (Python section) describes a water-filling
 * chunk-migration planner with expert-affinity batching, a makespan guard, a
 * cost-aware no-op and 128-aligned chunks; the TEMPO summary (section 2)
 * prices an expert on a device as an activation floor plus a cost per
 * 128-row M-tile.  With expert e homed on rank e / (E / ep_world_size), the
 * load of a rank is the sum over the experts it computes of
 *   activation_cost + tile_cost * ceil(rows / 128).
 * The planner repeatedly moves whole 128-row chunks of one expert from the
 * most to the least loaded rank (lowest index on ties): the move minimising
 * the pair's new maximum, ties to an expert the receiver already computes,
 * then the lower expert id, then fewer chunks; a move is admitted only if
 * the receiver stays below the current makespan; it stops when the two loads
 * differ by at most one tile, no move is admitted or max_moves are made, and
 * returns no move at all if the makespan fell by less than min_gain.
 *
 *  expert_counts   in  int32 [num_experts] (host): tokens per expert, >= 0,
 *                      e.g. the layout's expert_counts summed over ranks.
 *  ep_world_size   in  >= 1, dividing num_experts (<= 2^20).
 *  tile_cost, activation_cost, min_gain
 *                  in  integer cost units (tile_cost > 0, others >= 0).
 *  moves           out int32 [max_moves][4] (host): expert, source rank,
 *                      destination rank, rows (a multiple of 128).
 *  n_moves         out number of moves written.
 *  rank_loads      out int64 [ep_world_size] (host): loads after the plan.
 *  makespan_before, makespan_after, ideal
 *                  out (nullable): largest load before and after, and the
 *                      ideal bound ceil(sum of starting loads / ranks).
 * Returns MOE_ERR_INVALID_ARG for bad arguments; never touches the GPU.
 */
int moe_plan_compensation(const int32_t* expert_counts, int32_t num_experts,
                          int32_t ep_world_size, int64_t tile_cost, int64_t activation_cost,
                          int64_t min_gain, int32_t max_moves, int32_t* moves, int32_t* n_moves,
                          int64_t* rank_loads, int64_t* makespan_before, int64_t* makespan_after,
                          int64_t* ideal);

#ifdef __cplusplus
}
#endif

#endif /* MOE_DISPATCH_H */
