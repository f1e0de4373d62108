/*
 * pillar.h -- C ABI of the GB300 (sm_103a) PillarAttn unified step.
 *
 * The method ("SparseSpec-MLSys26", section 核心方法 / PillarAttn):
 *   - a draft request (one query token) attends only its critical-token list,
 *     one list per (request, KV head);
 *   - a verify request (k+1 query tokens, causal among themselves) attends
 *     its full context and, in the same pass, dumps the raw attention logits
 *     and the log-sum-exp of every row;
 *   - from that dump the exact softmax scores are rematerialised, averaged
 *     over the k draft rows and the GQA group's query heads, and the Top-K
 *     positions (K = ceil(s*len)) become the next stride's critical list.
 * With a page-size-1 KV pool every position reaches its K/V row through a
 * per-request slot table, so sparse and full attention share one pipeline
 * and mix freely in one batch (same page, section "Unified batch scheduler
 * + fused attention kernel").
 *
 * Conventions for every entry point:
 *   - All array pointers are DEVICE pointers owned by the caller (the
 *     phase-bucket functions at the end work on host memory).  The library
 *     allocates nothing and keeps no state between calls, except the launch
 *     attributes it sets once per device context (up to 64 devices) and the
 *     scratch array of pillar_topk_select_noalloc.  Scratch lives in the
 *     caller's workspace (sized by the *_workspace_bytes functions); the
 *     device error word sits inside that workspace.
 *   - bf16 tensors are passed as uint16_t bit patterns.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Calls are
 *     asynchronous on that stream: a return of PILLAR_OK means the work was
 *     validated and enqueued.  Data-dependent problems found on the device
 *     (an index or slot out of range, a bad mode or length) are skipped and
 *     recorded in the error word; read it with pillar_get_error.
 *   - Nothing on the device waits without a bound: a wait that runs past
 *     its bound (one second, or the shape's wait_timeout_us) records
 *     PILLAR_FLAG_TIMEOUT and the kernel returns.  The device error word
 *     of the workspace is cleared by every call and reports that call only.
 */
#ifndef PILLAR_H
#define PILLAR_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PILLAR_API __attribute__((visibility("default")))
#else
#define PILLAR_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
#define PILLAR_OK 0
#define PILLAR_ERR_ARG (-1)         /* null pointer, bad dimension or unsupported shape */
#define PILLAR_ERR_WORKSPACE (-2)   /* workspace null, misaligned or too small */
#define PILLAR_ERR_CUDA (-3)        /* a CUDA runtime call or launch failed */
#define PILLAR_ERR_DEVICE (-4)      /* pillar_get_error: the device error word is non-zero */
#define PILLAR_ERR_SCRATCH (-5)     /* pillar_topk_select_noalloc: the shape needs more than its built-in scratch */

/* Size of the scratch array compiled into the library for
 * pillar_topk_select_noalloc (16 MiB of scores plus a 256-byte header). */
#define PILLAR_NOALLOC_SCRATCH_BYTES (16u * 1024u * 1024u + 256u)

/* Bits of the device error word. */
#define PILLAR_FLAG_INDEX 1         /* a critical-list position outside [0, L_b) was skipped */
#define PILLAR_FLAG_SLOT 2          /* a slot outside [0, num_slots) was skipped */
#define PILLAR_FLAG_REQUEST 4       /* req_mode not 0/1, L_b < 0, L_b > max_len, or verify L_b < k+1 */
#define PILLAR_FLAG_COUNT 8         /* sparse_cnt outside [0, max_sparse] (clamped) */
#define PILLAR_FLAG_TIMEOUT 16      /* a bounded device wait gave up; outputs are incomplete */
#define PILLAR_FLAG_TOPK 32         /* a Top-K budget exceeded max_topk (clamped) */
#define PILLAR_FLAG_BLOCK 64        /* pillar_block_map: too few free blocks, or a bad free-ring state */
#define PILLAR_FLAG_VALUE 128       /* pillar_kv8_append, pillar_kv4_append: a NaN, infinity or bad scale; 4 bits: past 61440 */

typedef struct pillar_shape {
    int32_t B;             /* requests in the batch (>= 0) */
    int32_t Hq;            /* query heads */
    int32_t Hkv;           /* KV heads; G = Hq / Hkv query heads share one (1 <= G <= 8) */
    int32_t D;             /* head dimension: 64 or 128 */
    int32_t k;             /* stride: a verify request carries k+1 query rows; (k+1)*G <= 64 */
    int32_t max_sparse;    /* row stride of sparse_idx (>= 0) */
    int32_t max_len;       /* upper bound on every req_len; sizes the workspace (>= 1) */
    int32_t row_lo;        /* verify rows [row_lo, row_hi) are averaged by Top-K; */
    int32_t row_hi;        /*   the k draft rows are [1, k+1) */
    int32_t max_topk;      /* row stride of next_idx (>= 1) */
    int32_t verify_chunk;  /* keys per verify work item (multiple of 64, <= 2048); 0: 1024 for
                              contexts under 8192 positions, 2048 from 8192 on
                              (pillar_attn_kv4 may choose another: see there) */
    int32_t draft_chunk;   /* listed keys per draft work item (multiple of 64, <= 2048; 0 = 2048) */
    int64_t num_slots;     /* rows of k_pool / v_pool */
    float sm_scale;        /* logit scale; 0 means 1/sqrt(D) */
    int32_t schedule;      /* PILLAR_SCHEDULE_* (0: the unified pass) */
    int32_t wait_timeout_us; /* bound on every pipeline wait of pillar_attn_unified, in
                              microseconds (>= 0; 0 means 1000000, one second); a wait that
                              runs past it records PILLAR_FLAG_TIMEOUT and the kernel
                              returns with incomplete outputs.  The waits that let copies
                              and tensor-core work already in flight finish before a CTA
                              exits keep their own one-second bound. */
    int32_t reserved;      /* set to 0 */
} pillar_shape_t;

/*
 * Schedules of pillar_attn_unified.  The unified pass is the method's design
 * ("SparseSpec-MLSys26", Unified batch scheduler + fused attention kernel:
 * one persistent kernel serves draft and verify requests of one batch).  The
 * other schedules exist to measure it against the two alternatives that
 * section compares it with; all of them compute the same outputs.
 *   UNIFIED       draft and verify requests in one persistent pass.
 *   DRAFT_ONLY    the draft requests only; the outputs of verify requests
 *                 (their out rows, logits and LSEs) are left untouched.
 *   VERIFY_ONLY   the verify requests only; draft outputs left untouched.  A
 *                 DRAFT_ONLY call followed by a VERIFY_ONLY call on the same
 *                 buffers is the sequential two-kernel schedule; it writes
 *                 the same values as one UNIFIED call.
 *   UNIFORM_ROWS  one pass in which a draft item takes the verify item's row
 *                 layout (its G rows as the first G of the (k+1)*G row slots,
 *                 the slots of one TMEM lane quadrant) instead of its own
 *                 spread of the G rows over the four quadrants: a joint batch
 *                 without per-mode dispatch.
 *   NAIVE_JOINT   the naive joint batch: the UNIFORM_ROWS row layout for every
 *                 request, work items of the largest size the pipeline takes
 *                 (2048 keys, whatever verify_chunk and draft_chunk say), and
 *                 no dynamic load balancing -- each CTA of the persistent grid
 *                 takes the (request, KV head) units c, c + grid, c + 2 grid,
 *                 ... in batch order and works through all of their items.
 * The device error word is cleared by every call; it reports that call only.
 */
#define PILLAR_SCHEDULE_UNIFIED 0
#define PILLAR_SCHEDULE_DRAFT_ONLY 1
#define PILLAR_SCHEDULE_VERIFY_ONLY 2
#define PILLAR_SCHEDULE_UNIFORM_ROWS 3
#define PILLAR_SCHEDULE_NAIVE_JOINT 4

/*
 * pillar_attn_workspace_bytes -- bytes of workspace pillar_attn_unified
 * needs for this shape (a bound over every batch with req_len <= max_len and
 * sparse_cnt <= max_sparse).  Returns PILLAR_OK or PILLAR_ERR_ARG (a bad
 * shape, or one whose workspace bound would pass 2^50 bytes).
 */
PILLAR_API int pillar_attn_workspace_bytes(const pillar_shape_t *shape, size_t *bytes);

/*
 * pillar_attn_unified -- one unified draft/verify attention step.
 * ("SparseSpec-MLSys26", 核心方法 / PillarAttn: sparse draft attention over
 * the critical set, full verify attention with the logits/LSE dump; and the
 * unified-batch section: page size 1, one fused pass over mixed requests.)
 *
 *   q            [T_q, Hq, D] bf16.  Requests packed in batch order: one row
 *                for a draft request, k+1 rows for a verify request.
 *   k_pool,
 *   v_pool       [num_slots, Hkv, D] bf16: one slot = one token, all heads.
 *   slot_table   int32; request b's L_b slots start at sum_{b'<b} L_b'.
 *                slot_table[off_b + t] is the slot of position t.
 *   req_mode     [B] int32: 0 draft, 1 verify.
 *   req_len      [B] int32: L_b, the context length including the request's
 *                own new tokens.  Verify row j (0..k) sits at position
 *                L_b-(k+1)+j and attends positions [0, L_b-(k+1)+j].
 *   sparse_idx   [B, Hkv, max_sparse] int32 logical positions (draft only);
 *   sparse_cnt   [B, Hkv] int32 list lengths.  Query head h uses KV head
 *                h / G and that head's list, taken literally (a repeated
 *                position counts twice).  An empty list gives a zero output.
 *   out          [T_q, Hq, D] bf16: attention output of every query row.
 *   verify_logits  fp32, packed over the verify requests in batch order:
 *                [V][Hq][k+1][L_v], the scaled logits q.k*scale, -inf where
 *                the row may not look (t beyond its causal limit).
 *   verify_lse   [V][Hq][k+1] fp32: natural-log LSE of each verify row.
 *   workspace    device scratch of at least pillar_attn_workspace_bytes,
 *                256-byte aligned.  Must not be shared by concurrent calls.
 * All pointers are device memory.  Alignment: q, k_pool and v_pool 16 bytes,
 * verify_logits 8 bytes (pairs of logits are stored together), out and the
 * int32 and fp32 arrays 4 bytes; a misaligned pointer is PILLAR_ERR_ARG.
 *
 * Returns PILLAR_OK, PILLAR_ERR_ARG, PILLAR_ERR_WORKSPACE or PILLAR_ERR_CUDA.
 * With B == 0 nothing is launched.
 */
PILLAR_API int pillar_attn_unified(const pillar_shape_t *shape, const uint16_t *q, const uint16_t *k_pool,
                        const uint16_t *v_pool, const int32_t *slot_table, const int32_t *req_mode,
                        const int32_t *req_len, const int32_t *sparse_idx, const int32_t *sparse_cnt,
                        uint16_t *out, float *verify_logits, float *verify_lse, void *workspace,
                        size_t ws_bytes, void *stream);

/*
 * pillar_attn_unified_slotted -- pillar_attn_unified whose draft lists come
 * with their pool slots already translated (as pillar_draft_lists writes
 * them), so that a draft key's K/V rows are reached without the dependent
 * slot-table load ("SparseSpec-MLSys26", Unified batch scheduler + fused
 * attention kernel: page size 1 -- every listed position is one slot).
 *
 *   sparse_slot  [B, Hkv, max_sparse] int32, device memory, 4-byte aligned,
 *                or NULL (then exactly pillar_attn_unified): entry i of
 *                request b's list of KV head h is the slot of position
 *                sparse_idx[b, h, i], i.e. slot_table[off_b + that position].
 *                The positions are still read: one outside [0, L_b) is
 *                skipped and flagged (PILLAR_FLAG_INDEX), and a slot outside
 *                [0, num_slots) is skipped and flagged (PILLAR_FLAG_SLOT).
 *                Verify requests use slot_table as before.
 * All other arguments, results and return codes as pillar_attn_unified.
 */
PILLAR_API int pillar_attn_unified_slotted(const pillar_shape_t *shape, const uint16_t *q, const uint16_t *k_pool,
                                           const uint16_t *v_pool, const int32_t *slot_table,
                                           const int32_t *req_mode, const int32_t *req_len,
                                           const int32_t *sparse_idx, const int32_t *sparse_cnt,
                                           const int32_t *sparse_slot, uint16_t *out, float *verify_logits,
                                           float *verify_lse, void *workspace, size_t ws_bytes, void *stream);

/*
 * pillar_attn_plan + pillar_attn_run -- pillar_attn_unified in two calls, so
 * that one plan serves several runs.  The plan depends only on the batch
 * description (req_mode, req_len, sparse_cnt), which is the same for every
 * layer of a model step; the runs take what differs per layer (q, the pools,
 * the lists, the outputs).  pillar_attn_unified(_slotted) is exactly a plan
 * followed by a run.
 *
 * pillar_attn_plan(shape, req_mode, req_len, sparse_cnt, workspace, ...)
 *   launches the device planner: it clears the workspace's error word and
 *   writes the offsets, work items and partial-record layout into the
 *   workspace.  Arguments as in pillar_attn_unified; with B == 0 it only
 *   clears the error word.
 * pillar_attn_run(shape, q, k_pool, v_pool, slot_table, sparse_idx,
 *                 sparse_slot, out, verify_logits, verify_lse, workspace, ...)
 *   launches the attention kernel and the merge of split units on the plan in
 *   the workspace; sparse_slot may be NULL (as pillar_attn_unified_slotted).
 *   The shape must be the one the plan was made with, the inputs must have the
 *   plan's batch description (the same modes, lengths and list counts), and the
 *   plan must precede the run on the stream (or be complete).  Any number of
 *   runs may follow one plan, one after the other on a stream; the error word
 *   collects the flags of the plan and of every run until pillar_get_error
 *   reads and clears it.
 * Return codes as pillar_attn_unified; a run with B == 0 does nothing.
 */
PILLAR_API int pillar_attn_plan(const pillar_shape_t *shape, const int32_t *req_mode, const int32_t *req_len,
                                const int32_t *sparse_cnt, void *workspace, size_t ws_bytes, void *stream);
PILLAR_API int pillar_attn_run(const pillar_shape_t *shape, const uint16_t *q, const uint16_t *k_pool,
                               const uint16_t *v_pool, const int32_t *slot_table, const int32_t *sparse_idx,
                               const int32_t *sparse_slot, uint16_t *out, float *verify_logits, float *verify_lse,
                               void *workspace, size_t ws_bytes, void *stream);

/*
 * pillar_topk_workspace_bytes -- workspace of pillar_topk_select for V
 * verify requests of length <= max_len.  Returns PILLAR_OK or PILLAR_ERR_ARG
 * (a bad shape, V < 0, or V * Hkv * max_len fp32 scores past 2^50 bytes).
 */
PILLAR_API int pillar_topk_workspace_bytes(const pillar_shape_t *shape, int32_t V, size_t *bytes);

/*
 * pillar_topk_select -- the next stride's critical lists from one verify
 * pass ("SparseSpec-MLSys26", 核心方法 / PillarAttn: rematerialise exact
 * scores from the dumped logits and LSE, average over the k draft rows and
 * the GQA group's heads, take Top-K).
 *
 *   V              number of verify requests (host value).
 *   verify_logits,
 *   verify_lse     as written by pillar_attn_unified.
 *   req_len        [B] int32, as given to pillar_attn_unified.
 *   group_map      [V] int32: batch index b of the v-th verify request, in
 *                  increasing order (it fixes L_v and the logits offsets).
 *                  A request whose entry lies outside [0, B), or whose
 *                  length is negative or above max_len, is skipped
 *                  (next_cnt 0) and flagged PILLAR_FLAG_REQUEST; it counts
 *                  as length 0 in the offsets of the requests after it.
 *   K              [V] int32: K_v, the number of positions to keep; clamped
 *                  to [0, L_v], and to max_topk with PILLAR_FLAG_TOPK.
 *   next_idx       [V, Hkv, max_topk] int32: the selected positions of KV
 *                  head g, ascending; entries past next_cnt are untouched.
 *   next_cnt       [V, Hkv] int32: number of selected positions.
 * For KV head g and position t in [0, L_v):
 *   score[t] = 1/((row_hi-row_lo)*G) * sum_{r in [row_lo,row_hi)}
 *              sum_{h in group g} exp(logit[h][r][t] - lse[h][r])
 * (masked logits contribute 0, and so does a row that saw no position,
 * whose LSE is -inf).  The K_v largest scores are kept, equal scores taken
 * lowest position first.  Scores are formed in fp32.
 */
PILLAR_API int pillar_topk_select(const pillar_shape_t *shape, int32_t V, const float *verify_logits,
                       const float *verify_lse, const int32_t *req_len, const int32_t *group_map,
                       const int32_t *K, int32_t *next_idx, int32_t *next_cnt, void *workspace,
                       size_t ws_bytes, void *stream);

/*
 * pillar_topk_select_noalloc -- pillar_topk_select without a workspace.
 * (The paper has no counterpart: this is a convenience of this library.)
 *
 * For callers that cannot allocate device memory themselves -- their HBM is
 * owned by another allocator (a framework's caching allocator, an inference
 * server that reserves the whole budget up front), or they sit on a
 * latency-critical path where cudaMalloc's implicit device synchronisation
 * is not acceptable.  It computes exactly what pillar_topk_select computes,
 * with the same kernels; its scratch (error word and fp32 score rows) is one
 * array of PILLAR_NOALLOC_SCRATCH_BYTES compiled into the library, which
 * every GPU that loads the library holds until the process exits.  Nothing
 * is allocated or freed by this call.
 *
 *   arguments 1-9   as for pillar_topk_select (inputs and outputs, caller-owned
 *                   device memory);
 *   device_flags    NULL or a device int32 that receives the call's device
 *                   error word (PILLAR_FLAG_* bits) when the call completes.
 *
 * Returns PILLAR_ERR_SCRATCH, with nothing enqueued, when the shape needs
 * more scratch than the array holds (pillar_topk_workspace_bytes(shape, V)
 * > PILLAR_NOALLOC_SCRATCH_BYTES, about V * Hkv * max_len > 4M scores);
 * otherwise as pillar_topk_select.
 *
 * The first call in a device's context looks up the array's device address
 * (once per device context, with that device current: a context created
 * anew, after cudaDeviceReset for instance, gets a lookup of its own); make
 * that first call before any stream capture.  Every call shares the one array: calls whose work overlaps on
 * the GPU (different streams, or different host threads on one device) race
 * on it and must be serialised by the caller.  Each call clears the error
 * word itself; the score rows are fully rewritten before they are read.
 */
PILLAR_API int pillar_topk_select_noalloc(const pillar_shape_t *shape, int32_t V, const float *verify_logits,
                                          const float *verify_lse, const int32_t *req_len,
                                          const int32_t *group_map, const int32_t *K, int32_t *next_idx,
                                          int32_t *next_cnt, int32_t *device_flags, void *stream);

/*
 * pillar_draft_lists -- the critical lists of a draft step that follows a
 * verify step ("SparseSpec-MLSys26", 核心方法 / PillarAttn: the Top-K of the
 * verify step is the critical set of the next k draft steps; the tokens
 * appended since the verify step are attended as well).
 *
 * For verify request v of the earlier step, b = group_map[v] is its row in
 * the draft step's batch and p = req_len[b] - verify_len[v] the tokens it has
 * appended since; for every KV head h the kernel writes
 *   sparse_idx[b, h, :] = next_idx[v, h, :next_cnt[v, h]],
 *                         then verify_len[v], ..., verify_len[v] + p - 1
 *   sparse_cnt[b, h]    = next_cnt[v, h] + p
 * (ascending: the Top-K positions all lie below verify_len[v]), and with
 * sparse_slot non-NULL, sparse_slot[b, h, i] = slot_table[off_b + that
 * position], off_b = sum over b' < b of max(req_len[b'], 0), for
 * pillar_attn_unified_slotted.  Rows of other requests are left untouched.
 *
 *   V              number of verify requests (host value).
 *   next_idx,
 *   next_cnt       [V, Hkv, max_topk], [V, Hkv] int32 as pillar_topk_select
 *                  wrote them (shape->max_topk is the row stride).
 *   group_map      [V] int32: batch index of request v in the draft step.
 *   verify_len     [V] int32: request v's length at its verify step.
 *   req_len        [B] int32: the draft step's lengths (shape->B requests).
 *   slot_table     the draft step's slot table (needed with sparse_slot).
 *   sparse_idx,
 *   sparse_cnt,
 *   sparse_slot    the draft step's lists: [B, Hkv, max_sparse] (stride
 *                  shape->max_sparse), [B, Hkv], [B, Hkv, max_sparse] or NULL.
 *   device_flags   NULL or a device int32 the kernel OR-s flags into:
 *                  PILLAR_FLAG_REQUEST for a group_map entry outside [0, B)
 *                  or a length that shrank since the verify step (no list is
 *                  written; sparse_cnt 0 for the latter), PILLAR_FLAG_COUNT
 *                  for a list longer than max_sparse (cut to max_sparse) or a
 *                  next_cnt outside [0, max_topk] (clamped), PILLAR_FLAG_INDEX
 *                  / PILLAR_FLAG_SLOT for a position or slot out of range
 *                  (slot -1 written).
 * All arrays are device memory, 4-byte aligned.  Asynchronous on `stream`;
 * allocates nothing.  Returns PILLAR_OK, PILLAR_ERR_ARG or PILLAR_ERR_CUDA.
 */
PILLAR_API int pillar_draft_lists(const pillar_shape_t *shape, int32_t V, const int32_t *next_idx,
                                  const int32_t *next_cnt, const int32_t *group_map, const int32_t *verify_len,
                                  const int32_t *req_len, const int32_t *slot_table, int32_t *sparse_idx,
                                  int32_t *sparse_cnt, int32_t *sparse_slot, int32_t *device_flags, void *stream);

/*
 * pillar_get_error -- synchronises `stream`, then copies the device error
 * word of a workspace (either entry point's) into *flags and clears it.
 * Returns PILLAR_OK if it was zero, PILLAR_ERR_DEVICE if not,
 * PILLAR_ERR_ARG / PILLAR_ERR_CUDA on failure.
 */
PILLAR_API int pillar_get_error(void *workspace, void *stream, int32_t *flags);

/* pillar_status_string -- a static English description of a return code. */
PILLAR_API const char *pillar_status_string(int status);

/*
 * pillar_kv_append -- writes n new tokens' K and V rows into their page-size-1
 * slots (the step before the unified pass: the token a draft step appends or
 * the k+1 tokens of a verify step go to whatever slots the caller's allocator
 * handed out; "SparseSpec-MLSys26", Unified batch scheduler + fused attention
 * kernel: page size 1):
 *   k_pool[slots[i], h, :] = k_new[i, h, :],  v_pool[slots[i], h, :] = v_new[i, h, :]
 * for i < n and h < Hkv.  Only shape->Hkv, D and num_slots are used.
 *   k_new, v_new   [n, Hkv, D] bf16, device memory, 16-byte aligned
 *   slots          [n] int32, device memory; distinct (for a repeated slot one
 *                  of the writes wins)
 *   k_pool, v_pool [num_slots, Hkv, D] bf16, device memory, 16-byte aligned
 *   device_flags   device int32 or null: PILLAR_FLAG_SLOT is or-ed into it
 *                  when a slot lies outside [0, num_slots); that token is
 *                  skipped and no other row is touched
 * Asynchronous on `stream`; allocates nothing.  Returns PILLAR_OK,
 * PILLAR_ERR_ARG (bad shape, n < 0, a null or misaligned pointer) or
 * PILLAR_ERR_CUDA.
 */
PILLAR_API int pillar_kv_append(const pillar_shape_t *shape, const uint16_t *k_new, const uint16_t *v_new,
                                const int32_t *slots, int32_t n, uint16_t *k_pool, uint16_t *v_pool,
                                int32_t *device_flags, void *stream);

/*
 * Phase buckets of the unified batch (host side; "SparseSpec-MLSys26",
 * Unified batch scheduler + fused attention kernel, load balancing).  Every
 * request runs a cycle of k+1 steps: k draft steps (phases 1..k), then one
 * verify step (phase 0).  A request in bucket c is in phase (c + t) mod (k+1)
 * at step t, so the requests of one bucket verify together.  A new request
 * joins the bucket with the fewest requests (ties to the lowest index), which
 * keeps the verify requests of a step near B/(k+1) and the step's query rows
 * near (2k+1)/(k+1)*B instead of alternating between B and (k+1)*B.
 *
 * The state is a plain caller-owned struct; nothing is allocated and no GPU
 * is touched.  Every function returns PILLAR_OK or PILLAR_ERR_ARG (a null
 * pointer, k outside [0, PILLAR_MAX_BUCKETS - 1], a bucket outside
 * [0, k], retiring from an empty bucket, n < 0) and changes nothing on error.
 */
#define PILLAR_MAX_BUCKETS 64
typedef struct pillar_buckets {
    int32_t nbuckets;                    /* k + 1 */
    int32_t count[PILLAR_MAX_BUCKETS];   /* requests in each bucket */
} pillar_buckets_t;

/* pillar_buckets_init -- k+1 empty buckets. */
PILLAR_API int pillar_buckets_init(pillar_buckets_t *pb, int32_t k);

/* pillar_buckets_admit -- places a new request: *bucket gets the least
 * loaded bucket (the lowest index among equals), whose count grows by one. */
PILLAR_API int pillar_buckets_admit(pillar_buckets_t *pb, int32_t *bucket);

/* pillar_buckets_retire -- a request of `bucket` has finished. */
PILLAR_API int pillar_buckets_retire(pillar_buckets_t *pb, int32_t bucket);

/*
 * pillar_buckets_step -- the inputs of step `step` for n requests whose
 * buckets are bucket[0..n): req_mode[i] = 1 (verify) when the request's phase
 * is 0, else 0 (draft), and phase[i] in [0, k] (either output may be null).
 * *q_rows (nullable) gets the step's query rows, k+1 per verify request and
 * one per draft request (the T_q of pillar_attn_unified).  All pointers are
 * host memory.
 */
PILLAR_API int pillar_buckets_step(const pillar_buckets_t *pb, const int32_t *bucket, int32_t n, int64_t step,
                                   int32_t *req_mode, int32_t *phase, int64_t *q_rows);

/*
 * Host offload of KV ("SparseSpec-MLSys26", 动态 KV 管理 / the dynamic KV
 * manager: when device memory runs short, requests' KV goes to host memory
 * chunk by chunk, asynchronously, first in first out; requests that were
 * offloaded are scheduled again, ahead of new ones, as soon as device memory
 * is free).  Two parts: the copies of slot blocks between the page-size-1
 * pools and packed rows in host memory (device kernels), and the FIFO of
 * offloaded chunks (plain host code, caller-owned state).
 */

/*
 * pillar_kv_offload -- packs n slot blocks of the pools into rows of host
 * memory:
 *   host_k[i, h, :] = k_pool[slots[i], h, :],  host_v[i, h, :] = v_pool[slots[i], h, :]
 * for i < n and h < Hkv.  Only shape->Hkv, D and num_slots are used.
 *   k_pool, v_pool [num_slots, Hkv, D] bf16, device memory, 16-byte aligned
 *   slots          [n] int32, device memory (the slots of a request's chunk of
 *                  positions, in position order)
 *   host_k, host_v [n, Hkv, D] bf16, 16-byte aligned, page-locked host memory
 *                  (cudaHostAlloc / cudaMallocHost / cudaHostRegister; the
 *                  kernel writes it through its device mapping, over
 *                  NVLink-C2C on a Grace-Blackwell node) or device memory
 *   device_flags   device int32 or null: PILLAR_FLAG_SLOT is or-ed into it
 *                  for a slot outside [0, num_slots); that row is not written
 * Asynchronous on `stream` (the host rows are complete once the stream has
 * reached the call); allocates nothing.  Returns PILLAR_OK, PILLAR_ERR_ARG
 * (bad shape, n < 0, a null or misaligned pointer, or a host buffer the
 * device cannot address: pageable host memory is refused) or PILLAR_ERR_CUDA.
 */
PILLAR_API int pillar_kv_offload(const pillar_shape_t *shape, const uint16_t *k_pool, const uint16_t *v_pool,
                                 const int32_t *slots, int32_t n, uint16_t *host_k, uint16_t *host_v,
                                 int32_t *device_flags, void *stream);

/*
 * pillar_kv_reload -- the way back: the packed rows go to (new) slots,
 *   k_pool[slots[i], h, :] = host_k[i, h, :],  v_pool[slots[i], h, :] = host_v[i, h, :]
 * with the buffers, alignment, flags and status codes of pillar_kv_offload
 * (host_k and host_v are read, the pools written).  It is pillar_kv_append
 * with its new rows in host memory.
 */
PILLAR_API int pillar_kv_reload(const pillar_shape_t *shape, const uint16_t *host_k, const uint16_t *host_v,
                                const int32_t *slots, int32_t n, uint16_t *k_pool, uint16_t *v_pool,
                                int32_t *device_flags, void *stream);

/*
 * The FIFO of offloaded chunks.  The state counts the device slots held by
 * resident requests against a capacity, and queues the chunks of offloaded
 * requests (a request's positions [0, len) in chunks of `chunk` positions,
 * the last one possibly shorter) in the order they were offloaded.  A
 * request comes back whole: pillar_offload_reload pops the chunks of the
 * oldest offloaded requests while they fit in the free capacity, so a request
 * offloaded earlier is always reloaded earlier, and a request never runs
 * with part of its KV on the host.  Which request to offload is the caller's
 * choice (the pages leave it open).  Every function returns PILLAR_OK or
 * PILLAR_ERR_ARG (a null pointer or out-of-range argument) and changes
 * nothing on error.  Nothing is allocated and no GPU is touched.
 */
#define PILLAR_OFFLOAD_QUEUE 1024
typedef struct pillar_offload_chunk {
    int32_t req;    /* the caller's request id */
    int32_t first;  /* first position of the chunk */
    int32_t n;      /* positions in the chunk (chunk, or fewer for the request's last) */
    int32_t last;   /* 1 on the request's last chunk */
} pillar_offload_chunk_t;
typedef struct pillar_offload_fifo {
    int64_t capacity;  /* device slots available to requests' KV */
    int64_t resident;  /* slots held by resident requests */
    int32_t chunk;     /* positions per chunk (>= 1) */
    int32_t head;      /* queue index of the oldest chunk */
    int32_t count;     /* chunks queued */
    int32_t pad;
    pillar_offload_chunk_t q[PILLAR_OFFLOAD_QUEUE];
} pillar_offload_fifo_t;

/* pillar_offload_init -- no request resident, nothing queued. */
PILLAR_API int pillar_offload_init(pillar_offload_fifo_t *f, int64_t capacity, int32_t chunk);

/*
 * pillar_offload_reserve -- asks for n more device slots (a new request's KV,
 * or the tokens a running request appends).  *granted = 1 and the slots are
 * counted as resident if they fit; *granted = 0 otherwise, and also, for a
 * new request (new_request != 0), while offloaded requests wait: they are
 * brought back first.
 */
PILLAR_API int pillar_offload_reserve(pillar_offload_fifo_t *f, int64_t n, int32_t new_request, int32_t *granted);

/* pillar_offload_release -- a resident request finished: its n slots are free. */
PILLAR_API int pillar_offload_release(pillar_offload_fifo_t *f, int64_t n);

/*
 * pillar_offload_evict -- request `req` with len resident positions goes to
 * the host: its chunks join the queue (*nchunks of them, nullable) and its
 * slots stop counting as resident.  The caller copies each chunk's slot blocks
 * with pillar_kv_offload before it hands those slots out again.  Refused
 * (PILLAR_ERR_ARG) when the queue has no room for the chunks or len exceeds
 * the resident count.
 */
PILLAR_API int pillar_offload_evict(pillar_offload_fifo_t *f, int32_t req, int32_t len, int32_t *nchunks);

/*
 * pillar_offload_reload -- the chunks to bring back now: those of the oldest
 * offloaded requests, whole requests only, while their positions fit in the
 * free capacity and their chunks in out[0, max_out).  They leave the queue and
 * count as resident; *nout gets the number of chunks written (0: nothing fits
 * yet).  The caller allocates slots for them and copies with pillar_kv_reload.
 */
PILLAR_API int pillar_offload_reload(pillar_offload_fifo_t *f, pillar_offload_chunk_t *out, int32_t max_out,
                                     int32_t *nout);

/*
 * Cache blocks.  The operators below keep a request's context in blocks of
 * PILLAR_KV_BLOCK tokens: block_table[b, i] (int32, [B, max_blocks]) is the
 * block that holds positions [16 i, 16 i + 16) of request b, and position t
 * lives in slot block_table[b, t / 16] * 16 + t % 16 of a pool of
 * num_slots / 16 blocks (num_slots a multiple of 16).  Such slots are ordinary
 * page-size-1 slots: the slot table that pillar_block_map writes serves
 * pillar_attn_unified and its new slots serve pillar_kv_append.
 */
#define PILLAR_KV_BLOCK 16

/* pillar_block_map_workspace_bytes -- workspace of pillar_block_map for a
 * batch of shape->B requests. */
PILLAR_API int pillar_block_map_workspace_bytes(const pillar_shape_t *shape, size_t *bytes);

/*
 * pillar_block_map -- the block tables of a batch whose lengths change, and
 * the maps the other calls take, made on the device (no copy to the host
 * between a model step and the next one's tables).
 *
 * Request b goes from prev_len[b] to req_len[b] positions.  With
 * n = ceil(req_len / 16) and m = ceil(prev_len / 16) it takes n - m blocks
 * from the free ring when n > m, and gives its blocks n .. m-1 back when
 * n < m (a rollback of rejected tokens; req_len 0: the request is finished).
 * Blocks are taken in batch order from the ring's head and given back, in
 * batch order, at its tail, so the result does not depend on timing.  When
 * the ring runs short, the first request whose blocks do not fit and every
 * later one that needs blocks keep prev_len (PILLAR_FLAG_BLOCK); the others
 * are served.  When the blocks given back and those in the ring before the
 * call are more than the pool has (the tables and the ring disagree), none is
 * given back (PILLAR_FLAG_BLOCK): those blocks belong to nobody any more.
 *
 *   req_len,
 *   prev_len     [B] int32, in [0, max_len].  A bad req_len leaves the request
 *                at prev_len, a bad prev_len counts as an empty request of
 *                length 0 (PILLAR_FLAG_REQUEST).
 *   block_table  [B, max_blocks] int32: entries [0, m) are read, entries
 *                [m, n) written, all others left as they were.
 *   free_ring    [num_slots / 16] int32: the free blocks, from index head on,
 *                count of them, modulo the ring's size.
 *   free_state   [2] int32: {head, count}, read and updated.
 *   granted_len  [B] int32: the length each request has after the call.
 *   kv_off       [B+1] int64: exclusive prefix sums of granted_len.
 *   slot_table   int32: slot_table[kv_off[b] + t] is the slot of position t of
 *                request b (the slot table of pillar_attn_unified with
 *                req_len = granted_len).  Entries at or past kv_off[B] are left
 *                as they were, and so are entries at or past slot_capacity
 *                (PILLAR_FLAG_COUNT).
 *   new_off      [B+1] int32: exclusive prefix sums of the new tokens,
 *                max(granted_len - prev_len, 0).
 *   new_slots    int32: new_slots[new_off[b] + i] is the slot of position
 *                prev_len[b] + i (the slots of pillar_kv_append);
 *                new_capacity entries, as slot_capacity.
 *   workspace    pillar_block_map_workspace_bytes bytes, 256-byte aligned; its
 *                error word is cleared by the call and read with
 *                pillar_get_error.  A block outside [0, num_slots / 16) gives
 *                slot -1 (PILLAR_FLAG_SLOT).
 * Only shape->B, max_len and num_slots are used (the whole shape is checked).
 * All arrays are device memory, 4-byte aligned (kv_off 8, slot_table 16) and
 * must not overlap (granted_len in the place of prev_len or req_len is
 * PILLAR_ERR_ARG).  Asynchronous on `stream`; allocates nothing.  Returns
 * PILLAR_OK, PILLAR_ERR_ARG, PILLAR_ERR_WORKSPACE or PILLAR_ERR_CUDA.
 */
PILLAR_API int pillar_block_map(const pillar_shape_t *shape, const int32_t *req_len, const int32_t *prev_len,
                                int32_t *block_table, int32_t max_blocks, int32_t *free_ring, int32_t *free_state,
                                int32_t *granted_len, int64_t *kv_off, int32_t *slot_table, int64_t slot_capacity,
                                int32_t *new_off, int32_t *new_slots, int64_t new_capacity, void *workspace,
                                size_t ws_bytes, void *stream);

/*
 * The 8-bit cache.  K and V are held as e4m3 codes (4 exponent bits of bias
 * 7, 3 fraction bits, largest value 448) with one fp32 scale per block of 16
 * tokens and KV head: value = code * scale.
 *   k8_pool, v8_pool  [num_slots / 16, Hkv, 16, D] codes, one byte each: the 16
 *                     rows of a (block, KV head) lie together
 *   k_scale, v_scale  [num_slots / 16, Hkv] fp32
 * Blocks and block tables are those of pillar_block_map.
 */

/*
 * pillar_kv8_append -- rounds the new tokens' K and V rows into the cache
 * (the 8-bit form of pillar_kv_append).  Request b's new tokens are its last
 * ones: with n_b = new_off[b+1] - new_off[b], packed row new_off[b] + i is
 * position req_len[b] - n_b + i.  For the new rows x of one (block, KV head),
 * a = max |x| and e the smallest integer >= -126 with a <= 448 * 2^e:
 *   scale' = 2^e when row 0 of the block is among them, else max(scale, 2^e)
 *   codes  = x / scale' rounded to the nearest e4m3 (ties to even); where the
 *            block holds earlier rows and its scale grew, all of its other rows
 *            become code * scale / scale' rounded the same way
 * Otherwise the other rows of the block are left as they were, and a block
 * without new rows is not touched.  A call with the same new rows again leaves
 * what the first one did.  A block that gets new rows must belong to one
 * request only.
 *
 *   k_new, v_new  bf16, row i at i * k_stride (v_stride) elements: [Hkv, D] each,
 *                 16-byte aligned rows (a stride is a multiple of 8, at least
 *                 Hkv * D; 0 means Hkv * D)
 *   n             rows of k_new and v_new; rows at or past new_off[B] are not read
 *   req_len       [B] int32, the lengths that include the new tokens
 *   new_off       [B+1] int32, ascending from 0 (as pillar_block_map writes it)
 *   block_table   [B, max_blocks] int32
 *   device_flags  device int32 or null, or-ed: PILLAR_FLAG_REQUEST for offsets or
 *                 lengths that do not fit together, n, max_len or max_blocks (the
 *                 rows concerned are skipped), PILLAR_FLAG_SLOT for a block
 *                 outside the pool (skipped), PILLAR_FLAG_VALUE for a NaN (stored
 *                 as 0), an infinity (stored as the largest value of its sign;
 *                 the scale goes by the finite values), or a scale of earlier
 *                 rows that is negative or not finite (taken as 0)
 * Only shape->B, Hkv, D, max_len and num_slots are used.  Pools are 16-byte
 * aligned, the other arrays 4.  Asynchronous on `stream`; allocates nothing.
 * Returns PILLAR_OK, PILLAR_ERR_ARG or PILLAR_ERR_CUDA.
 */
PILLAR_API int pillar_kv8_append(const pillar_shape_t *shape, const uint16_t *k_new, int64_t k_stride,
                                 const uint16_t *v_new, int64_t v_stride, int32_t n, const int32_t *req_len,
                                 const int32_t *new_off, const int32_t *block_table, int32_t max_blocks,
                                 uint8_t *k8_pool, uint8_t *v8_pool, float *k_scale, float *v_scale,
                                 int32_t *device_flags, void *stream);

/*
 * pillar_attn_kv8 -- the unified draft/verify step over the 8-bit cache:
 * pillar_attn_unified with k8_pool, v8_pool, k_scale, v_scale and block_table
 * in the place of the bf16 pools and the slot table.  Position t of request b
 * is row t % 16 of block block_table[b, t / 16].  With k = 0 and every request
 * in verify mode it is plain decoding: one query row over its whole context.
 *   verify_logits  as pillar_attn_unified writes them (so that
 *                  pillar_topk_select follows unchanged), or NULL: no dump
 *   workspace      pillar_attn_workspace_bytes
 * A probability is rounded to f16 with its key's value scale in it, relative to
 * the largest value scale among the keys before it in the context (the keys
 * that its row does not see included): a key whose scale is 2^24 or more below
 * that one's keeps eight bits of its weight, or fewer, and its part of the row's
 * output is off by up to 2^-32 of the largest value among those keys.
 * Alignment: q, out and the pools 16 bytes, verify_logits 8, the other arrays
 * 4.  The schedule is UNIFIED, DRAFT_ONLY or VERIFY_ONLY (PILLAR_ERR_ARG
 * otherwise); wait_timeout_us has no meaning here (nothing waits on the
 * device).  A block outside [0, num_slots / 16) or a position past
 * max_blocks is skipped and flagged PILLAR_FLAG_SLOT.  A NaN in q makes its
 * row NaN.  A NaN scale of K, or code, does so to the rows of its request and
 * KV head that see the key, a NaN scale of V to those that do not as well, a
 * NaN code of V in its dimension; verify_lse is NaN where the scores are.  All
 * that holds however the context is split.  pillar_kv8_append writes no NaN.
 *
 * pillar_attn_run_kv8 -- the same on the plan that pillar_attn_plan left in the
 * workspace (as pillar_attn_run): one plan for the layers of a model step.
 *
 * Returns PILLAR_OK, PILLAR_ERR_ARG, PILLAR_ERR_WORKSPACE or PILLAR_ERR_CUDA.
 */
PILLAR_API int pillar_attn_kv8(const pillar_shape_t *shape, const uint16_t *q, const uint8_t *k8_pool,
                               const uint8_t *v8_pool, const float *k_scale, const float *v_scale,
                               const int32_t *block_table, int32_t max_blocks, const int32_t *req_mode,
                               const int32_t *req_len, const int32_t *sparse_idx, const int32_t *sparse_cnt,
                               uint16_t *out, float *verify_logits, float *verify_lse, void *workspace,
                               size_t ws_bytes, void *stream);
PILLAR_API int pillar_attn_run_kv8(const pillar_shape_t *shape, const uint16_t *q, const uint8_t *k8_pool,
                                   const uint8_t *v8_pool, const float *k_scale, const float *v_scale,
                                   const int32_t *block_table, int32_t max_blocks, const int32_t *sparse_idx,
                                   uint16_t *out, float *verify_logits, float *verify_lse, void *workspace,
                                   size_t ws_bytes, void *stream);

/*
 * pillar_kv8_read -- positions of the 8-bit cache as bf16 rows: a prefix for a
 * call that takes bf16 keys, or a context on its way to the bf16 pools
 * (pillar_kv_append).  Packed row out_off[b] + i is position first[b] + i of
 * request b, value = code * scale rounded to bf16 (exact under the scales that
 * pillar_kv8_append writes, but past the ends of bf16's range).
 *
 *   block_table   [B, max_blocks] int32
 *   first         [B] int32, the requests' first positions
 *   out_off       [B+1] int32, ascending from 0: the rows of each request
 *   n             rows of k_out and v_out; rows at or past out_off[B] are left
 *                 as they were
 *   k_out, v_out  bf16, row i at i * k_stride (v_stride) elements: [Hkv, D] each,
 *                 16-byte aligned rows (a stride is a multiple of 8, at least
 *                 Hkv * D; 0 means Hkv * D).  They overlap nothing.
 *   device_flags  device int32 or null, or-ed: PILLAR_FLAG_REQUEST for offsets or
 *                 positions that do not fit together, n, max_len (the end of a
 *                 request's rows) or max_blocks, PILLAR_FLAG_SLOT for a block
 *                 outside the pool; the rows concerned are left as they were
 * Only shape->B, Hkv, D, max_len and num_slots are used; Hkv * D is at most
 * 2^26.  Pools are 16-byte aligned, the other arrays 4.  Asynchronous on
 * `stream`; allocates nothing.  Returns PILLAR_OK, PILLAR_ERR_ARG or
 * PILLAR_ERR_CUDA.
 */
PILLAR_API int pillar_kv8_read(const pillar_shape_t *shape, const uint8_t *k8_pool, const uint8_t *v8_pool,
                               const float *k_scale, const float *v_scale, const int32_t *block_table,
                               int32_t max_blocks, const int32_t *first, const int32_t *out_off, int32_t n,
                               uint16_t *k_out, int64_t k_stride, uint16_t *v_out, int64_t v_stride,
                               int32_t *device_flags, void *stream);

/*
 * The 4-bit cache.  K and V are held as e2m1 codes (sign, two exponent bits of
 * bias 1, one fraction bit: magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6) with a scale
 * byte for every PILLAR_KV4_GROUP neighbouring values of a row: value =
 * code * scale.  A scale byte holds five exponent bits of bias 15 and three
 * fraction bits, no sign: byte 8 e + m is (1 + m / 8) 2^(e - 15), or m 2^-17
 * where e is 0.  4.5 bits a value; every value is exact in bf16 and f16.
 *   k4_pool, v4_pool  [num_slots / 16, Hkv, 16, D / 2] bytes: dimension 2 i in the
 *                     low half of byte i, 2 i + 1 in the high half
 *   k_scale, v_scale  [num_slots / 16, Hkv, 16, D / 16] bytes
 * Blocks and block tables are those of pillar_block_map.
 */
#define PILLAR_KV4_GROUP 16

/*
 * pillar_kv4_append -- rounds the new tokens' K and V rows into the cache.
 * Request b's new tokens are its last ones, as in pillar_kv8_append.  For 16
 * neighbouring values x of a row, with a = max |x|:
 *   scale = the smallest scale s with a <= 6 s, at least 2^-17 and at most
 *           10240 (six times that is the largest value held, 61440)
 *   codes = x / s rounded to the nearest e2m1 value (ties to even), magnitudes
 *           past 6 to 6; the sign of a code that stands for 0 has no meaning
 * A row's codes and scales depend on that row alone: no other row is touched,
 * and rows may be appended again (after a rollback) in any order.
 *
 * Arguments as pillar_kv8_append's.  device_flags: PILLAR_FLAG_REQUEST and
 * PILLAR_FLAG_SLOT as there; PILLAR_FLAG_VALUE for a NaN (stored as 0), an
 * infinity (stored as 6 s of its sign; the scale goes by the finite values) or
 * a magnitude past 61440 (stored as 61440).
 * Only shape->B, Hkv, D, max_len and num_slots are used; Hkv * D is at most
 * 2^26.  k_new, v_new and the pools are 16-byte aligned, the scales 8, the other
 * arrays 4.  Asynchronous on `stream`; allocates nothing.  Returns PILLAR_OK,
 * PILLAR_ERR_ARG or PILLAR_ERR_CUDA.
 */
PILLAR_API int pillar_kv4_append(const pillar_shape_t *shape, const uint16_t *k_new, int64_t k_stride,
                                 const uint16_t *v_new, int64_t v_stride, int32_t n, const int32_t *req_len,
                                 const int32_t *new_off, const int32_t *block_table, int32_t max_blocks,
                                 uint8_t *k4_pool, uint8_t *v4_pool, uint8_t *k_scale, uint8_t *v_scale,
                                 int32_t *device_flags, void *stream);

/*
 * pillar_kv4_read -- positions of the 4-bit cache as bf16 rows: exact under the
 * scales that pillar_kv4_append writes; under larger ones a value past f16's range
 * is infinite.  The arguments are pillar_kv8_read's, the scales 8-byte aligned.
 */
PILLAR_API int pillar_kv4_read(const pillar_shape_t *shape, const uint8_t *k4_pool, const uint8_t *v4_pool,
                               const uint8_t *k_scale, const uint8_t *v_scale, const int32_t *block_table,
                               int32_t max_blocks, const int32_t *first, const int32_t *out_off, int32_t n,
                               uint16_t *k_out, int64_t k_stride, uint16_t *v_out, int64_t v_stride,
                               int32_t *device_flags, void *stream);

/*
 * pillar_attn_kv4 -- the unified draft/verify step over the 4-bit cache:
 * pillar_attn_kv8 with k4_pool, v4_pool and the scale bytes in the place of the
 * 8-bit pools and scales.  With k = 0 and every request in verify mode it is
 * plain decoding.  Alignment: q, out and the pools 16 bytes, verify_logits and
 * the scales 8, the other arrays 4.  Schedules, workspace, skipped blocks and
 * positions and their flags are as there.
 *
 * The products are exact (cache values and scaled queries are f16 values; an
 * element of a query row is off by up to 2^-39 of the row's largest), their
 * sums fp32.  A probability is rounded to f16: one below 2^-20 of the largest
 * among the keys that it is summed with keeps fewer than eleven bits and is off
 * by up to 2^-31 of that.
 *
 * Verify items of many rows go through a pipeline whose waits are bounded by
 * the shape's wait_timeout_us (0: one second); past it PILLAR_FLAG_TIMEOUT is
 * recorded, the outputs are incomplete and the next call on the workspace is
 * whole.  (A wait is also given up after four million polls, were the bound longer
 * than these; an item takes microseconds.)
 *
 * Where verify_chunk is 0, max_len at least 8192 and (k+1)*G at most 16, the call
 * plans with a verify_chunk of its own: the share of max_len that gives each of
 * 4 CTAs an SM a piece, rounded up to 64 and at least 1024, if that is less than
 * 2048.  pillar_attn_plan does not: what pillar_attn_run_kv4 computes on its plan
 * may differ in the last bits, and a shape with that verify_chunk gives both the
 * same items.
 *
 * A NaN or infinity in q makes its row of out and verify_lse NaN, unless the row
 * has no position to see (one that is skipped counts).  The append writes scale
 * bytes of 1 to 226; under others (0 is a scale of 0) a value past f16's range is
 * infinite, and one may be NaN.  A score that such a K row makes NaN or +inf makes
 * the row of out and verify_lse NaN; a key whose score is -inf counts as one that
 * is not there.  A value of a V row that is NaN or infinite makes its dimension so
 * in the rows that see the key (an infinity may make it NaN), and may make it NaN
 * in other rows of the request and KV head.  All that holds however the context is
 * split.
 *
 * pillar_attn_run_kv4 -- the same on the plan that pillar_attn_plan left in the
 * workspace (as pillar_attn_run): one plan for the layers of a model step.
 *
 * Returns PILLAR_OK, PILLAR_ERR_ARG, PILLAR_ERR_WORKSPACE or PILLAR_ERR_CUDA.
 */
PILLAR_API int pillar_attn_kv4(const pillar_shape_t *shape, const uint16_t *q, const uint8_t *k4_pool,
                               const uint8_t *v4_pool, const uint8_t *k_scale, const uint8_t *v_scale,
                               const int32_t *block_table, int32_t max_blocks, const int32_t *req_mode,
                               const int32_t *req_len, const int32_t *sparse_idx, const int32_t *sparse_cnt,
                               uint16_t *out, float *verify_logits, float *verify_lse, void *workspace,
                               size_t ws_bytes, void *stream);
PILLAR_API int pillar_attn_run_kv4(const pillar_shape_t *shape, const uint16_t *q, const uint8_t *k4_pool,
                                   const uint8_t *v4_pool, const uint8_t *k_scale, const uint8_t *v_scale,
                                   const int32_t *block_table, int32_t max_blocks, const int32_t *sparse_idx,
                                   uint16_t *out, float *verify_logits, float *verify_lse, void *workspace,
                                   size_t ws_bytes, void *stream);

/* pillar_prompt_attn_workspace_bytes -- workspace of pillar_prompt_attn for
 * shape->B sequences of n tokens in all. */
PILLAR_API int pillar_prompt_attn_workspace_bytes(const pillar_shape_t *shape, int32_t n, size_t *bytes);

/*
 * pillar_prompt_attn -- causal attention over whole prompts, packed one after
 * another: what fills a context before its first draft step.  With rows
 * [seq_off[b], seq_off[b+1]) the tokens of sequence b, row i of it and query
 * head h attend rows 0 .. i of the sequence under KV head h / G:
 *   out[i, h] = sum_j softmax_j(scale * q[i, h] . k[j, h / G]) v[j, h / G]
 *   lse[i, h] = log sum_j exp(scale * q[i, h] . k[j, h / G])   (natural log)
 *
 *   q             bf16, token i's [Hq, D] at i * q_stride elements
 *   k, v          bf16, token i's [Hkv, D] at i * k_stride (v_stride)
 *                 (a stride of 0 means packed rows; others are multiples of 8
 *                 and at least the row, e.g. slices of one projection's output)
 *   n             tokens in q, k, v, out and lse
 *   seq_off       [B+1] int32, ascending, within [0, n].  A sequence whose
 *                 offsets descend, leave [0, n] or are more than max_len apart
 *                 is skipped (PILLAR_FLAG_REQUEST); so are all when they
 *                 overlap by more than the workspace has room for.  Empty ones
 *                 are allowed.  Rows of no sequence are left as they were.
 *   out           [n, Hq, D] bf16
 *   lse           [n, Hq] fp32, or NULL
 *   workspace     pillar_prompt_attn_workspace_bytes bytes, 256-byte aligned; its
 *                 error word is cleared by the call and read with
 *                 pillar_get_error
 * Only shape->B, Hq, Hkv, D, max_len, sm_scale and wait_timeout_us are used (the
 * whole shape is checked; k = 0 fits).  q, k, v and out are 16-byte aligned,
 * seq_off and lse 4.  A NaN or infinity in a token's v may reach rows of its own
 * sequence that precede it by less than 128 positions; it never reaches another
 * sequence.  Every wait on the device is bounded as in pillar_attn_unified.
 * Asynchronous on `stream`; allocates nothing.  Returns PILLAR_OK,
 * PILLAR_ERR_ARG, PILLAR_ERR_WORKSPACE or PILLAR_ERR_CUDA; with n == 0 or
 * B == 0 nothing is launched.
 */
PILLAR_API int pillar_prompt_attn(const pillar_shape_t *shape, const uint16_t *q, int64_t q_stride, const uint16_t *k,
                                  int64_t k_stride, const uint16_t *v, int64_t v_stride, int32_t n,
                                  const int32_t *seq_off, uint16_t *out, float *lse, void *workspace, size_t ws_bytes,
                                  void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PILLAR_H */
