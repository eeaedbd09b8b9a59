/*
 * libpa — paged decode attention for NVIDIA GB300 (sm_103a), C ABI.
 *
 * One decode step of attention for a batch of sequences whose keys and
 * values live in a paged KV cache addressed through a per-sequence block
 * table.  Two algorithms compute the same result:
 *
 *   V1  one pass over each sequence (one CTA per sequence and KV head);
 *   V2  the partitioned form of the "paged_attention_v2" commit note
 *       (project_6, commit 96f4baf "Dockerfile", section "Implementation"):
 *       Phase 1 computes, for every (sequence, head, partition of
 *       partition_size tokens), the max logit, the exp-sum and the
 *       normalised weighted V sum; Phase 2 merges the partitions with the
 *       log-sum-exp rescale (global max, rescale by exp(m_p - M) times the
 *       partition's exp-sum, normalised sum of the partials).
 *
 * Both reach out[s][h] = softmax_t(scale * q[s][h] . K_t) @ V over the
 * seq_lens[s] tokens of sequence s, kvh = h / (num_heads / num_kv_heads).
 *
 * Layouts (row-major, contiguous, device memory):
 *   query, out         [num_seqs][num_heads][head_size]          (dtype)
 *   key_cache,
 *   value_cache        [num_blocks][num_kv_heads][block_size][head_size]
 *   block_tables       int32 [num_seqs][max_blocks_per_seq]; entry j of row s
 *                      is the physical block holding tokens
 *                      [j*block_size, (j+1)*block_size) of sequence s.
 *                      Entries past ceil(seq_lens[s]/block_size) are never read.
 *   seq_lens           int32 [num_seqs], each in [0, max_seq_len]
 *
 * Ownership: the caller owns every buffer and the stream.  The library
 * allocates no device memory, never synchronises in the forward calls, and
 * only enqueues kernels on `stream` (a cudaStream_t passed as void*; NULL is
 * the legacy default stream).  Calls on one workspace must not overlap.
 *
 * Errors: argument problems are found on the host and returned before any
 * launch.  A failed launch returns PA_ERR_CUDA (see pa_last_cuda_error).
 * Problems in the data, found by the kernels (a block-table entry outside
 * [0, num_blocks), a sequence length outside [0, max_seq_len]) or a bounded
 * device wait that ran out, are recorded in the workspace's status word and
 * read with pa_read_device_status.  Kernels never trap.
 *
 * Supported: dtype f32, bf16, f16 (query, caches and out share it);
 * head_size 64, 128, 256; block_size 8, 16, 32, 64; num_heads / num_kv_heads
 * in [1, 16]; partition_size a multiple of 64 and of block_size, at most
 * 8192.  K and V caches, query and out 16-byte aligned; workspace 256-byte
 * aligned; num_blocks * num_kv_heads * block_size < 2^31.
 */
#ifndef PA_H_
#define PA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  PA_OK = 0,
  PA_ERR_INVALID_ARG = 1,         /* bad pointer, size or combination      */
  PA_ERR_UNSUPPORTED = 2,         /* legal but not built (dtype, sizes)    */
  PA_ERR_WORKSPACE_TOO_SMALL = 3, /* workspace_bytes < pa_workspace_bytes  */
  PA_ERR_CUDA = 4,                /* a CUDA runtime call failed            */
  PA_ERR_DEVICE_BAD_INPUT = 5,    /* kernel saw a bad block id / length    */
  PA_ERR_DEVICE_TIMEOUT = 6       /* a bounded device wait ran out         */
} pa_status_t;

typedef enum { PA_DTYPE_F32 = 0, PA_DTYPE_BF16 = 1, PA_DTYPE_F16 = 2 } pa_dtype_t;

typedef enum { PA_VARIANT_AUTO = 0, PA_VARIANT_V1 = 1, PA_VARIANT_V2 = 2 } pa_variant_t;

/* Arithmetic of QK^T and PV.  AUTO: tensor cores (mma, fp32 accumulate) for
 * bf16/f16, CUDA-core fp32 FMA for f32.  SIMT forces the CUDA-core path. */
typedef enum { PA_MATH_AUTO = 0, PA_MATH_SIMT = 1, PA_MATH_TENSOR = 2 } pa_math_t;

/* Optional knobs for pa_forward.  Zero-initialise, then set what you need. */
typedef struct {
  int32_t variant;        /* pa_variant_t                                   */
  int32_t math;           /* pa_math_t                                      */
  int32_t num_stages;     /* KV pipeline depth per CTA, 0 = library choice  */
  int32_t debug_flags;    /* PA_DEBUG_*; 0 in production                    */
  uint64_t wait_limit_ns; /* bound on each device wait, 0 = 1 second        */
  void *phase1_event;     /* cudaEvent_t or NULL: for V2, recorded on the
                             stream between the Phase 1 and Phase 2 kernels
                             (lets a caller time the phases with events)   */
  int32_t ctas_per_sm;    /* persistent CTAs per SM, 0 = as many as fit     */
  int32_t fuse_partitions;/* V2: sequences of at most this many partitions
                             (capped at 16) get the cross-partition combine
                             inside the Phase 1 kernel; 0 (the default) or
                             negative = never: the Phase 2 kernel does it */
  int32_t share_kv;       /* query chunks on the tcgen05 kernel (head_size
                             128, more than 16 rows per KV head) with 256 or
                             more rows per KV head: 1 = the CTAs of the row
                             groups of the same keys form a thread-block
                             cluster (of 2 or 4) and share every K/V stage
                             through multicast copies, so that K/V cross HBM
                             once instead of once per row group; slower on
                             GB300 when HBM is not the limit (measured
                             2.5-10 %); 0 (the default) = each CTA loads its
                             own */
} pa_options_t;

/* Debug: every consumer warp waits on a barrier that nothing ever releases,
 * so the bounded wait runs out and the kernel reports PA_ERR_DEVICE_TIMEOUT
 * (after letting its own in-flight copies land).  Used to test the timeout
 * path without hanging or faulting the GPU. */
#define PA_DEBUG_STALL_CONSUMERS 1

/* Debug: query chunks never take the tcgen05 kernel (chunks of more than 16
 * rows per KV head at head_size 128 then run on the mma.sync row-owning
 * kernel), for comparisons of the two. */
#define PA_DEBUG_NO_TCGEN05 2

/* Option: every call that the tcgen05 kernel of small items can serve takes
 * it: head_size 128, bf16/f16, at most 16 query rows per KV head and item
 * (decode with any group, query chunks of up to 16 / group tokens an item),
 * without the fused combine.  The keys of a stage are the MMA's M and the
 * item's rows its N, so no tensor-core lane computes a missing row.  Off by
 * default: on GB300 the mma.sync kernels are faster on every such workload
 * measured (decode with 16 query heads a KV head: 0.116-0.146 ms against
 * 0.098 ms a step).  PA_DEBUG_NO_TCGEN05 wins over it. */
#define PA_DEBUG_TCGEN05_KEYS 4


/* Bytes of workspace that pa_v2_forward needs (V1 needs only the 256-byte
 * status block).  The partials are the three per-partition arrays that the
 * "paged_attention_v2" commit note (project_6, commit 96f4baf "Dockerfile",
 * section "Implementation", "Phase 1") has Phase 1 store for Phase 2:
 * tmp_output, exp_sums and max_logits, kept in fp32 here.
 * Layout, each part 256-byte aligned, in this order:
 *   status      int32 status word + work-queue counters (a 256-byte block)
 *   max_logits  f32 [num_seqs][num_heads][max_parts]   Phase 1 max logit
 *   exp_sums    f32 [num_seqs][num_heads][max_parts]   sum exp(logit - max)
 *   tmp_out     f32 [num_seqs][num_heads][max_parts][head_size]  normalised
 *   counters    int32 [num_seqs][num_heads]: partitions finished per
 *               (sequence, KV head), for the fused cross-partition combine
 * with max_parts = ceil(max_seq_len / partition_size).  Returns 0 on bad
 * arguments. */
size_t pa_workspace_bytes(int num_seqs, int num_heads, int head_size,
                          int max_seq_len, int partition_size);

/* Byte offsets of the five workspace parts above (offsets[0..4]); returns
 * PA_ERR_INVALID_ARG on bad arguments.  Lets callers read Phase 1 results. */
pa_status_t pa_workspace_layout(int num_seqs, int num_heads, int head_size,
                                int max_seq_len, int partition_size,
                                size_t offsets[5]);

/* Zero a new workspace (enqueued on `stream`).  Call once after allocating
 * it, and again after a call reported a device error.  Kernels only ever
 * set the status word to a nonzero code; the work-queue and combine
 * counters are left at zero by every launch that completes. */
pa_status_t pa_workspace_init(void *workspace, size_t workspace_bytes,
                              void *stream);

/* V1: single pass over each whole sequence, the kernel the "paged_attention_v2"
 * commit note (project_6, commit 96f4baf "Dockerfile") opens with: "V1
 * limitation" describes it as one launch over the entire KV sequence, and its
 * "Integration" list keeps it for sequences of up to 8192 tokens.  Here a
 * work item is one (sequence, KV head), computing all num_heads/num_kv_heads
 * query heads of the group with an online softmax; items are spread over a
 * persistent grid.  partition_size is validated but otherwise unused.
 * The workspace needs >= 256 bytes (its status block). */
pa_status_t pa_v1_forward(void *out, const void *query, const void *key_cache,
                          const void *value_cache, const int32_t *block_tables,
                          const int32_t *seq_lens, int num_seqs, int num_heads,
                          int num_kv_heads, int head_size, int num_blocks,
                          int block_size, int max_blocks_per_seq,
                          int max_seq_len, float scale, int partition_size,
                          int dtype, void *workspace, size_t workspace_bytes,
                          void *stream);

/* V2: the Phase 1 kernel computes every (sequence, KV head, partition) and
 * writes max_logits / exp_sums / tmp_out into the workspace; then the
 * log-sum-exp combine (Phase 2 kernel) writes out.  With
 * pa_options_t.fuse_partitions = n > 0, for a sequence of at most min(n, 16)
 * partitions the last Phase 1 work item of each (sequence, KV head) does
 * that combine instead, and the Phase 2 kernel is launched only if
 * max_seq_len allows a longer sequence.  Same arguments
 * as V1; the workspace must hold pa_workspace_bytes(...) bytes. */
pa_status_t pa_v2_forward(void *out, const void *query, const void *key_cache,
                          const void *value_cache, const int32_t *block_tables,
                          const int32_t *seq_lens, int num_seqs, int num_heads,
                          int num_kv_heads, int head_size, int num_blocks,
                          int block_size, int max_blocks_per_seq,
                          int max_seq_len, float scale, int partition_size,
                          int dtype, void *workspace, size_t workspace_bytes,
                          void *stream);

/* The same call with the V1/V2 choice made by pa_choose_v2 (the device's SM
 * count is queried once per device), or forced through `opts` (NULL = all
 * defaults).  For V2 the workspace must hold pa_workspace_bytes(...). */
pa_status_t pa_forward(void *out, const void *query, const void *key_cache,
                       const void *value_cache, const int32_t *block_tables,
                       const int32_t *seq_lens, int num_seqs, int num_heads,
                       int num_kv_heads, int head_size, int num_blocks,
                       int block_size, int max_blocks_per_seq, int max_seq_len,
                       float scale, int partition_size, int dtype,
                       void *workspace, size_t workspace_bytes, void *stream,
                       const pa_options_t *opts);

/* The two phases of V2 as separate calls, for splitting long sequences over
 * several GPUs (context parallelism).  The "paged_attention_v2" commit note
 * (project_6, commit 96f4baf "Dockerfile", section "Implementation") defines
 * Phase 1 per partition and Phase 2 as the log-sum-exp reduction over a
 * sequence's partitions; the partitions are independent until Phase 2, so
 * GPU r can run Phase 1 over its own range of partitions, the GPUs exchange
 * their partials (one all-gather of max_logits, exp_sums and tmp_out slots,
 * done by the caller), and Phase 2 over the gathered slots gives the
 * single-GPU result.
 *
 * pa_v2_partials: Phase 1 only, for the partitions p with
 *   part_begin <= p < min(part_end, ceil(seq_lens[s] / partition_size))
 * of every sequence s.  It writes their max_logits / exp_sums / tmp_out
 * slots of the workspace (the layout of pa_workspace_layout, sized by
 * pa_workspace_bytes for the whole sequences) and nothing else: slots of
 * other partitions keep their contents, and there is no output.  Block-table
 * entries of pages outside the range are never read, so a GPU that holds only
 * its own range's pages may pass -1 there.  The arguments are those of
 * pa_v2_forward (seq_lens are the whole lengths), without out, plus
 * 0 <= part_begin <= part_end (PA_ERR_INVALID_ARG otherwise; part_end may
 * exceed the partition count).  [0, INT32_MAX) is Phase 1 of pa_v2_forward.
 * Errors as pa_v2_forward; device-detected ones land in this workspace's
 * status word. */
pa_status_t pa_v2_partials(const void *query, const void *key_cache,
                           const void *value_cache, const int32_t *block_tables,
                           const int32_t *seq_lens, int num_seqs, int num_heads,
                           int num_kv_heads, int head_size, int num_blocks,
                           int block_size, int max_blocks_per_seq,
                           int max_seq_len, float scale, int partition_size,
                           int dtype, int part_begin, int part_end,
                           void *workspace, size_t workspace_bytes,
                           void *stream);

/* pa_v2_combine: Phase 2 only.  For every sequence s and head h, the
 * log-sum-exp combine of the slots of partitions 0 .. ceil(seq_lens[s] /
 * partition_size) - 1 in the workspace, written to out[s][h] in dtype (zeros
 * for an empty sequence).  Every one of those slots must hold a Phase 1
 * result (pa_v2_partials here, or slots copied in from other GPUs); the
 * workspace is only read.  seq_lens and out on the device, layouts and the
 * other arguments as pa_v2_forward; head_size, dtype and partition_size are
 * checked as there.  Enqueued on `stream` after whatever precedes it. */
pa_status_t pa_v2_combine(void *out, const int32_t *seq_lens, int num_seqs,
                          int num_heads, int head_size, int max_seq_len,
                          int partition_size, int dtype, const void *workspace,
                          size_t workspace_bytes, void *stream);

/* Multi-token queries over the paged cache: the query of sequence s is a
 * chunk of its LAST n_s = q_start[s+1] - q_start[s] cached tokens (for
 * example draft tokens to verify, or a small prefill chunk whose keys and
 * values are already in the cache), rows q_start[s] .. q_start[s+1]-1 of
 * query and out ([num_rows][num_heads][head_size]).  Chunk token i, at cache
 * position L - n_s + i with L = seq_lens[s], attends causally to the cache
 * tokens [0, L - n_s + i].  The pages give no formula for this; it is the
 * plain causal reading of attention over a paged prefix (the prefill patch
 * of project_6 tunes such a kernel).
 *
 * q_start: device int32 [num_seqs + 1], non-decreasing, q_start[0] = 0,
 * q_start[num_seqs] = num_rows, 0 <= n_s <= min(seq_lens[s], max_chunk).
 * The other arguments as pa_forward (opts->variant picks V1/V2/auto); the V2
 * workspace is sized as pa_workspace_bytes(num_rows, ...).  bf16 and f16 only
 * (PA_ERR_UNSUPPORTED for f32).  An item covers 16 / (num_heads /
 * num_kv_heads) tokens of a chunk, so longer chunks re-read their prefix once
 * per such group (from L2 when the groups of a partition run together).  A
 * chunk that breaks the rules above is reported as PA_ERR_DEVICE_BAD_INPUT
 * and its rows hold no meaningful values (the other sequences' rows are
 * computed as usual). */
pa_status_t pa_chunks_forward(void *out, const void *query,
                              const void *key_cache, const void *value_cache,
                              const int32_t *block_tables,
                              const int32_t *seq_lens, const int32_t *q_start,
                              int num_seqs, int num_rows, int max_chunk,
                              int num_heads, int num_kv_heads, int head_size,
                              int num_blocks, int block_size,
                              int max_blocks_per_seq, int max_seq_len,
                              float scale, int partition_size, int dtype,
                              void *workspace, size_t workspace_bytes,
                              void *stream, const pa_options_t *opts);

/* Device bytes of the staging buffer pa_forward_host needs: the query and
 * the output ([num_seqs][num_heads][head_size] in the dtype), the block
 * tables and seq_lens, each part 256-byte aligned.  Returns 0 on bad
 * arguments. */
size_t pa_host_staging_bytes(int num_seqs, int num_heads, int head_size,
                             int max_blocks_per_seq, int dtype);

/* pa_forward with the per-step data in HOST memory: query_host,
 * block_tables_host and seq_lens_host are read from the host and out_host is
 * written on the host (same layouts as pa_forward).  The KV caches and the
 * workspace stay on the device.  `staging` is a caller-owned device buffer of
 * at least pa_host_staging_bytes(...) bytes, 256-byte aligned.
 *
 * When all four host buffers are pinned (page-locked, hence mapped into the
 * device's address space; out_host 16-byte aligned), nothing goes through a
 * copy engine: one kernel reads the lengths, block tables and queries from
 * the host buffers into the staging buffer over the host link, and the last
 * kernel of the forward stores the output straight into out_host.  Otherwise
 * the call enqueues one host-to-device cudaMemcpyAsync each of seq_lens, the
 * block tables and the query into the staging buffer, the kernels of
 * pa_forward, and one device-to-host copy of the output (pageable buffers
 * make those copies synchronise the host with the stream).
 *
 * Either way it returns when everything is enqueued on `stream`: synchronise
 * the stream before reading out_host.  The host buffers and the staging
 * buffer must stay untouched until the stream reaches the end of the call.
 * Errors: as pa_forward, plus PA_ERR_INVALID_ARG for a null host pointer or
 * a staging buffer that is null, misaligned or smaller than
 * pa_host_staging_bytes(...); argument errors come back before anything is
 * enqueued. */
pa_status_t pa_forward_host(void *out_host, const void *query_host,
                            const void *key_cache, const void *value_cache,
                            const int32_t *block_tables_host,
                            const int32_t *seq_lens_host, int num_seqs,
                            int num_heads, int num_kv_heads, int head_size,
                            int num_blocks, int block_size,
                            int max_blocks_per_seq, int max_seq_len,
                            float scale, int partition_size, int dtype,
                            void *staging, size_t staging_bytes,
                            void *workspace, size_t workspace_bytes,
                            void *stream, const pa_options_t *opts);

/* V2 for callers that cannot allocate device memory, for example a plug-in
 * whose host framework owns all device memory and forbids cudaMalloc while
 * it serves a request, or a serving loop that must not pay cudaMalloc's
 * implicit synchronisation.  The paged_attention_v2 pages have no
 * counterpart: this entry point exists only for such callers.
 *
 * Same arguments as pa_v2_forward, minus the workspace.  V2's scratch comes
 * from a fixed 32 MiB array in device memory owned by the library.  Every
 * GPU that loads the library holds the array until the process exits.
 * Requests whose pa_workspace_bytes(...) exceeds 32 MiB return
 * PA_ERR_WORKSPACE_TOO_SMALL.  The call allocates nothing and calls no
 * allocating routine.
 *
 * The first call on a device looks up the array's device address (with that
 * device current); make that first call before any stream capture.  All
 * calls on a device share the one array and each overwrites what the last
 * left there, so calls whose kernels overlap on the GPU race: serialise
 * them.  Device-detected data errors land in the shared array's status word,
 * which each call clears; callers that need pa_read_device_status use
 * pa_v2_forward with their own workspace. */
pa_status_t pa_v2_forward_noalloc(void *out, const void *query,
                                  const void *key_cache,
                                  const void *value_cache,
                                  const int32_t *block_tables,
                                  const int32_t *seq_lens, int num_seqs,
                                  int num_heads, int num_kv_heads,
                                  int head_size, int num_blocks,
                                  int block_size, int max_blocks_per_seq,
                                  int max_seq_len, float scale,
                                  int partition_size, int dtype, void *stream);

/* Append new keys and values to the paged cache, rotating keys (and queries)
 * by their positions on the way, and keeping the pages' key bounds.
 *
 * The rows are the tokens that the sequences gain: with q_start (device int32
 * [num_seqs + 1], as for pa_chunks_forward) row r of sequence s is token
 * t = seq_lens[s] - n_s + (r - q_start[s]), n_s = q_start[s+1] - q_start[s];
 * with q_start NULL there is one row a sequence (num_rows = num_seqs), its
 * last token, and a sequence of length 0 is an empty slot, skipped.  seq_lens
 * are the lengths AFTER the append.  Rows from q_start[num_seqs] on are
 * padding: they need no positions, nothing is appended for them, and their
 * query_out is left as it was.
 *
 *   key, value         [num_rows][num_kv_heads][head_size]; rows key_stride /
 *                      value_stride elements apart (16-byte multiples), so
 *                      they may be slices of one projection's output
 *   query, query_out   [num_rows][num_heads][head_size], rows of query
 *                      query_stride apart, query_out contiguous; both NULL
 *                      when there are no queries to rotate; may be the same
 *                      contiguous buffer
 *   cos_sin            f32 [max_position][rotary_dim]: rotary_dim / 2 cosines,
 *                      then the sines; NULL if rotary_dim is 0
 *   positions          int32 [num_rows], or NULL for t (a sequence behind a
 *                      shared prefix starts at the prefix's length)
 *   key_bounds         [num_blocks][num_kv_heads][2][head_size] in dtype, or
 *                      NULL: per page and channel the largest ([0]) and the
 *                      smallest ([1]) key stored, as pa_select_blocks reads it
 *
 * The first rotary_dim elements of a head (a multiple of 16, at most
 * head_size) turn in pairs, in fp32 with one rounding to dtype:
 * y1 = x1 cos - x2 sin, y2 = x2 cos + x1 sin, the pairs being (j, j +
 * rotary_dim / 2) with interleaved = 0, (2j, 2j + 1) with 1; the rest and the
 * values are copied.  A page's bounds start anew with its first token (so they
 * are kept from there on or not at all) and otherwise only widen: tokens
 * overwritten later (rejected drafts) leave theirs in, so the bounds then still
 * hold but are wider than need be.  NaN keys are passed over.
 *
 * dtype as the caches; f32, bf16 and f16.  No two sequences may append to the
 * same page.  The workspace needs only its 256-byte status block (any
 * workspace of this library serves); bad tables, lengths, chunks or positions
 * are reported there as PA_ERR_DEVICE_BAD_INPUT, and nothing of the rows in
 * question is written. */
pa_status_t pa_append_kv(void *key_cache, void *value_cache, void *key_bounds,
                         void *query_out, const void *query, const void *key,
                         const void *value, long long query_stride,
                         long long key_stride, long long value_stride,
                         const float *cos_sin, const int32_t *positions,
                         const int32_t *block_tables, const int32_t *seq_lens,
                         const int32_t *q_start, int num_seqs, int num_rows,
                         int num_heads, int num_kv_heads, int head_size,
                         int num_blocks, int block_size, int max_blocks_per_seq,
                         int max_seq_len, int rotary_dim, int interleaved,
                         int max_position, int dtype, void *workspace,
                         size_t workspace_bytes, void *stream);

/* Decode attention over the blocks that a cheap score selects.
 *
 * For a query row and a KV head, with the pages' key bounds (pa_append_kv),
 * page j scores the sum over the group's heads of the largest q . k that its
 * bounds allow:
 *   score_j = sum_h sum_d max(q_hd max_jd, q_hd min_jd)
 *           = sum_d Q+_d max_jd + Q-_d min_jd,
 * Q+_d and Q-_d the sums of the heads' positive and negative q_hd (the second
 * form counts where a bound is infinite).  Of the pages that hold keys the
 * row sees, the first sink_blocks and the last recent_blocks are selected
 * always, the others by their score, ties to the lower page, num_selected in
 * all; every page if there are no more than that.
 * The selection is the one that exact scores give (nearly equal ones are
 * computed again to 45 bits of the sum's magnitude); a NaN score ranks lowest,
 * one beyond fp32's range as infinite.
 *
 * Rows: one a sequence (q_start NULL, num_rows = num_seqs, the row sees the
 * sequence's seq_lens keys), or chunks as in pa_chunks_forward (row i of a
 * chunk of n sees seq_lens - n + i + 1 keys; every row selects for itself).
 * Rows behind the last chunk, and rows of empty sequences, select nothing.
 *
 *   key_bounds  [num_blocks][num_kv_heads][2][head_size] (dtype), 16-byte
 *               aligned: largest, then smallest key a channel
 *   selected    int32 [num_rows][num_kv_heads][num_selected]: page numbers of
 *               the sequence, ascending, -1 behind the last
 * 0 <= sink_blocks, 1 <= recent_blocks, sink_blocks + recent_blocks <=
 * num_selected.  query, block_tables, seq_lens and the limits on sizes as in
 * pa_forward, f32 included, and max_seq_len at most 2^30; query contiguous [num_rows][num_heads][head_size].
 * The workspace holds pa_sparse_workspace_bytes(...) bytes, initialised once by
 * pa_workspace_init (one sized for the largest call serves smaller ones too);
 * partition_size is the one it was sized with, and the largest partition of
 * the attention (with few rows the library takes smaller ones).  A bad table
 * entry, length or chunk is reported as PA_ERR_DEVICE_BAD_INPUT: a page with a
 * bad entry scores lowest, a row with a bad length selects nothing. */
pa_status_t pa_select_blocks(int32_t *selected, const void *query,
                             const void *key_bounds,
                             const int32_t *block_tables,
                             const int32_t *seq_lens, const int32_t *q_start,
                             int num_seqs, int num_rows, int num_heads,
                             int num_kv_heads, int head_size, int num_blocks,
                             int block_size, int max_blocks_per_seq,
                             int max_seq_len, int num_selected,
                             int sink_blocks, int recent_blocks,
                             int partition_size, int dtype, void *workspace,
                             size_t workspace_bytes, void *stream);

/* Attention over selected blocks: out[r][h] = softmax over the keys that row
 * r sees in the blocks selected for (r, h's KV head), in the V1/V2 kernels.
 * With key_bounds, the blocks are selected as by pa_select_blocks in the same
 * call, and written to `selected` unless that is NULL.  With key_bounds NULL,
 * `selected` is read: any choice of the row's pages, ascending, -1 behind the
 * last (another order, or a page that the row does not see, is reported as
 * PA_ERR_DEVICE_BAD_INPUT, and the row's head group gets zeros); sink_blocks
 * and recent_blocks must still be valid but are not used.  Nothing selected:
 * zeros.  Other arguments as pa_select_blocks and pa_forward. */
pa_status_t pa_sparse_forward(void *out, int32_t *selected, const void *query,
                              const void *key_cache, const void *value_cache,
                              const void *key_bounds,
                              const int32_t *block_tables,
                              const int32_t *seq_lens, const int32_t *q_start,
                              int num_seqs, int num_rows, int num_heads,
                              int num_kv_heads, int head_size, int num_blocks,
                              int block_size, int max_blocks_per_seq,
                              int max_seq_len, int num_selected,
                              int sink_blocks, int recent_blocks, float scale,
                              int partition_size, int dtype, void *workspace,
                              size_t workspace_bytes, void *stream);

/* Bytes of workspace for the two calls above (0 on bad arguments). */
size_t pa_sparse_workspace_bytes(int num_rows, int num_heads, int num_kv_heads,
                                 int head_size, int block_size,
                                 int max_seq_len, int num_selected,
                                 int partition_size);

/* Decode attention for sequences that share prefixes (a system prompt, a
 * document, the prompt of several samples): sequence s attends to the
 * prefix_lens[g] tokens of its group's prefix and to its own seq_lens[s]
 * tokens,
 *   out[s][h] = softmax over both of (scale q[s][h] . K) @ V.
 * The prefix's keys and values are read once for all the rows (sequence, head)
 * of a group, as a matrix product on the tensor cores; the own tokens run as
 * in pa_v2_forward, and Phase 2 merges the partitions of both.  Keys carry
 * their positions' rotation already, so the own tokens are appended with the
 * prefix's length added to their positions (pa_append_kv).
 *
 *   prefix_tables  int32 [num_prefixes][max_prefix_blocks]: the prefixes'
 *                  pages, in the same caches
 *   prefix_lens    int32 [num_prefixes], each in [0, max_prefix_len], of any
 *                  length (the last page may be partly filled)
 *   prefix_start   int32 [num_prefixes + 1], non-decreasing, from 0 to
 *                  num_seqs: sequences prefix_start[g] .. prefix_start[g+1]-1
 *                  are group g; a group may be empty
 * block_tables and seq_lens hold the own tokens only, with max_seq_len their
 * bound (0 if no sequence has any).  Sequences with no tokens at all get
 * zeros.  bf16 and f16 (PA_ERR_UNSUPPORTED for f32); max_seq_len and
 * max_prefix_len at most 2^30; the other arguments and limits as
 * pa_v2_forward.  The workspace holds pa_prefix_workspace_bytes(...)
 * bytes, initialised once by pa_workspace_init (any workspace that is large
 * enough serves calls of any shape, one after another).  The prefix is split as
 * these sizes and the workspace's suggest, and the splits' sums are rounded
 * apart: the same call on workspaces of other sizes may differ in last bits.
 * A max_prefix_len far above the longest prefix makes fewer and longer items
 * of it than the GPU has room for: give the batch's own where it is known.
 * Bad tables, lengths or groups are reported as PA_ERR_DEVICE_BAD_INPUT; the
 * rows in question (with starts out of order, any row) then hold no meaningful
 * values.  opts as in pa_forward (variant V2 or auto; no fused combine, no
 * CUDA-core path). */
pa_status_t pa_prefix_forward(void *out, const void *query,
                              const void *key_cache, const void *value_cache,
                              const int32_t *block_tables,
                              const int32_t *seq_lens,
                              const int32_t *prefix_tables,
                              const int32_t *prefix_lens,
                              const int32_t *prefix_start, int num_seqs,
                              int num_prefixes, int num_heads,
                              int num_kv_heads, int head_size, int num_blocks,
                              int block_size, int max_blocks_per_seq,
                              int max_prefix_blocks, int max_seq_len,
                              int max_prefix_len, float scale,
                              int partition_size, int dtype, void *workspace,
                              size_t workspace_bytes, void *stream,
                              const pa_options_t *opts);

/* Bytes of workspace for pa_prefix_forward (0 on bad arguments): as
 * pa_workspace_bytes with slots for the prefix's splits behind every row's own
 * partitions.  A workspace for the largest num_seqs, num_prefixes, max_seq_len
 * and max_prefix_len serves calls with smaller ones (the other sizes alike):
 * they take as many splits as it holds. */
size_t pa_prefix_workspace_bytes(int num_seqs, int num_prefixes, int num_heads,
                                 int num_kv_heads, int head_size,
                                 int max_seq_len, int max_prefix_len,
                                 int partition_size);

/* Append new keys and values to a paged cache that holds them in 4 bits.
 *
 * Of every 64 elements of a head (a group) the cache holds the lowest value and
 * a step, both f16, and for each element a code of 4 bits:
 *   lo   = f16(min x)                 (no further from 0 than f16's largest, 65504)
 *   step = f16((max x - lo) * (1/15)) (the same)
 *   code = (x - lo) * (1 / step) rounded to even, 0 .. 15 (0 where step is 0)
 * in fp32, each operation rounded by itself; a code stands for lo + code * step.
 * NaN is coded as the group's lowest value.
 *
 *   key_cache, value_cache    uint8 [num_blocks][num_kv_heads][block_size]
 *                             [head_size / 2]: element 2i of a head in the low
 *                             half of byte i, 2i + 1 in the high half
 *   key_scales, value_scales  f16 [num_blocks][num_kv_heads][block_size]
 *                             [head_size / 64][2]: lo, step
 * A token takes 9/16 of a byte an element (72 bytes at head_size 128 for a head),
 * scales included.  Keys are rotated and rounded to dtype as by pa_append_kv
 * (with the three operations of each element rounded apart), then coded; query
 * is rotated into query_out.  key_out, value_out [num_rows][num_kv_heads]
 * [head_size] (dtype), or NULL, receive what the appended codes stand for, for
 * attention among a prompt's own tokens that agrees with later decode steps; they
 * may be key and value themselves where those are contiguous (other strides in
 * place are PA_ERR_INVALID_ARG).
 *
 * Rows, q_start, seq_lens, positions, strides, rotation, the workspace and bad
 * data as in pa_append_kv; padding rows leave query_out, key_out and value_out
 * as they were.  bf16 and f16 (PA_ERR_UNSUPPORTED for f32); caches and scales
 * 16-byte aligned.  Two rows never share a byte, so any rows may be appended at
 * once. */
pa_status_t pa_q4_append(void *key_cache, void *value_cache, void *key_scales,
                         void *value_scales, void *query_out, void *key_out,
                         void *value_out, const void *query, const void *key,
                         const void *value, long long query_stride,
                         long long key_stride, long long value_stride,
                         const float *cos_sin, const int32_t *positions,
                         const int32_t *block_tables, const int32_t *seq_lens,
                         const int32_t *q_start, int num_seqs, int num_rows,
                         int num_heads, int num_kv_heads, int head_size,
                         int num_blocks, int block_size, int max_blocks_per_seq,
                         int max_seq_len, int rotary_dim, int interleaved,
                         int max_position, int dtype, void *workspace,
                         size_t workspace_bytes, void *stream);

/* Decode attention over a cache in 4 bits: out[r][h] = softmax over the keys
 * that row r sees of (scale q . K) @ V, with the values that the codes stand
 * for, accumulated in fp32.  Rows: one a sequence (q_start NULL, num_rows =
 * num_seqs, the row sees the sequence's seq_lens keys; an empty sequence gets
 * zeros), or chunks of a sequence's last tokens as in pa_chunks_forward, of any
 * lengths (rows behind the last chunk are left as they were).  Every 16 /
 * (num_heads / num_kv_heads) tokens of a chunk read the keys once more: made for
 * decode steps and a few draft tokens, right for pieces of prompts, but slower there
 * than pa_chunks_forward over 16-bit keys and values (8 sequences of 8192 tokens,
 * 32/4 heads of 128, GB300: 5 tokens each 62 against 56 us, 64 tokens 388 against
 * 167, 256 tokens 1430 against 365).
 *
 * The work is cut into equal shares of keys whatever the lengths are, so there
 * is no partition size to choose, and a workspace of pa_q4_workspace_bytes(
 * head_size) bytes, initialised once by pa_workspace_init, serves calls of any
 * batch, one after another.  Which keys share a partial sum follows from all the
 * lengths and the GPU's SM count, so last bits of a sequence's output may differ
 * between batches.  query and out contiguous [num_rows][num_heads][head_size];
 * bf16 and f16 (PA_ERR_UNSUPPORTED for f32); max_seq_len at most 2^30; the
 * other arguments and limits as pa_forward.  Scales must be finite (a step may be
 * negative: a code stands for lo + code * step).  A bad table entry, length or
 * chunk is reported as PA_ERR_DEVICE_BAD_INPUT; the rows in question then hold no
 * meaningful values (zeros for a bad length without q_start), or are left as they
 * were (a bad chunk; rows that starts out of order give to two sequences hold
 * either's). */
pa_status_t pa_q4_forward(void *out, const void *query, const void *key_cache,
                          const void *value_cache, const void *key_scales,
                          const void *value_scales, const int32_t *block_tables,
                          const int32_t *seq_lens, const int32_t *q_start,
                          int num_seqs, int num_rows, int num_heads,
                          int num_kv_heads, int head_size, int num_blocks,
                          int block_size, int max_blocks_per_seq, int max_seq_len,
                          float scale, int dtype, void *workspace,
                          size_t workspace_bytes, void *stream);

/* Bytes of workspace for pa_q4_forward, any batch (0 on a bad head size): 41, 81
 * and 161 MB at head sizes 64, 128 and 256. */
size_t pa_q4_workspace_bytes(int head_size);

/* Append to a paged cache of shared latents.  A token's row is [latent_dim |
 * rope_dim]: the latent vector that the keys and values of every head are
 * projections of, and one key part that carries the position, shared by all
 * heads.
 *
 *   cache        [num_blocks][block_size][latent_dim + rope_dim]
 *   latent       [num_rows][latent_dim], rows latent_stride elements apart
 *   rope_key     [num_rows][rope_dim], rows rope_key_stride apart (both may be
 *                slices of one projection's output)
 *   norm_weight  [latent_dim] or NULL (the latent is stored as it is): the
 *                latent is x * (mean(x^2) + eps)^-1/2 * norm_weight
 *   query_rope   [num_rows][num_heads][rope_dim] or NULL, heads
 *                query_head_stride and rows query_stride apart (either the
 *                further, no two overlapping): the queries' parts that carry the
 *                position; rotated into
 *   query        [num_rows][num_heads][latent_dim + rope_dim], contiguous: the
 *                last rope_dim elements of every head; the first latent_dim,
 *                the queries through the keys' up-projection, are the caller's
 *                and are not touched.  query_rope may be those last elements
 *                themselves; words of it that are written for another head or
 *                row are PA_ERR_INVALID_ARG
 *
 * All of rope_dim turns, in pairs as interleaved says; everything in fp32 with
 * one rounding to dtype.  cos_sin, positions, rows, q_start, seq_lens and bad
 * data as in pa_append_kv; strides in multiples of 8, pointers 16-byte aligned;
 * latent_dim 256 or 512, rope_dim 64, num_heads at most 128, block_size 8, 16,
 * 32 or 64; bf16 and f16 (PA_ERR_UNSUPPORTED otherwise).  eps >= 0. */
pa_status_t pa_latent_append(void *cache, void *query, const void *query_rope,
                             const void *latent, const void *rope_key,
                             const void *norm_weight, float eps,
                             long long query_stride, long long query_head_stride,
                             long long latent_stride, long long rope_key_stride,
                             const float *cos_sin, const int32_t *positions,
                             const int32_t *block_tables,
                             const int32_t *seq_lens, const int32_t *q_start,
                             int num_seqs, int num_rows, int num_heads,
                             int latent_dim, int rope_dim, int num_blocks,
                             int block_size, int max_blocks_per_seq,
                             int max_seq_len, int interleaved, int max_position,
                             int dtype, void *workspace, size_t workspace_bytes,
                             void *stream);

/* Decode attention over a cache of shared latents, in the absorbed form: with
 * c_t and r_t the two parts of a token's row and q = [q_c | q_r] a head's query
 * (q_c having gone through the keys' up-projection),
 *   out[r][h] = sum_t softmax_t(scale (q_c . c_t + q_r . r_t)) c_t,
 * a vector of latent_dim that the caller's value up-projection takes on.
 *
 *   query  [num_rows][num_heads][latent_dim + rope_dim]
 *   out    [num_rows][num_heads][latent_dim]
 * Rows as in pa_q4_forward: one a sequence (an empty sequence gets zeros), or
 * chunks of a sequence's last tokens (rows behind the last chunk are left as
 * they were).  Shares of the work, last bits, the workspace (of
 * pa_latent_workspace_bytes(latent_dim) bytes, for any batch) and bad data as
 * there; limits as in pa_latent_append, max_seq_len at most 2^30.  Keys that a
 * row does not see because they are later tokens of its chunk must be finite.
 * opts (or NULL): debug_flags (PA_DEBUG_STALL_CONSUMERS) and wait_limit_ns. */
pa_status_t pa_latent_forward(void *out, const void *query, const void *cache,
                              const int32_t *block_tables,
                              const int32_t *seq_lens, const int32_t *q_start,
                              int num_seqs, int num_rows, int num_heads,
                              int latent_dim, int rope_dim, int num_blocks,
                              int block_size, int max_blocks_per_seq,
                              int max_seq_len, float scale, int dtype,
                              void *workspace, size_t workspace_bytes,
                              void *stream, const pa_options_t *opts);

/* Bytes of workspace for pa_latent_forward, any batch (0 on a bad latent_dim): 25
 * and 51 MB at latent_dim 256 and 512. */
size_t pa_latent_workspace_bytes(int latent_dim);

/* The four calls above with their arguments in an array of 64-bit words, in
 * order (pointers and integers as they are, floats as doubles), for bindings
 * that pay for every argument of a foreign call: `call` is a pa_call_t.  The
 * words are read before the call returns.  An int that does not fit 32 bits is
 * PA_ERR_INVALID_ARG. */
typedef enum {
  PA_CALL_Q4_APPEND = 0,
  PA_CALL_Q4_FORWARD = 1,
  PA_CALL_LATENT_APPEND = 2,
  PA_CALL_LATENT_FORWARD = 3
} pa_call_t;
pa_status_t pa_call(int call, const void *words);

/* Host heuristic: 1 if V2 should serve this batch on a GPU with sm_count
 * SMs, 0 for V1.  The pages switch on sequence length alone: the commit note
 * for computility-run.yaml (project_6, commit a2a5dd8) lists the decode path
 * as V1 up to 8192 tokens and V2 above, and GROUND_TRUTH_STATUS_v2.md
 * (project_6_baseline5, section "路径 3") says the partitioning should follow
 * the SM count.  Here: V1 when every sequence fits in one partition;
 * otherwise V2 unless the batch alone fills the GPU several times over with
 * short sequences (the length bound and the fill factor are set from
 * measurements on GB300). */
int pa_choose_v2(int num_seqs, int num_kv_heads, int max_seq_len,
                 int partition_size, int sm_count);

/* The same heuristic for query chunks (pa_chunks_forward with the automatic
 * variant): 1 for V2, 0 for V1, for chunks of at most max_chunk tokens.  V1
 * when every sequence fits in one partition; with at most 8 (token, head)
 * rows per KV head, pa_choose_v2's answer; otherwise V1 when the batch has
 * at least 8 work items per SM (4 on the tcgen05 kernel), counting an item
 * per (sequence, KV head) and row group as the chunk kernels cut them (128
 * rows on the tcgen05 kernel: more than 16 rows per KV head at head_size
 * 128; 64 on the row-owning kernel: more than 32 rows per KV head at
 * head_size 64, a group dividing 64; else 16), V2 below (measured on GB300).
 * Pure host arithmetic on its arguments. */
int pa_choose_v2_chunks(int num_seqs, int num_heads, int num_kv_heads, int head_size,
                        int max_chunk, int max_seq_len, int partition_size, int sm_count);

/* Synchronise `stream`, return the workspace's status word as a pa_status_t
 * (PA_OK if no kernel reported a problem) and reset it to 0.  The pages have
 * no counterpart: this is how the library reports data errors its kernels
 * find (a block-table entry outside [0, num_blocks), a length outside
 * [0, max_seq_len]) or a bounded device wait that ran out, since kernels
 * never trap.  Not for use inside a stream capture (it synchronises). */
pa_status_t pa_read_device_status(void *workspace, void *stream);

/* Static English text for a status code. */
const char *pa_status_string(int status);

/* Text of the last CUDA error seen by this thread inside the library. */
const char *pa_last_cuda_error(void);

/* Library version, major * 10000 + minor * 100 + patch. */
int pa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PA_H_ */
