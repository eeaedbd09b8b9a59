// Launch parameters of the operators around the attention kernels: appending
// to the paged cache, shared prefixes, block selection.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pa {

constexpr int kAppendMaxRows = 4;  // rows of a CTA

struct AppendParams {
  void *key_cache, *value_cache;  // [num_blocks][Hkv][bs][D]
  void *key_bounds;               // [num_blocks][Hkv][2][D] or null
  void *query_out;                // [rows][H][D] or null
  const void *query, *key, *value;  // [rows][heads][D], row strides below (elements)
  long long query_stride, key_stride, value_stride;
  const float *cos_sin;      // [max_position][rotary_dim]: cosines, then sines
  const int32_t *positions;  // [rows], or null: the token's place in its sequence
  const int32_t *block_tables, *seq_lens, *q_start;
  int *status;
  int num_seqs, num_rows, num_heads, num_kv_heads, num_blocks;
  int block_size, log2_block_size, max_blocks_per_seq, max_seq_len;
  int rotary_dim, interleaved, max_position;
  int tile_rows;  // rows of a CTA
};

// The block of the view in which every (row, KV head) is a sequence of one KV
// head: cache [num_blocks * Hkv][1][bs][D].  A bad entry stays out of range,
// for the attention kernels to report.
__host__ __device__ __forceinline__ int view_block(int blk, int kv_head, int num_kv_heads,
                                                   int num_blocks) {
  return (unsigned)blk < (unsigned)num_blocks ? blk * num_kv_heads + kv_head : -1;
}

// The longest prefix, and the longest sequence beside one or with selected
// blocks: lengths stay 31-bit numbers with a split or a page added (and no
// cache that fits the GPU holds more).
constexpr int kMaxTokens = 1 << 30;

// Every split is one more partial of every row, and the plan tries each number
// of them on the host.  (With one KV head and one tile of rows, 64 CTAs are
// fewer than the SMs; more splits there are left to be measured.)
constexpr int kMaxPrefixSplits = 64;
constexpr int kPrefixSms = 152;  // what the splits are planned for
constexpr int kPrefixDebugStall = 1;  // PA_DEBUG_STALL_CONSUMERS

struct PrefixParams {
  const void *query;                   // [B][H][D]
  const int32_t *prefix_tables;        // [num_prefixes][max_prefix_blocks]
  const int32_t *prefix_lens;          // [num_prefixes]
  const int32_t *prefix_start;         // [num_prefixes + 1]: sequences of each group
  const int32_t *seq_lens;             // [B]: own keys
  float *max_logits, *exp_sums, *tmp_out;  // [B][H][max_parts](, [D])
  int *row_limit;                      // [B]: partitions x partition_size, for Phase 2
  int *status;
  int *sched;  // the own tokens' count of items, if they run beside (else null)
  int num_seqs, num_prefixes, num_heads, num_kv_heads, group, num_blocks;
  int block_size, log2_block_size, max_prefix_blocks, max_prefix_len;
  int max_seq_len, partition_size, max_parts;
  uint64_t group_magic;  // ceil(2^36 / group): x / group for x < 2^28 is x * it >> 36
  int split_tokens;  // keys of a split, a multiple of the kernel's stage
  int debug_flags;
  float scale_log2;  // scale * log2(e)
  uint64_t wait_limit_ns;
};

struct PrefixKernelInfo {
  const void *fn;
  int threads;
  size_t smem;
  int tile_rows;   // rows of an item
  int stage_keys;  // keys of a stage
};
PrefixKernelInfo prefix_kernel(int dtype_bf16, int head_size);
void prefix_plan(int num_seqs, int num_prefixes, int num_heads, int num_kv_heads, int head_size,
                 int max_seq_len, int max_prefix_len, int partition_size, int most_splits,
                 int *split_tokens, int *max_splits);

// An item scored and selected from in one CTA, or scored by several and
// selected from in a second launch.
enum SelectMode { kSelBoth, kSelScore, kSelPick };

struct SelectParams {
  const void *query;       // [rows][H][D]
  const void *key_bounds;  // [num_blocks][Hkv][2][D]
  const int32_t *block_tables, *seq_lens, *q_start;
  int32_t *selected;       // [rows][Hkv][num_selected] or null
  const int32_t *given;    // a given selection instead
  int32_t *table, *lens;   // the view's block table and lengths, or null
  float *sizes;            // [rows * Hkv][chunks] largest sum of magnitudes
  uint32_t *keys;          // [rows * Hkv][max_pages] scores as ordered integers
  uint64_t *fine;          // [rows * Hkv][max_pages] keys of scores in pairs, where needed
  int *status;
  int num_seqs, num_rows, num_heads, num_kv_heads, num_blocks;
  int block_size, log2_block_size, max_blocks_per_seq, max_seq_len, max_pages;
  int num_selected, sinks, recent;
  int mode;                 // SelectMode
  int chunks, chunk_pages;  // CTAs that score an item, pages of each
  int smem_pages;           // keys that the shared memory holds
};

}  // namespace pa
