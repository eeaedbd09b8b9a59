// Launch parameters of the operators around the attention kernels: appending
// to the paged cache, shared prefixes, block selection.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

constexpr int kAppendMaxRows = 32;  // rows of a CTA's tile, one lane each

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

}  // namespace pa
