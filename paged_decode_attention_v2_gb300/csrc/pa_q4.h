// The cache in 4 bits: what the append and the attention share.
//
// Every 64 elements of a head (a group) have a lowest value and a step in f16;
// an element is a code c of 0 .. 15, two a byte (element 2i in the low half of
// byte i), and stands for lowest + c * step.
#pragma once

#include <stdint.h>

namespace pa {

constexpr int kQ4Group = 64;

struct Q4Params {
  const uint8_t *key_codes, *value_codes;  // [num_blocks][Hkv][bs][D / 2]
  const void *key_scales, *value_scales;   // half2 [num_blocks][Hkv][bs][D / 64]: lowest, step
  const void *query;                       // [rows][H][D]
  void *out;
  const int32_t *block_tables, *seq_lens, *q_start;
  int *status;
  int num_seqs, num_rows, num_heads, num_kv_heads, group, num_blocks;
  int block_size, log2_block_size, max_blocks_per_seq, max_seq_len;
  int chunk_tokens;  // query tokens of a unit
  float scale_log2;  // scale * log2(e)
};

}  // namespace pa
