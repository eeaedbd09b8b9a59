// pa_q4_append: new keys and values into a cache in 4 bits (pa_q4.h), keys and
// queries rotated on the way as by pa_append_kv.
//
// Of every 64 elements, in fp32 with each operation rounded by itself (so that
// plain tensor operations give the same bits):
//   lo   = f16(min x),  step = f16((max x - lo) / 15),  both within f16's range
//   code = round((x - lo) / step), 0 .. 15;  it stands for lo + code step.
// A key is rounded to the inputs' type after its rotation, as it would be
// stored, then coded.
//
// A lane has 16 elements of a head, four lanes a group, so a group's range
// takes two exchanges.  Rotated halves may lie in two groups: such a head goes
// through shared memory, a warp's own kilobyte.  A CTA takes up to four rows,
// whose heads (keys, values, queries) its warps take in turn.
//
// Bound, on GB300: a decode step is one launch and a chain of dependent loads
// (256 sequences 3.8 us); 8947 rows of prompts, 16/2 heads, D 256, 191 MB take
// 37 us (5.1 TB/s, 28.5 at the copy rate), next to the issue slots.
#include <math_constants.h>

#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_ops.h"
#include "pa_q4.h"
#include "pa_rows.cuh"

namespace pa {
namespace {

constexpr int kQ4AppendThreads = 128;
constexpr int kQ4AppendWarps = kQ4AppendThreads / 32;

struct Q4AppendParams {
  uint8_t *key_codes, *value_codes;  // [num_blocks][Hkv][bs][D / 2]
  __half2 *key_scales, *value_scales;  // [num_blocks][Hkv][bs][D / 64]
  void *query_out, *key_out, *value_out;  // contiguous rows, or null
  const void *query, *key, *value;
  long long query_stride, key_stride, value_stride;
  const float *cos_sin;
  const int32_t *positions, *block_tables, *seq_lens, *q_start;
  int *status;
  int num_seqs, num_rows, num_heads, num_kv_heads, num_blocks;
  int block_size, log2_block_size, max_blocks_per_seq, max_seq_len;
  int rotary_dim, interleaved, max_position;
  int tile_rows;
};

// 16 elements of a group whose other 48 are in the lanes next to this one: its
// codes (8 bytes), the group's scales, and the values that the codes stand for.
__device__ __forceinline__ uint2 quantise(float (&x)[16], __half2 &scales) {
  float mn = CUDART_INF_F, mx = -CUDART_INF_F;
#pragma unroll
  for (int i = 0; i < 16; ++i) mn = fminf(mn, x[i]), mx = fmaxf(mx, x[i]);  // (NaN passed over)
#pragma unroll
  for (int d = 1; d < 4; d <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, d));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
  }
  if (mn > mx) mn = mx = 0.f;  // no number in the group
  constexpr float kMost = 65504.f;
  const __half lo_h = __float2half_rn(fminf(fmaxf(mn, -kMost), kMost));
  const float lo = __half2float(lo_h);
  const float range = __fmul_rn(__fsub_rn(mx, lo), 1.f / 15.f);
  const __half step_h = __float2half_rn(fminf(fmaxf(range, 0.f), kMost));
  const float step = __half2float(step_h);
  const float inv = step > 0.f ? __frcp_rn(step) : 0.f;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float c = fminf(fmaxf(__fmul_rn(__fsub_rn(x[i], lo), inv), 0.f), 15.f);  // (NaN: 0)
    // 1.5 2^23 more: rounded to even, the code in the lowest bits (conversions run at a
    // quarter of the rate)
    const float r = __fadd_rn(c, 12582912.f);
    w[i >> 3] |= (__float_as_uint(r) & 15u) << (4 * (i & 7));
    x[i] = __fadd_rn(lo, __fmul_rn(__fsub_rn(r, 12582912.f), step));
  }
  scales = __halves2half2(lo_h, step_h);
  return make_uint2(w[0], w[1]);
}

}  // namespace

template <typename T, int D>
__global__ void __launch_bounds__(kQ4AppendThreads, 6)
    pa_q4_append_kernel(const __grid_constant__ Q4AppendParams p) {
  constexpr int N = Chunk2<T>::N;     // elements of a 16-byte chunk
  constexpr int UNITS = D / (2 * N);  // lanes of a head
  constexpr int HEADS = 32 / UNITS;   // a warp's at a time
  __shared__ int s_pos[kAppendMaxRows];      // -1: no work for the row
  __shared__ size_t s_slot[kAppendMaxRows];  // (page * Hkv) * bs + place in it
  __shared__ uint4 s_turn[kQ4AppendWarps][64];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * p.tile_rows;
  const int rows = min(p.tile_rows, p.num_rows - row0);
  const bool il = p.interleaved != 0;
  const int rot = p.rotary_dim / (2 * N), half = p.rotary_dim / 2;

  // the rows on their way to L2 while they are located
  {
    const int kvl = p.num_kv_heads * D * (int)sizeof(T) / 128, ql = p.query ? p.num_heads * D * (int)sizeof(T) / 128 : 0;
    const int lines = 2 * kvl + ql;
    for (int i = threadIdx.x; i < rows * lines; i += kQ4AppendThreads) {
      const int r = i / lines, l = i - r * lines;
      const T *src = l < kvl       ? static_cast<const T *>(p.key) + (row0 + r) * p.key_stride
                     : l < 2 * kvl ? static_cast<const T *>(p.value) + (row0 + r) * p.value_stride
                                   : static_cast<const T *>(p.query) + (row0 + r) * p.query_stride;
      prefetch_l2(reinterpret_cast<const char *>(src) + (l < kvl ? l : l < 2 * kvl ? l - kvl : l - 2 * kvl) * 128);
    }
  }
  pdl_wait_primary();
  pdl_launch_dependents();
  if (warp < rows) {
    RowInfo o;
    int pos = -1;
    if (locate_row(p, row0 + warp, o)) {
      pos = row_position(p, row0 + warp, o.tok);
      if ((unsigned)o.blk >= (unsigned)p.num_blocks) {  // nothing of the row is written
        pos = -1;
        if (lane == 0) report(p.status, kStatusBadInput);
      }
    }
    if (lane == 0) {
      s_pos[warp] = pos;
      s_slot[warp] = pos < 0 ? 0 : (size_t)o.blk * p.num_kv_heads * p.block_size + (o.tok & (p.block_size - 1));
    }
  }
  __syncthreads();

  const int u = lane % UNITS;
  const int per_row = 2 * p.num_kv_heads + (p.query ? p.num_heads : 0);
  for (int v0 = warp * HEADS; v0 < rows * per_row; v0 += kQ4AppendWarps * HEADS) {
    const int v = v0 + lane / UNITS;
    const int lr = min(v / per_row, rows - 1), hd = v - lr * per_row, row = row0 + lr;
    const int pos = s_pos[lr];
    const bool live = v < rows * per_row && pos >= 0;
    // keys, then values, then queries of a row
    const int kind = hd < p.num_kv_heads ? 0 : hd < 2 * p.num_kv_heads ? 1 : 2;
    const int h = kind == 0 ? hd : kind == 1 ? hd - p.num_kv_heads : hd - 2 * p.num_kv_heads;
    int ca = 2 * u, cb = 2 * u + 1;
    if (kind != 1) unit_chunks(u, rot, il, ca, cb);
    Chunk2<T> x{make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
    if (live) {
      // (query_out may be the query: no read-only path)
      const T *from = kind == 0   ? static_cast<const T *>(p.key) + row * p.key_stride
                      : kind == 1 ? static_cast<const T *>(p.value) + row * p.value_stride
                                  : static_cast<const T *>(p.query) + row * p.query_stride;
      const uint4 *src = reinterpret_cast<const uint4 *>(from + (size_t)h * D);
      x.a = src[ca];
      x.b = src[cb];
      if (kind != 1 && u < rot) {
        Angles<N> r;
        r.load(p.cos_sin + (size_t)pos * p.rotary_dim, u, half);
        rotate_unit<T, true>(x, r, il);
      }
      if (kind == 2) {
        uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(p.query_out) + ((size_t)row * p.num_heads + h) * D);
        dst[ca] = x.a;
        dst[cb] = x.b;
      }
    }
    if (!__any_sync(0xffffffffu, live && kind != 2)) continue;
    if (!il && rot > 0) {  // halves of pairs back to their places
      uint4 *turn = s_turn[warp] + (lane - u) * 2;
      turn[ca] = x.a;
      turn[cb] = x.b;
      __syncwarp();
      x.a = turn[2 * u];
      x.b = turn[2 * u + 1];
      __syncwarp();
    }
    float f[16], f8[8];
    widen<T>(x.a, f8);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = f8[i];
    widen<T>(x.b, f8);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[8 + i] = f8[i];
    __half2 scales;
    const uint2 codes = quantise(f, scales);
    if (live && kind != 2) {
      const size_t slot = s_slot[lr] + (size_t)h * p.block_size;
      *reinterpret_cast<uint2 *>((kind ? p.value_codes : p.key_codes) + slot * (D / 2) + 8 * u) = codes;
      if ((u & 3) == 0) (kind ? p.value_scales : p.key_scales)[slot * (D / kQ4Group) + (u >> 2)] = scales;
      T *out = static_cast<T *>(kind ? p.value_out : p.key_out);
      if (out) {
        uint4 *dst = reinterpret_cast<uint4 *>(out + ((size_t)row * p.num_kv_heads + h) * D) + 2 * u;
#pragma unroll
        for (int i = 0; i < 8; ++i) f8[i] = f[i];
        dst[0] = narrow<T>(f8);
#pragma unroll
        for (int i = 0; i < 8; ++i) f8[i] = f[8 + i];
        dst[1] = narrow<T>(f8);
      }
    }
  }
}

namespace {

template <typename T>
const void *q4_append_pick(int head_size) {
  switch (head_size) {
    case 64: return reinterpret_cast<const void *>(&pa_q4_append_kernel<T, 64>);
    case 128: return reinterpret_cast<const void *>(&pa_q4_append_kernel<T, 128>);
    case 256: return reinterpret_cast<const void *>(&pa_q4_append_kernel<T, 256>);
  }
  return nullptr;
}

}  // namespace
}  // namespace pa

extern "C" pa_status_t pa_q4_append(
    void *key_cache, void *value_cache, void *key_scales, void *value_scales, void *query_out,
    void *key_out, void *value_out, const void *query, const void *key, const void *value,
    long long query_stride, long long key_stride, long long value_stride, const float *cos_sin,
    const int32_t *positions, const int32_t *block_tables, const int32_t *seq_lens,
    const int32_t *q_start, int num_seqs, int num_rows, int num_heads, int num_kv_heads,
    int head_size, int num_blocks, int block_size, int max_blocks_per_seq, int max_seq_len,
    int rotary_dim, int interleaved, int max_position, int dtype, void *workspace,
    size_t workspace_bytes, void *stream) {
  using namespace pa;
  pa_status_t st = host_check_cache(dtype, num_heads, num_kv_heads, head_size, num_blocks,
                                    block_size, max_blocks_per_seq, max_seq_len);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || num_rows < 0 || (!q_start && num_rows != num_seqs)) return PA_ERR_INVALID_ARG;
  if (rotary_dim < 0 || rotary_dim > head_size || rotary_dim % 16) return PA_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return PA_ERR_INVALID_ARG;
  if (dtype == PA_DTYPE_F32) return PA_ERR_UNSUPPORTED;  // as the attention over such a cache
  if (num_rows == 0 || num_seqs == 0) return PA_OK;      // (empty tensors have no address)
  if (rotary_dim > 0 && (!cos_sin || max_position < 1)) return PA_ERR_INVALID_ARG;
  if ((query == nullptr) != (query_out == nullptr)) return PA_ERR_INVALID_ARG;
  if (!key_cache || !value_cache || !key_scales || !value_scales || !key || !value ||
      !block_tables || !seq_lens || !workspace)
    return PA_ERR_INVALID_ARG;
  const void *wide[] = {key_cache, value_cache, key_scales, value_scales, query_out, key_out,
                        value_out, query,       key,        value,        cos_sin};
  for (const void *q : wide)
    if (!host_aligned(q, 16)) return PA_ERR_INVALID_ARG;
  const void *ints[] = {positions, block_tables, seq_lens, q_start};
  for (const void *q : ints)
    if (!host_aligned(q, 4)) return PA_ERR_INVALID_ARG;
  if (!host_aligned(workspace, 256)) return PA_ERR_INVALID_ARG;
  const long long kv_row = (long long)num_kv_heads * head_size;
  if (key_stride < kv_row || value_stride < kv_row || key_stride % 8 || value_stride % 8)
    return PA_ERR_INVALID_ARG;
  if (query && (query_stride < (long long)num_heads * head_size || query_stride % 8))
    return PA_ERR_INVALID_ARG;
  // in place only row by row: another stride would write rows not yet read
  if (query && query == query_out && query_stride != (long long)num_heads * head_size)
    return PA_ERR_INVALID_ARG;
  if (workspace_bytes < (size_t)kStatusBytes) return PA_ERR_WORKSPACE_TOO_SMALL;
  if (num_rows > 1 && ((key == key_out && key_stride != kv_row) || (value == value_out && value_stride != kv_row)))
    return PA_ERR_INVALID_ARG;

  Q4AppendParams p{};
  p.key_codes = static_cast<uint8_t *>(key_cache);
  p.value_codes = static_cast<uint8_t *>(value_cache);
  p.key_scales = static_cast<__half2 *>(key_scales);
  p.value_scales = static_cast<__half2 *>(value_scales);
  p.query_out = query_out;
  p.key_out = key_out;
  p.value_out = value_out;
  p.query = query;
  p.key = key;
  p.value = value;
  p.query_stride = query_stride;
  p.key_stride = key_stride;
  p.value_stride = value_stride;
  p.cos_sin = cos_sin;
  p.positions = positions;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.q_start = q_start;
  p.status = static_cast<int *>(workspace);
  p.num_seqs = num_seqs;
  p.num_rows = num_rows;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  while ((1 << p.log2_block_size) < block_size) ++p.log2_block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_seq_len = max_seq_len;
  p.rotary_dim = rotary_dim;
  p.interleaved = interleaved;
  p.max_position = max_position;
  int sms = 0;
  st = host_sm_count(&sms);
  if (st != PA_OK) return st;
  // rows a CTA: two of 8 KB or more, four of less (8947 prompt rows, f16: 10 KB each 37.3
  // and 41.2 us with two and four, 20 KB 72.7 and 82.5, 3 KB 19.3 and 16.4)
  const long long row_bytes = 2ll * head_size * (2 * num_kv_heads + (query ? num_heads : 0));
  const int most = row_bytes >= 8192 ? 2 : kAppendMaxRows;
  p.tile_rows = 1;
  while (p.tile_rows < most && num_rows > 4ll * sms * p.tile_rows) p.tile_rows *= 2;
  const void *fn = dtype == PA_DTYPE_BF16 ? q4_append_pick<__nv_bfloat16>(head_size)
                                          : q4_append_pick<__half>(head_size);
  void *args[1] = {&p};
  const unsigned grid = (unsigned)(((long long)num_rows + p.tile_rows - 1) / p.tile_rows);
  return host_launch(fn, grid, 1, kQ4AppendThreads, 0, stream, args, "launch 4-bit append kernel");
}
