// pa_append_kv: new keys and values into the paged cache, the position
// rotation of keys (and queries) and the pages' key bounds on the way.
//
// Row r of the inputs is token t = L - n + i of its sequence (i-th row of a
// chunk of the sequence's last n tokens).  With c, s the cosine and sine of
// its position's angles, a rotated pair is
//   y1 = x1 c - x2 s,   y2 = x2 c + x1 s
// in fp32, rounded once to the cache's type.  A page's bounds are, channel by
// channel, the largest and smallest key stored in it.
//
// A thread's unit of work is two 16-byte chunks of a head that hold both
// halves of its pairs (half-split: chunk u and the one rotary_dim / 2 further
// on; adjacent pairs: chunks 2u and 2u + 1), so no pair crosses threads.  A
// CTA takes up to four rows: all its threads rotate the rows' queries, and its
// warps take the (page, KV head) pairs whose first appended token is one of
// its rows.  So exactly one warp touches a page's bounds: they need no
// atomics, and the result does not depend on the order of anything.
//
// Bound: bytes (each input read once, each output written once): 8947 ragged
// prompt rows (32/4 heads, D 128, bf16, with bounds), 189 MB, take 34.9 us,
// 5.4 TB/s, 0.80 of the copy peak.  A decode step's bytes are a few MB or
// less; there the launch and one dependent chain of loads (lengths, table,
// angles) are all there is: 3.2 us for one row, 3.9 us for 256, one launch after
// another.  So what can be is read before a row is located: its queries, and
// its keys and values as far as L2.  A row is found in q_start by a warp, 32
// entries at a time.
#include <math_constants.h>

#include <type_traits>

#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_ops.h"
#include "pa_rows.cuh"

namespace pa {
namespace {

constexpr int kAppendThreads = 128;
constexpr int kAppendWarps = kAppendThreads / 32;
constexpr int kAppendHeads = 4;  // of a row's queries, a thread

// Element-wise maximum (minimum) of the words of stored keys: one fp32 value
// or two 16-bit ones a word, NaN passed over.
template <typename T>
__device__ __forceinline__ uint32_t word_max(uint32_t a, uint32_t b) {
  if constexpr (sizeof(T) == 4) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  } else {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const T2 r = __hmax2(*reinterpret_cast<const T2 *>(&a), *reinterpret_cast<const T2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
  }
}
template <typename T>
__device__ __forceinline__ uint32_t word_min(uint32_t a, uint32_t b) {
  if constexpr (sizeof(T) == 4) {
    return __float_as_uint(fminf(__uint_as_float(a), __uint_as_float(b)));
  } else {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const T2 r = __hmin2(*reinterpret_cast<const T2 *>(&a), *reinterpret_cast<const T2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
  }
}
// -inf in every element of a word (its sign flipped: +inf)
template <typename T>
__device__ __forceinline__ uint32_t word_low() {
  return sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00fc00u : 0xff80ff80u;
}

}  // namespace

template <typename T, int D>
__global__ void __launch_bounds__(kAppendThreads, 6)
    pa_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int N = Chunk2<T>::N;             // elements of a 16-byte chunk
  constexpr int UNITS = D / (2 * N);          // units of a head
  constexpr int LANES = 32 / UNITS;           // tokens a warp takes at a time
  __shared__ int s_pos[kAppendMaxRows];       // -1: no work for the row
  __shared__ bool s_first[kAppendMaxRows];    // the row starts a page of its chunk
  __shared__ RowInfo s_row[kAppendMaxRows];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * p.tile_rows;
  const int rows = min(p.tile_rows, p.num_rows - row0);
  const bool il = p.interleaved != 0;
  const int rot = p.rotary_dim / (2 * N), half = p.rotary_dim / 2;

  // keys and values on their way to L2 while the rows are located
  {
    const int lines = p.num_kv_heads * D * (int)sizeof(T) / 128;  // of a row
    for (int i = threadIdx.x; i < 2 * rows * lines; i += kAppendThreads) {
      const int r = i / 2 / lines;
      const T *src = static_cast<const T *>(i & 1 ? p.value : p.key) +
                     (row0 + r) * (i & 1 ? p.value_stride : p.key_stride);
      prefetch_l2(reinterpret_cast<const char *>(src) + (i / 2 - r * lines) * 128);
    }
  }
  pdl_wait_primary();
  pdl_launch_dependents();

  // queries: a thread takes its unit of kAppendHeads heads of a row, whose
  // angles it loads once; the first ones are read while the rows are located
  const int u = threadIdx.x % UNITS;
  int ca, cb;
  unit_chunks(u, rot, il, ca, cb);
  const int groups = (p.num_heads + kAppendHeads - 1) / kAppendHeads;
  const int queries = p.query ? rows * groups : 0;
  Chunk2<T> q[kAppendHeads];  // query_out may be the query: no read-only path
  auto load_queries = [&](int j) {
    const int lr = j / groups, h0 = (j - lr * groups) * kAppendHeads;
    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.query) +
                                                       (row0 + lr) * p.query_stride + (size_t)h0 * D);
#pragma unroll
    for (int e = 0; e < kAppendHeads; ++e)
      if (h0 + e < p.num_heads) q[e] = {src[e * (D / N) + ca], src[e * (D / N) + cb]};
  };
  int j = threadIdx.x / UNITS;
  if (j < queries) load_queries(j);

  if (warp < rows) {
    RowInfo o;
    int pos = -1;
    bool first = false;
    if (locate_row(p, row0 + warp, o)) {
      pos = row_position(p, row0 + warp, o.tok);
      if ((unsigned)o.blk < (unsigned)p.num_blocks) {
        first = o.starts || o.tok % p.block_size == 0;  // the first token of its page here
        if (lane == 0) s_row[warp] = o;
      } else {  // nothing of the row is written, its queries neither
        pos = -1;
        if (lane == 0) report(p.status, kStatusBadInput);
      }
    }
    if (lane == 0) {
      s_pos[warp] = pos;
      s_first[warp] = first;
    }
  }
  __syncthreads();

  while (j < queries) {
    const int lr = j / groups, h0 = (j - lr * groups) * kAppendHeads;
    const int pos = s_pos[lr];
    if (pos >= 0) {
      if (u < rot) {
        Angles<N> r;
        r.load(p.cos_sin + (size_t)pos * p.rotary_dim, u, half);
#pragma unroll
        for (int e = 0; e < kAppendHeads; ++e) rotate_unit(q[e], r, il);
      }
      uint4 *dst = reinterpret_cast<uint4 *>(static_cast<T *>(p.query_out) +
                                             ((size_t)(row0 + lr) * p.num_heads + h0) * D);
#pragma unroll
      for (int e = 0; e < kAppendHeads; ++e)
        if (h0 + e < p.num_heads) {
          dst[e * (D / N) + ca] = q[e].a;
          dst[e * (D / N) + cb] = q[e].b;
        }
    }
    j += kAppendThreads / UNITS;
    if (j < queries) load_queries(j);
  }

  // keys and values: a warp takes one page of one KV head
  const int tl = lane / UNITS;
  for (int task = warp; task < rows * p.num_kv_heads; task += kAppendWarps) {
    const int lr = task / p.num_kv_heads, h = task - lr * p.num_kv_heads;
    if (!s_first[lr]) continue;
    const RowInfo o = s_row[lr];
    const int blk = o.blk;
    const int off0 = o.tok & (p.block_size - 1);
    const int n = min(o.tok_end - o.tok, p.block_size - off0);
    const size_t slot0 = ((size_t)blk * p.num_kv_heads + h) * p.block_size + off0;
    uint4 *kdst = reinterpret_cast<uint4 *>(static_cast<T *>(p.key_cache) + slot0 * D);
    uint4 *vdst = reinterpret_cast<uint4 *>(static_cast<T *>(p.value_cache) + slot0 * D);
    // the page's bounds so far, in words of the stored type
    uint32_t hi[8], lo[8];
    uint4 *bnd = nullptr;
    if (p.key_bounds) {
      bnd = reinterpret_cast<uint4 *>(static_cast<T *>(p.key_bounds) +
                                      ((size_t)blk * p.num_kv_heads + h) * 2 * D);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hi[e] = word_low<T>();
        lo[e] = word_low<T>() ^ (sizeof(T) == 4 ? 0x80000000u : 0x80008000u);
      }
    }
    auto join = [&](const uint4 &x, const uint4 &y, int e) {  // words e .. e + 3 of both
      hi[e] = word_max<T>(hi[e], x.x), lo[e] = word_min<T>(lo[e], y.x);
      hi[e + 1] = word_max<T>(hi[e + 1], x.y), lo[e + 1] = word_min<T>(lo[e + 1], y.y);
      hi[e + 2] = word_max<T>(hi[e + 2], x.z), lo[e + 2] = word_min<T>(lo[e + 2], y.z);
      hi[e + 3] = word_max<T>(hi[e + 3], x.w), lo[e + 3] = word_min<T>(lo[e + 3], y.w);
    };
    bool wrote = false;
#pragma unroll 1
    for (int i = tl; i < n; i += LANES) {
      const int row = row0 + lr + i;
      const int pos = row_position(p, row, o.tok + i);
      if (pos < 0) continue;
      wrote = true;
      const uint4 *ks = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.key) +
                                                        row * p.key_stride + (size_t)h * D);
      const uint4 *vs = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.value) +
                                                        row * p.value_stride + (size_t)h * D);
      Chunk2<T> k{__ldg(ks + ca), __ldg(ks + cb)};
      const Chunk2<T> v{__ldg(vs + 2 * u), __ldg(vs + 2 * u + 1)};
      if (u < rot) {
        Angles<N> r;
        r.load(p.cos_sin + (size_t)pos * p.rotary_dim, u, half);
        rotate_unit(k, r, il);
      }
      kdst[i * (D / N) + ca] = k.a;
      kdst[i * (D / N) + cb] = k.b;
      vdst[i * (D / N) + 2 * u] = v.a;
      vdst[i * (D / N) + 2 * u + 1] = v.b;
      if (bnd) {
        join(k.a, k.a, 0);
        join(k.b, k.b, 4);
      }
    }
    // (positions that are all bad leave the page as it was)
    if (!bnd || !__any_sync(0xffffffffu, wrote)) continue;
#pragma unroll
    for (int d = UNITS; d < 32; d <<= 1)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        hi[e] = word_max<T>(hi[e], __shfl_xor_sync(0xffffffffu, hi[e], d));
        lo[e] = word_min<T>(lo[e], __shfl_xor_sync(0xffffffffu, lo[e], d));
      }
    if (tl == 0) {
      if (off0 > 0) {  // the page held tokens before: their bounds join
        join(bnd[ca], bnd[D / N + ca], 0);
        join(bnd[cb], bnd[D / N + cb], 4);
      }
      bnd[ca] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      bnd[cb] = make_uint4(hi[4], hi[5], hi[6], hi[7]);
      bnd[D / N + ca] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      bnd[D / N + cb] = make_uint4(lo[4], lo[5], lo[6], lo[7]);
    }
  }
}

namespace {

template <typename T>
const void *pick_head(int head_size) {
  switch (head_size) {
    case 64: return reinterpret_cast<const void *>(&pa_append_kernel<T, 64>);
    case 128: return reinterpret_cast<const void *>(&pa_append_kernel<T, 128>);
    case 256: return reinterpret_cast<const void *>(&pa_append_kernel<T, 256>);
  }
  return nullptr;
}

}  // namespace

}  // namespace pa

extern "C" pa_status_t pa_append_kv(
    void *key_cache, void *value_cache, void *key_bounds, void *query_out, const void *query,
    const void *key, const void *value, long long query_stride, long long key_stride,
    long long value_stride, const float *cos_sin, const int32_t *positions,
    const int32_t *block_tables, const int32_t *seq_lens, const int32_t *q_start, int num_seqs,
    int num_rows, int num_heads, int num_kv_heads, int head_size, int num_blocks, int block_size,
    int max_blocks_per_seq, int max_seq_len, int rotary_dim, int interleaved, int max_position,
    int dtype, void *workspace, size_t workspace_bytes, void *stream) {
  using namespace pa;
  pa_status_t st = host_check_cache(dtype, num_heads, num_kv_heads, head_size, num_blocks,
                                    block_size, max_blocks_per_seq, max_seq_len);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || num_rows < 0 || (!q_start && num_rows != num_seqs)) return PA_ERR_INVALID_ARG;
  if (rotary_dim < 0 || rotary_dim > head_size || rotary_dim % 16) return PA_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return PA_ERR_INVALID_ARG;
  if (num_rows == 0 || num_seqs == 0) return PA_OK;  // (empty tensors have no address)
  if (rotary_dim > 0 && (!cos_sin || max_position < 1)) return PA_ERR_INVALID_ARG;
  if ((query == nullptr) != (query_out == nullptr)) return PA_ERR_INVALID_ARG;
  if (!key_cache || !value_cache || !key || !value || !block_tables || !seq_lens || !workspace)
    return PA_ERR_INVALID_ARG;
  const int chunk = dtype == PA_DTYPE_F32 ? 4 : 8;  // elements of 16 bytes
  const void *wide[] = {key_cache, value_cache, key_bounds, query_out, query, key, value, cos_sin};
  for (const void *q : wide)
    if (!host_aligned(q, 16)) return PA_ERR_INVALID_ARG;
  const void *ints[] = {positions, block_tables, seq_lens, q_start};
  for (const void *q : ints)
    if (!host_aligned(q, 4)) return PA_ERR_INVALID_ARG;
  if (!host_aligned(workspace, 256)) return PA_ERR_INVALID_ARG;
  const long long kv_row = (long long)num_kv_heads * head_size;
  if (key_stride < kv_row || value_stride < kv_row || key_stride % chunk || value_stride % chunk)
    return PA_ERR_INVALID_ARG;
  if (query && (query_stride < (long long)num_heads * head_size || query_stride % chunk))
    return PA_ERR_INVALID_ARG;
  // in place only row by row: another stride would write rows not yet read
  if (query && query == query_out && query_stride != (long long)num_heads * head_size)
    return PA_ERR_INVALID_ARG;
  if (workspace_bytes < (size_t)kStatusBytes) return PA_ERR_WORKSPACE_TOO_SMALL;

  AppendParams p{};
  p.key_cache = key_cache;
  p.value_cache = value_cache;
  p.key_bounds = key_bounds;
  p.query_out = query_out;
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
  // One row a CTA until every SM has four, then up to four, which share the
  // CTA's start-up (8193 rows: 48.7 us with one, 39.1 with two, 36.1 with
  // four, 36.6 with eight; 256 rows: 4.4 us with one, 6.2 with four).
  p.tile_rows = 1;
  while (p.tile_rows < kAppendMaxRows && num_rows > 4ll * sms * p.tile_rows) p.tile_rows *= 2;
  const void *fn = dtype == PA_DTYPE_F32    ? pick_head<float>(head_size)
                   : dtype == PA_DTYPE_BF16 ? pick_head<__nv_bfloat16>(head_size)
                                            : pick_head<__half>(head_size);
  void *args[1] = {&p};
  const unsigned grid = (unsigned)(((long long)num_rows + p.tile_rows - 1) / p.tile_rows);
  return host_launch(fn, grid, 1, kAppendThreads, 0, stream, args, "launch append kernel");
}
