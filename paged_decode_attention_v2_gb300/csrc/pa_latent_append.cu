// pa_latent_append: new rows of a paged cache of shared latents, the latent
// part normalised, the key part rotated by its position, and the queries'
// rotated parts beside their absorbed ones.
//
//   c = x (mean(x^2) + eps)^-1/2 w      y1 = x1 cos - x2 sin, y2 = x2 cos + x1 sin
// in fp32, rounded once.
//
// A warp takes a latent at a time, 8 or 16 elements a lane, and rotates eight
// heads at a time, four lanes each (16 elements of both halves of their pairs).
// A CTA takes up to four rows, whose latent, key part and query heads its warps
// take in turn.  Bound: a decode step's bytes are a few MB, so the launch and a
// chain of dependent loads (256 sequences, 32 heads, on GB300: 2.8 us); prompts
// are bytes (38 MB in 13 us, 5.8 at the copy rate: of 1707 CTAs of four rows 1216
// fit at once by their registers, so a second wave fills 40 % of the GPU; two rows
// a CTA took the same).
#include <math.h>

#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_ops.h"
#include "pa_rows.cuh"

namespace pa {
namespace {

constexpr int kLatentAppendThreads = 128;
constexpr int kLatentAppendWarps = kLatentAppendThreads / 32;
constexpr int kRope = 64;

struct LatentAppendParams {
  void *cache;  // [num_blocks][bs][latent_dim + 64]
  void *query;  // [rows][H][latent_dim + 64] or null
  const void *query_rope, *latent, *rope_key, *norm_weight;
  float eps;
  long long query_stride, query_head_stride, latent_stride, rope_key_stride;
  const float *cos_sin;
  const int32_t *positions, *block_tables, *seq_lens, *q_start;
  int *status;
  int num_seqs, num_rows, num_heads, num_blocks;
  int block_size, log2_block_size, max_blocks_per_seq, max_seq_len;
  int rotary_dim, interleaved, max_position;
  int tile_rows;
};

}  // namespace

template <typename T, int LAT>
__global__ void __launch_bounds__(kLatentAppendThreads, 6)
    pa_latent_append_kernel(const __grid_constant__ LatentAppendParams p) {
  constexpr int W = LAT + kRope, N = 8;  // elements of a row, of a 16-byte chunk
  constexpr int CH = LAT / 256;          // chunks of a latent, a lane
  constexpr int UNITS = kRope / (2 * N), HEADS = 32 / UNITS;
  __shared__ int s_pos[kAppendMaxRows];      // -1: no work for the row
  __shared__ size_t s_slot[kAppendMaxRows];  // the row's place in the cache

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = blockIdx.x * p.tile_rows;
  const int rows = min(p.tile_rows, p.num_rows - row0);
  const bool il = p.interleaved != 0;

  // the rows on their way to L2 while they are located
  {
    const int lines = W * (int)sizeof(T) / 128 + (p.query ? p.num_heads : 0);
    for (int i = threadIdx.x; i < rows * lines; i += kLatentAppendThreads) {
      const int r = row0 + i / lines, l = i % lines;
      const T *src = l < LAT / 64    ? static_cast<const T *>(p.latent) + r * p.latent_stride + l * 64
                     : l == LAT / 64 ? static_cast<const T *>(p.rope_key) + r * p.rope_key_stride
                                     : static_cast<const T *>(p.query_rope) + r * p.query_stride +
                                           (l - LAT / 64 - 1) * p.query_head_stride;
      prefetch_l2(src);
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
      s_slot[warp] = pos < 0 ? 0 : (size_t)o.blk * p.block_size + (o.tok & (p.block_size - 1));
    }
  }
  __syncthreads();

  // a row's tasks: its latent, then its key part and query heads, eight at a time
  const int heads = 1 + (p.query ? p.num_heads : 0), tasks = 1 + (heads + HEADS - 1) / HEADS;
  for (int v = warp; v < rows * tasks; v += kLatentAppendWarps) {
    const int lr = v / tasks, k = v - lr * tasks, row = row0 + lr;
    const int pos = s_pos[lr];
    if (pos < 0) continue;
    T *to = static_cast<T *>(p.cache) + s_slot[lr] * W;
    if (k == 0) {
      const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.latent) + row * p.latent_stride);
      uint4 x[CH];
#pragma unroll
      for (int c = 0; c < CH; ++c) x[c] = __ldg(src + lane + 32 * c);
      if (p.norm_weight) {
        const uint4 *wsrc = static_cast<const uint4 *>(p.norm_weight);
        float f[CH][N], w[N], sum = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          widen<T>(x[c], f[c]);
#pragma unroll
          for (int i = 0; i < N; ++i) sum = fmaf(f[c][i], f[c][i], sum);
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        const float r = 1.f / sqrtf(sum * (1.f / LAT) + p.eps);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          widen<T>(__ldg(wsrc + lane + 32 * c), w);
#pragma unroll
          for (int i = 0; i < N; ++i) f[c][i] = f[c][i] * r * w[i];
          x[c] = narrow<T>(f[c]);
        }
      }
#pragma unroll
      for (int c = 0; c < CH; ++c) reinterpret_cast<uint4 *>(to)[lane + 32 * c] = x[c];
    } else {
      const int h = (k - 1) * HEADS + lane / UNITS - 1, u = lane % UNITS;  // -1: the key part
      if (h + 1 >= heads) continue;
      int ca, cb;
      unit_chunks(u, UNITS, il, ca, cb);
      const T *from = h < 0 ? static_cast<const T *>(p.rope_key) + row * p.rope_key_stride
                            : static_cast<const T *>(p.query_rope) + row * p.query_stride + h * p.query_head_stride;
      const uint4 *src = reinterpret_cast<const uint4 *>(from);
      Chunk2<T> x{src[ca], src[cb]};  // (which may be the query itself: no read-only path)
      Angles<N> r;
      r.load(p.cos_sin + (size_t)pos * kRope, u, kRope / 2);
      rotate_unit(x, r, il);
      uint4 *dst = reinterpret_cast<uint4 *>(
          (h < 0 ? to : static_cast<T *>(p.query) + ((size_t)row * p.num_heads + h) * W) + LAT);
      dst[ca] = x.a;
      dst[cb] = x.b;
    }
  }
}

namespace {

template <typename T>
const void *latent_append_pick(int latent_dim) {
  return latent_dim == 512 ? reinterpret_cast<const void *>(&pa_latent_append_kernel<T, 512>)
                           : reinterpret_cast<const void *>(&pa_latent_append_kernel<T, 256>);
}

// Whether no thread reads of query_rope what another writes of query: they do not
// meet, or heads are as far apart in both and a head's words are those that they
// are rotated into, or none that are written.
bool rope_apart(const void *query, const void *query_rope, long long stride, long long head_stride,
                int num_rows, int num_heads, int latent_dim) {
  const __int128 width = latent_dim + kRope;
  const __int128 from =
      (reinterpret_cast<intptr_t>(query_rope) - reinterpret_cast<intptr_t>(query)) / 2;  // elements
  const __int128 span = (__int128)(num_rows - 1) * stride + (__int128)(num_heads - 1) * head_stride + kRope;
  if (from >= num_rows * (num_heads * width) || from + span <= latent_dim) return true;
  if (num_heads > 1 && head_stride != width) return false;
  if (num_rows > 1 && stride != num_heads * width) return false;
  if (from == latent_dim) return true;
  const __int128 at = ((from - latent_dim) % width + width) % width;  // in a head, from its written words on
  return at >= kRope && at <= width - kRope;
}

}  // namespace
}  // namespace pa

extern "C" pa_status_t pa_latent_append(
    void *cache, void *query, const void *query_rope, const void *latent, const void *rope_key,
    const void *norm_weight, float eps, long long query_stride, long long query_head_stride,
    long long latent_stride, long long rope_key_stride, const float *cos_sin,
    const int32_t *positions, const int32_t *block_tables, const int32_t *seq_lens,
    const int32_t *q_start, int num_seqs, int num_rows, int num_heads, int latent_dim, int rope_dim,
    int num_blocks, int block_size, int max_blocks_per_seq, int max_seq_len, int interleaved,
    int max_position, int dtype, void *workspace, size_t workspace_bytes, void *stream) {
  using namespace pa;
  pa_status_t st = latent_check_cache(dtype, num_heads, latent_dim, rope_dim, num_blocks, block_size,
                                      max_blocks_per_seq, max_seq_len);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || num_rows < 0 || (!q_start && num_rows != num_seqs)) return PA_ERR_INVALID_ARG;
  if (interleaved != 0 && interleaved != 1) return PA_ERR_INVALID_ARG;
  if (!(eps >= 0.f) || !isfinite(eps)) return PA_ERR_INVALID_ARG;
  if (num_rows == 0 || num_seqs == 0) return PA_OK;  // (empty tensors have no address)
  if ((query == nullptr) != (query_rope == nullptr)) return PA_ERR_INVALID_ARG;
  if (!cache || !latent || !rope_key || !cos_sin || max_position < 1 || !block_tables || !seq_lens || !workspace)
    return PA_ERR_INVALID_ARG;
  const void *wide[] = {cache, query, query_rope, latent, rope_key, norm_weight, cos_sin};
  for (const void *q : wide)
    if (!host_aligned(q, 16)) return PA_ERR_INVALID_ARG;
  const void *ints[] = {positions, block_tables, seq_lens, q_start};
  for (const void *q : ints)
    if (!host_aligned(q, 4)) return PA_ERR_INVALID_ARG;
  if (!host_aligned(workspace, 256)) return PA_ERR_INVALID_ARG;
  if (latent_stride < latent_dim || latent_stride % 8 || rope_key_stride < rope_dim || rope_key_stride % 8)
    return PA_ERR_INVALID_ARG;
  if (query) {  // a row's heads do not reach into the next row's, or a head's rows into the next head's
    if (query_head_stride < rope_dim || query_stride < rope_dim || query_head_stride % 8 || query_stride % 8)
      return PA_ERR_INVALID_ARG;
    const __int128 row = query_stride, head = query_head_stride;
    if (row < (num_heads - 1) * head + rope_dim && head < (num_rows - 1) * row + rope_dim) return PA_ERR_INVALID_ARG;
  }
  if (workspace_bytes < (size_t)kStatusBytes) return PA_ERR_WORKSPACE_TOO_SMALL;
  if (query && !rope_apart(query, query_rope, query_stride, query_head_stride, num_rows, num_heads, latent_dim))
    return PA_ERR_INVALID_ARG;

  LatentAppendParams p{};
  p.cache = cache;
  p.query = query;
  p.query_rope = query_rope;
  p.latent = latent;
  p.rope_key = rope_key;
  p.norm_weight = norm_weight;
  p.eps = eps;
  p.query_stride = query_stride;
  p.query_head_stride = query_head_stride;
  p.latent_stride = latent_stride;
  p.rope_key_stride = rope_key_stride;
  p.cos_sin = cos_sin;
  p.positions = positions;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.q_start = q_start;
  p.status = static_cast<int *>(workspace);
  p.num_seqs = num_seqs;
  p.num_rows = num_rows;
  p.num_heads = num_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  while ((1 << p.log2_block_size) < block_size) ++p.log2_block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_seq_len = max_seq_len;
  p.rotary_dim = rope_dim;
  p.interleaved = interleaved;
  p.max_position = max_position;
  int sms = 0;
  st = host_sm_count(&sms);
  if (st != PA_OK) return st;
  p.tile_rows = 1;
  while (p.tile_rows < kAppendMaxRows && num_rows > 4ll * sms * p.tile_rows) p.tile_rows *= 2;
  const void *fn = dtype == PA_DTYPE_BF16 ? latent_append_pick<__nv_bfloat16>(latent_dim)
                                          : latent_append_pick<__half>(latent_dim);
  void *args[1] = {&p};
  const unsigned grid = (unsigned)(((long long)num_rows + p.tile_rows - 1) / p.tile_rows);
  return host_launch(fn, grid, 1, kLatentAppendThreads, 0, stream, args, "launch latent append kernel");
}
