// pa_select_blocks and pa_sparse_forward: decode attention over the blocks
// that a cheap score selects.
//
// The score of page j for a query row and a KV head is the sum, over the
// heads of its group, of the upper bound that the page's key bounds put on
// q . k:  sum_h sum_d max(q_hd max_jd, q_hd min_jd).  Its terms split by the
// sign of q_hd, so it is one product of 2 D numbers,
//   score_j = sum_d Q+_d max_jd + Q-_d min_jd,
//   Q+_d = sum_h max(q_hd, 0),  Q-_d = sum_h min(q_hd, 0),
// whatever the group's size: the bounds are read once a row.
//
// Which block is read must not hang on a rounding, so the selection is the
// one that exact scores give (ties to the lower page).  Scores in fp32 are
// within eps of the exact ones, eps = 48 2^-24 W A, with W = sum |Q| and A the
// largest bound: Q has up to 15 additions of one sign (relative error 15
// 2^-24), a lane's chain up to 16 products, the warp's sum 5 more, and 48 >
// 15 + 16 + 5 + 1 leaves room for W and A themselves.  A page more than 2 eps
// above the k-th largest fp32 score is in, one more than 2 eps below is out;
// the few between are scored again in fp64, where products of 16-bit numbers
// are exact.
//
// Layout of the work: an item is one (row, KV head); its pages are cut into
// chunks, one CTA each, so that a single long sequence fills the GPU; the CTA
// that finishes an item's last chunk selects.  The selected pages come out in
// page order with the last page last, as a block table of the view in which
// every (row, KV head) is a sequence of one KV head: the attention kernels
// then need nothing new.
//
// Bound: the bytes of the key bounds (2 D numbers a page and KV head).
#include <math_constants.h>

#include <type_traits>

#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_ops.h"

namespace pa {
namespace {

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 512;       // of the score histogram, two a thread
constexpr int kSelList = 256;       // pages scored again in shared memory
constexpr int kSelSegment = 8;      // pages of a warp at a time
constexpr int kSelSmemPages = 8192; // scores kept in shared memory

template <typename T>
__device__ __forceinline__ void widen(const uint4 &c, float (&f)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4) {
    chunk_to_float(c, f);
  } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
    chunk_to_float_bf16(c, f);
  } else {
    chunk_to_float_f16(c, f);
  }
}

// An order-preserving map of doubles (no NaN) to unsigned integers; -0 is 0.
__device__ __forceinline__ unsigned long long order64(double x) {
  const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
  return (u >> 63) ? ~u : u | (1ull << 63);
}

// The item's row: its sequence and the keys it sees (0: none, or bad input).
__device__ __forceinline__ void locate(const SelectParams &p, int row, int &seq, int &vis) {
  seq = row;
  vis = 0;
  int before = 0, n = 1;  // the row's index in its chunk, the chunk's rows
  if (p.q_start) {
    int lo = 0, hi = p.num_seqs + 1;  // the first entry above row
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(p.q_start + mid) > row)
        hi = mid;
      else
        lo = mid + 1;
    }
    if (lo > p.num_seqs) {  // behind the last sequence: nothing to see
      seq = 0;
      return;
    }
    if (lo == 0) {
      seq = 0;
      report(p.status, kStatusBadInput);
      return;
    }
    seq = lo - 1;
    const int q0 = __ldg(p.q_start + seq);
    before = row - q0;
    n = __ldg(p.q_start + lo) - q0;
    if (q0 < 0 || before < 0 || before >= n) {
      report(p.status, kStatusBadInput);
      return;
    }
  }
  const int L = __ldg(p.seq_lens + seq);
  if (L < 0 || L > p.max_seq_len || (p.q_start && L < n)) {
    report(p.status, kStatusBadInput);
    return;
  }
  vis = L - n + before + 1;
  if (!p.q_start) vis = L;
}

struct SelShared {
  double w[512];  // Q+ then Q-, 2 D numbers
  double fine[kSelList];
  int list[kSelList];
  int hist[kSelBins];
  float red_f[2 * kSelWarps];
  int red_i[kSelWarps];
  int bin, above, flag, count;
};

// Sum (or maximum) over the CTA; every thread gets it.
__device__ __forceinline__ int block_sum(int v, int *red) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int i = 0; i < kSelWarps; ++i) t += red[i];
  return t;
}
__device__ __forceinline__ void block_min_max(float &lo, float &hi, float *red) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, d));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, d));
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    red[threadIdx.x >> 5] = lo;
    red[kSelWarps + (threadIdx.x >> 5)] = hi;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSelWarps; ++i) {
    lo = fminf(lo, red[i]);
    hi = fmaxf(hi, red[kSelWarps + i]);
  }
}

__device__ __forceinline__ int bin_of(float s, float lo, float inv) {
  const float x = (s - lo) * inv;  // non-decreasing in s
  return !(x >= 0.f) ? 0 : x >= (float)kSelBins ? kSelBins - 1 : min((int)x, kSelBins - 1);
}

}  // namespace

// Dynamic shared memory: the scores of min(max_pages, kSelSmemPages) pages.
template <typename T, int D>
__global__ void __launch_bounds__(kSelThreads) pa_select_kernel(const __grid_constant__ SelectParams p) {
  constexpr int N = 16 / (int)sizeof(T);       // elements of a 16-byte piece
  constexpr int PIECES = 2 * D / N;            // of a page's bounds
  constexpr int LPP = PIECES < 32 ? PIECES : 32;  // lanes of a page
  constexpr int VPL = PIECES / LPP;            // pieces a lane
  constexpr int PPW = 32 / LPP;                // pages of a warp side by side
  __shared__ SelShared sh;
  extern __shared__ __align__(16) float s_scores[];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int item = blockIdx.x / p.chunks, chunk = blockIdx.x % p.chunks;
  const int row = item / p.num_kv_heads, h = item % p.num_kv_heads;
  const int G = p.num_heads / p.num_kv_heads;

  pdl_wait_primary();
  pdl_launch_dependents();
  int seq, vis;
  locate(p, row, seq, vis);
  const int n = (vis + p.block_size - 1) >> p.log2_block_size;  // pages the row sees
  const int32_t *bt = p.block_tables + (size_t)seq * p.max_blocks_per_seq;
  const int k = p.num_selected;
  const bool all = n <= k;
  const int nch = all ? 1 : (n + p.chunk_pages - 1) / p.chunk_pages;
  if (chunk >= nch) return;
  const int first = p.sinks, last = n - p.recent;  // pages [first, last) go by their score
  const bool local = n <= kSelSmemPages && n <= p.smem_pages;  // the selecting CTA's scores: in smem
  float *gscores = p.scores + (size_t)item * p.max_pages;
  const T *q = static_cast<const T *>(p.query) + ((size_t)row * p.num_heads + h * G) * D;

  float *sc = s_scores;
  if (!all) {
    // ---- scores of the chunk's pages ----
    float w[VPL][N];
    float wsum = 0.f;
    const int lp = lane % LPP;
#pragma unroll
    for (int v = 0; v < VPL; ++v) {
      const int piece = v * LPP + lp;
      const bool pos = piece < PIECES / 2;
      const int d0 = (pos ? piece : piece - PIECES / 2) * N;
#pragma unroll
      for (int e = 0; e < N; ++e) w[v][e] = 0.f;
      for (int g = 0; g < G; ++g) {
        float f[N];
        widen<T>(__ldg(reinterpret_cast<const uint4 *>(q + (size_t)g * D + d0)), f);
#pragma unroll
        for (int e = 0; e < N; ++e) w[v][e] += pos ? fmaxf(f[e], 0.f) : fminf(f[e], 0.f);
      }
#pragma unroll
      for (int e = 0; e < N; ++e) wsum += fabsf(w[v][e]);
    }
#pragma unroll
    for (int d = LPP / 2; d > 0; d >>= 1) wsum += __shfl_xor_sync(0xffffffffu, wsum, d);
    float amax = 0.f;
    const int c_end = min(n, (chunk + 1) * p.chunk_pages);
    float *out = p.chunks == 1 && local ? s_scores : gscores;
    for (int p0 = chunk * p.chunk_pages + warp * kSelSegment; p0 < c_end;
         p0 += kSelWarps * kSelSegment) {
      int blk = -1;  // also past the chunk: those lanes load nothing
      if (lane < kSelSegment && p0 + lane < c_end) {
        blk = __ldg(bt + p0 + lane);
        if ((unsigned)blk >= (unsigned)p.num_blocks) {
          report(p.status, kStatusBadInput);
          blk = -1;
        }
      }
      constexpr int STEPS = kSelSegment / PPW;
      float acc[STEPS];
      uint4 x[STEPS][VPL];
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        const int b = __shfl_sync(0xffffffffu, blk, j * PPW + lane / LPP);
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.key_bounds) +
                                                           ((size_t)max(b, 0) * p.num_kv_heads + h) * 2 * D);
#pragma unroll
        for (int v = 0; v < VPL; ++v)
          x[j][v] = b >= 0 ? __ldg(src + v * LPP + lp) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        acc[j] = 0.f;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          float f[N];
          widen<T>(x[j][v], f);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            acc[j] = fmaf(w[v][e], f[e], acc[j]);
            amax = fmaxf(amax, fabsf(f[e]));
          }
        }
      }
#pragma unroll
      for (int d = LPP / 2; d > 0; d >>= 1)
#pragma unroll
        for (int j = 0; j < STEPS; ++j) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], d);
      // lane j PPW + i takes the score of that page
      float mine = 0.f;
#pragma unroll
      for (int j = 0; j < STEPS; ++j) {
        const float t = __shfl_sync(0xffffffffu, acc[j], (lane % PPW) * LPP);
        if (lane / PPW == j) mine = t;
      }
      if (lane < kSelSegment && p0 + lane < c_end)
        out[p0 + lane] = blk < 0 || mine != mine ? -CUDART_INF_F : mine;
    }
    float lo = 0.f;
    block_min_max(lo, amax, sh.red_f);
    if (p.chunks > 1) {
      if (tid == 0) p.amax[(size_t)item * p.chunks + chunk] = amax;
      __syncthreads();
      if (tid == 0) sh.flag = atomic_add_acq_rel_gpu(p.counters + item, 1) == nch - 1;
      __syncthreads();
      if (!sh.flag) return;
      if (tid == 0) p.counters[item] = 0;  // every chunk is in: ready for the next call
      amax = 0.f;
      for (int c = tid; c < nch; c += kSelThreads)
        amax = fmaxf(amax, __ldcg(p.amax + (size_t)item * p.chunks + c));
      block_min_max(lo, amax, sh.red_f);
    }
    if (!local) {
      sc = gscores;
    } else if (p.chunks > 1) {
      for (int i = tid; i < n; i += kSelThreads) s_scores[i] = __ldcg(gscores + i);
    }
    __syncthreads();

    // ---- the need best of pages [first, last) ----
    const int need = k - p.sinks - p.recent;
    float hi_in = CUDART_INF_F, lo_in = CUDART_INF_F;  // in above hi_in, out below lo_in
    bool marked = false;  // those in between carry +inf (in) or -inf (out)
    if (need > 0) {
      const float eps = 48.f * 5.9604644775390625e-8f * wsum * amax + 1e-36f;
      float lo = CUDART_INF_F, hi = -CUDART_INF_F;  // finite scores' range
      for (int i = first + tid; i < last; i += kSelThreads) {
        const float s = sc[i];
        if (fabsf(s) <= 3.402823466e38f) {
          lo = fminf(lo, s);
          hi = fmaxf(hi, s);
        }
      }
      block_min_max(lo, hi, sh.red_f);
      // The bin of a histogram over [lo, hi] that holds the need-th score;
      // then, if too many scores are that close, over that bin's own range.
      int m = 0;
      float t_lo = -CUDART_INF_F, t_hi = CUDART_INF_F;
      int above0 = 0;  // scores above the histogram's range
      for (int pass = 0; pass < 4; ++pass) {
        const float inv = hi > lo ? (float)kSelBins / (hi - lo) : 0.f;
        const bool ranged = pass > 0;
        for (int b = tid; b < kSelBins; b += kSelThreads) sh.hist[b] = 0;
        __syncthreads();
        for (int i = first + tid; i < last; i += kSelThreads) {
          const float s = sc[i];
          if (!ranged || (s >= t_lo && s <= t_hi)) atomicAdd(&sh.hist[bin_of(s, lo, inv)], 1);
        }
        __syncthreads();
        // bins from the top: thread t holds bins (511 - 2t, 510 - 2t)
        const int b1 = sh.hist[kSelBins - 1 - 2 * tid], b0 = sh.hist[kSelBins - 2 - 2 * tid];
        int run = b0 + b1;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, run, d);
          if (lane >= d) run += t;
        }
        if (lane == 31) sh.red_i[warp] = run;
        __syncthreads();
        int base = above0;
        for (int i = 0; i < warp; ++i) base += sh.red_i[i];
        const int before = base + run - b0 - b1;  // scores above this thread's bins
        if (before < need && before + b1 >= need) {
          sh.bin = kSelBins - 1 - 2 * tid;
          sh.above = before;
        } else if (before + b1 < need && before + b1 + b0 >= need) {
          sh.bin = kSelBins - 2 - 2 * tid;
          sh.above = before + b1;
        }
        __syncthreads();
        const int bin = sh.bin, above = sh.above;
        float blo = CUDART_INF_F, bhi = -CUDART_INF_F;  // the bin's own range
        for (int i = first + tid; i < last; i += kSelThreads) {
          const float s = sc[i];
          if ((!ranged || (s >= t_lo && s <= t_hi)) && bin_of(s, lo, inv) == bin) {
            blo = fminf(blo, s);
            bhi = fmaxf(bhi, s);
          }
        }
        block_min_max(blo, bhi, sh.red_f);
        t_lo = blo;
        t_hi = bhi;
        above0 = above;
        hi_in = t_hi + 2.f * eps;
        lo_in = t_lo - 2.f * eps;
        int c = 0;
        for (int i = first + tid; i < last; i += kSelThreads) c += !(sc[i] > hi_in) && !(sc[i] < lo_in);
        m = block_sum(c, sh.red_i);
        if (m <= kSelList || !(t_hi > t_lo) || !(t_hi - t_lo > 4.f * eps)) break;
        lo = t_lo;
        hi = t_hi;
      }
      int c = 0;
      for (int i = first + tid; i < last; i += kSelThreads) c += sc[i] > hi_in;
      const int more = need - block_sum(c, sh.red_i);  // of the m in between
      if (more < m) {
        // ---- score those m again in fp64 ----
        for (int d = tid; d < 2 * D; d += kSelThreads) {
          double a = 0.0;
          for (int g = 0; g < G; ++g) {
            const double f = (double)to_float(q[(size_t)g * D + d % D]);
            a += d < D ? fmax(f, 0.0) : fmin(f, 0.0);
          }
          sh.w[d] = a;
        }
        if (tid == 0) sh.count = 0;
        __syncthreads();
        const bool small = m <= kSelList;
        if (small) {
          for (int i = first + tid; i < last; i += kSelThreads)
            if (!(sc[i] > hi_in) && !(sc[i] < lo_in)) sh.list[atomicAdd(&sh.count, 1)] = i;
          __syncthreads();
        }
        double *gfine = p.fine + (size_t)item * p.max_pages;
        const int jobs = small ? m : last - first;
        for (int j = warp; j < jobs; j += kSelWarps) {
          const int i = small ? sh.list[j] : first + j;
          if (!small && (sc[i] > hi_in || sc[i] < lo_in)) continue;
          const int blk = __ldg(bt + i);
          double s = -CUDART_INF;
          if ((unsigned)blk < (unsigned)p.num_blocks) {
            s = 0.0;
            const T *b = static_cast<const T *>(p.key_bounds) + ((size_t)blk * p.num_kv_heads + h) * 2 * D;
#pragma unroll 4
            for (int d = lane; d < 2 * D; d += 32) s += sh.w[d] * (double)to_float(b[d]);
#pragma unroll
            for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            if (s != s) s = -CUDART_INF;
          }
          if (lane == 0) {
            if (small)
              sh.fine[j] = s;
            else
              gfine[i] = s;
          }
        }
        __syncthreads();
        // mark: +inf for the `more` best (ties to the lower page), -inf for
        // the others
        if (small) {
          if (tid < m) {
            const double s = sh.fine[tid];
            const int i = sh.list[tid];
            int rank = 0;
            for (int j = 0; j < m; ++j) {
              const double t = sh.fine[j];
              rank += t > s || (t == s && sh.list[j] < i);
            }
            sc[i] = rank < more ? CUDART_INF_F : -CUDART_INF_F;
          }
        } else {
          // the more-th largest by bisection, then its ties in page order
          unsigned long long t = 0;
          for (int bit = 63; bit >= 0; --bit) {
            const unsigned long long cand = t | (1ull << bit);
            int cnt = 0;
            for (int i = first + tid; i < last; i += kSelThreads)
              if (!(sc[i] > hi_in) && !(sc[i] < lo_in)) cnt += order64(gfine[i]) >= cand;
            if (block_sum(cnt, sh.red_i) >= more) t = cand;
          }
          int cnt = 0;
          for (int i = first + tid; i < last; i += kSelThreads)
            if (!(sc[i] > hi_in) && !(sc[i] < lo_in)) cnt += order64(gfine[i]) > t;
          int ties = more - block_sum(cnt, sh.red_i);
          if (warp == 0) {
            for (int i0 = first; i0 < last; i0 += 32) {
              const int i = i0 + lane;
              const bool in = i < last && !(sc[i] > hi_in) && !(sc[i] < lo_in);
              const unsigned long long u = in ? order64(gfine[i]) : 0;
              const unsigned eq = __ballot_sync(0xffffffffu, in && u == t);
              const bool keep = in && (u > t || (u == t && __popc(eq & ((1u << lane) - 1u)) < ties));
              ties = max(0, ties - __popc(eq));
              if (in) sc[i] = keep ? CUDART_INF_F : -CUDART_INF_F;
            }
          }
        }
        __syncthreads();
        marked = true;
      }  // else all of them are in
    }
    // ---- the selected pages in page order ----
    auto selected = [&](int i) -> bool {
      if (i < first || i >= last) return true;
      if (need <= 0) return false;
      const float s = sc[i];
      return marked ? s > hi_in || s == CUDART_INF_F : !(s < lo_in);
    };
    const int seg = ((n + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
    const int s0 = min(n, warp * seg), s1 = min(n, s0 + seg);
    int cnt = 0;
    for (int i0 = s0; i0 < s1; i0 += 32) {
      const int i = i0 + lane;
      cnt += __popc(__ballot_sync(0xffffffffu, i < s1 && selected(i)));
    }
    __syncthreads();
    if (lane == 0) sh.red_i[warp] = cnt;
    __syncthreads();
    int at = 0;
    for (int i = 0; i < warp; ++i) at += sh.red_i[i];
    for (int i0 = s0; i0 < s1; i0 += 32) {
      const int i = i0 + lane;
      const bool in = i < s1 && selected(i);
      const unsigned m = __ballot_sync(0xffffffffu, in);
      const int o = at + __popc(m & ((1u << lane) - 1u));
      if (in && o < k) {
        if (p.selected) p.selected[(size_t)item * k + o] = i;
        if (p.table) p.table[(size_t)item * k + o] = view_block(__ldg(bt + i), h, p.num_kv_heads, p.num_blocks);
      }
      at += __popc(m);
    }
    if (tid == 0 && p.lens) p.lens[item] = (k - 1) * p.block_size + vis - (n - 1) * p.block_size;
  } else {
    for (int o = tid; o < k; o += kSelThreads) {
      if (p.selected) p.selected[(size_t)item * k + o] = o < n ? o : -1;
      if (p.table)
        p.table[(size_t)item * k + o] =
            o < n ? view_block(__ldg(bt + o), h, p.num_kv_heads, p.num_blocks) : -1;
    }
    if (tid == 0 && p.lens) p.lens[item] = vis;
  }
}

// A given selection (pages in ascending order, -1 behind the last) as the
// view's block table: one warp an item.
__global__ void __launch_bounds__(128) pa_given_blocks_kernel(const __grid_constant__ SelectParams p) {
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.x * 4 + (threadIdx.x >> 5);
  pdl_wait_primary();
  pdl_launch_dependents();
  if (item >= p.num_rows * p.num_kv_heads) return;
  const int row = item / p.num_kv_heads, h = item % p.num_kv_heads;
  int seq, vis;
  locate(p, row, seq, vis);
  const int n = (vis + p.block_size - 1) >> p.log2_block_size;
  const int32_t *bt = p.block_tables + (size_t)seq * p.max_blocks_per_seq;
  const int32_t *given = p.given + (size_t)item * p.num_selected;
  int count = 0, prev = -1;  // blocks so far, the last of them
  bool ok = true, open = true;
  for (int o0 = 0; o0 < p.num_selected; o0 += 32) {
    const int o = o0 + lane;
    const int j = o < p.num_selected ? __ldg(given + o) : -1;
    const int left = __shfl_up_sync(0xffffffffu, j, 1);
    const int before = lane == 0 ? prev : left;
    // ascending pages that the row sees, then only -1
    const bool good = j == -1 || (j >= 0 && j < n && (lane == 0 && o0 == 0 ? true : j > before) &&
                                  (lane == 0 ? open : left >= 0));
    ok = ok && __all_sync(0xffffffffu, good);
    const unsigned live = __ballot_sync(0xffffffffu, j >= 0);
    count += __popc(live);
    prev = __shfl_sync(0xffffffffu, j, 31);
    open = prev >= 0;
    if (o < p.num_selected)
      p.table[(size_t)item * p.num_selected + o] =
          good && j >= 0 ? view_block(__ldg(bt + j), h, p.num_kv_heads, p.num_blocks) : -1;
  }
  // the length: whole pages, but for the row's last one if it is among them
  int top = -1;
  if (ok && count > 0) top = __ldg(given + count - 1);
  if (lane == 0) {
    if (!ok) report(p.status, kStatusBadInput);
    const int len = !ok || count == 0 ? 0
                    : top == n - 1    ? (count - 1) * p.block_size + vis - (n - 1) * p.block_size
                                      : count * p.block_size;
    p.lens[item] = len;
  }
}

namespace {

template <typename T>
const void *pick_select(int head_size) {
  switch (head_size) {
    case 64: return reinterpret_cast<const void *>(&pa_select_kernel<T, 64>);
    case 128: return reinterpret_cast<const void *>(&pa_select_kernel<T, 128>);
    case 256: return reinterpret_cast<const void *>(&pa_select_kernel<T, 256>);
  }
  return nullptr;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// The workspace: the attention's over the view, then table, lengths, counters
// and what the selection keeps a page.
struct SparseLayout {
  size_t table, lens, counters, amax, scores, fine, total;
  int max_pages, view_len;
};
constexpr int kSelMaxChunks = 1024;  // of an item

bool sparse_layout(int num_rows, int num_heads, int num_kv_heads, int head_size, int block_size,
                   int max_seq_len, int num_selected, int partition_size, SparseLayout *o) {
  if (num_rows < 0 || num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads ||
      head_size < 1 || block_size < 1 || max_seq_len < 0 || num_selected < 1 || partition_size < 1)
    return false;
  const long long items = (long long)num_rows * num_kv_heads;
  const long long cap = (long long)num_selected * block_size;
  if (items > 0x7fffffffll || cap > 0x7fffffffll) return false;
  o->max_pages = (int)(((long long)max_seq_len + block_size - 1) / block_size);
  o->view_len = (int)(cap < max_seq_len ? cap : max_seq_len);
  const size_t attn = pa_workspace_bytes((int)items, num_heads / num_kv_heads, head_size,
                                         o->view_len, partition_size);
  if (attn == 0) return false;
  o->table = align256(attn);
  o->lens = o->table + align256((size_t)items * num_selected * 4);
  o->counters = o->lens + align256((size_t)items * 4);
  o->amax = o->counters + align256((size_t)items * 4);
  const int chunks = (o->max_pages + 63) / 64;
  o->scores = o->amax + align256((size_t)items * (chunks < kSelMaxChunks ? chunks : kSelMaxChunks) * 4);
  o->fine = o->scores + align256((size_t)items * o->max_pages * 4);
  o->total = o->fine + align256((size_t)items * o->max_pages * 8);
  return true;
}

struct SparseCall {
  int32_t *selected;  // written
  const int32_t *given;
  const void *query, *key_bounds;
  const int32_t *block_tables, *seq_lens, *q_start;
  int num_seqs, num_rows, num_heads, num_kv_heads, head_size, num_blocks, block_size;
  int max_blocks_per_seq, max_seq_len, num_selected, sinks, recent, partition_size, dtype;
  void *workspace;
  size_t workspace_bytes;
  void *stream;
};

pa_status_t check_sparse(const SparseCall &c, SparseLayout *lay) {
  pa_status_t st = host_check_cache(c.dtype, c.num_heads, c.num_kv_heads, c.head_size,
                                    c.num_blocks, c.block_size, c.max_blocks_per_seq, c.max_seq_len);
  if (st != PA_OK) return st;
  if (c.num_seqs < 0 || c.num_rows < 0 || (!c.q_start && c.num_rows != c.num_seqs) ||
      (c.num_rows > 0 && c.num_seqs == 0))
    return PA_ERR_INVALID_ARG;
  if (c.num_selected < 1 || c.sinks < 0 || c.recent < 1 || c.sinks > c.num_selected ||
      c.recent > c.num_selected - c.sinks)
    return PA_ERR_INVALID_ARG;
  if (c.partition_size < 1) return PA_ERR_INVALID_ARG;
  if (c.partition_size % 64 || c.partition_size % c.block_size || c.partition_size > 8192)
    return PA_ERR_UNSUPPORTED;
  if (!c.block_tables || !c.seq_lens || !c.workspace) return PA_ERR_INVALID_ARG;
  if (!host_aligned(c.query, 16) || !host_aligned(c.key_bounds, 16) ||
      !host_aligned(c.block_tables, 4) || !host_aligned(c.seq_lens, 4) ||
      !host_aligned(c.q_start, 4) || !host_aligned(c.selected, 4) || !host_aligned(c.given, 4) ||
      !host_aligned(c.workspace, 256))
    return PA_ERR_INVALID_ARG;
  if (!sparse_layout(c.num_rows, c.num_heads, c.num_kv_heads, c.head_size, c.block_size,
                     c.max_seq_len, c.num_selected, c.partition_size, lay))
    return PA_ERR_UNSUPPORTED;
  if (c.workspace_bytes < lay->total) return PA_ERR_WORKSPACE_TOO_SMALL;
  return PA_OK;
}

// Enqueue the selection (or the translation of a given one); with `table`,
// the view's block table and lengths too.
pa_status_t run_select(const SparseCall &c, const SparseLayout &lay, bool table) {
  int sms = 0;
  pa_status_t st = host_sm_count(&sms);
  if (st != PA_OK) return st;
  uint8_t *ws = static_cast<uint8_t *>(c.workspace);
  SelectParams p{};
  p.query = c.query;
  p.key_bounds = c.key_bounds;
  p.block_tables = c.block_tables;
  p.seq_lens = c.seq_lens;
  p.q_start = c.q_start;
  p.selected = c.selected;
  p.given = c.given;
  p.table = table ? reinterpret_cast<int32_t *>(ws + lay.table) : nullptr;
  p.lens = table ? reinterpret_cast<int32_t *>(ws + lay.lens) : nullptr;
  p.counters = reinterpret_cast<int *>(ws + lay.counters);
  p.amax = reinterpret_cast<float *>(ws + lay.amax);
  p.scores = reinterpret_cast<float *>(ws + lay.scores);
  p.fine = reinterpret_cast<double *>(ws + lay.fine);
  p.status = reinterpret_cast<int *>(ws);
  p.num_seqs = c.num_seqs;
  p.num_rows = c.num_rows;
  p.num_heads = c.num_heads;
  p.num_kv_heads = c.num_kv_heads;
  p.num_blocks = c.num_blocks;
  p.block_size = c.block_size;
  while ((1 << p.log2_block_size) < c.block_size) ++p.log2_block_size;
  p.max_blocks_per_seq = c.max_blocks_per_seq;
  p.max_seq_len = c.max_seq_len;
  p.max_pages = lay.max_pages;
  p.num_selected = c.num_selected;
  p.sinks = c.sinks;
  p.recent = c.recent;
  const long long items = (long long)c.num_rows * c.num_kv_heads;
  void *args[1] = {&p};
  if (c.given)
    return host_launch(reinterpret_cast<const void *>(&pa_given_blocks_kernel),
                       (unsigned)((items + 3) / 4), 1, 128, 0, c.stream, args,
                       "launch given-blocks kernel");
  // One CTA an item if that gives every SM four; otherwise chunks of at least
  // 64 pages (a round of the CTA's warps) towards that number.
  p.chunks = 1;
  p.chunk_pages = lay.max_pages > 0 ? lay.max_pages : 1;
  if (items < 4ll * sms) {
    long long want = (4ll * sms + items - 1) / items;
    const long long most = (lay.max_pages + 63) / 64;
    if (want > most) want = most;
    if (want > kSelMaxChunks) want = kSelMaxChunks;
    if (want > 1) {
      p.chunk_pages = (int)(((lay.max_pages + want - 1) / want + 63) / 64 * 64);
      p.chunks = (lay.max_pages + p.chunk_pages - 1) / p.chunk_pages;
    }
  }
  if (items * p.chunks > 0x7fffffffll) return PA_ERR_UNSUPPORTED;
  p.smem_pages = lay.max_pages < kSelSmemPages ? lay.max_pages : kSelSmemPages;
  const size_t smem = (size_t)(p.smem_pages > 0 ? p.smem_pages : 1) * 4;
  const void *fn = c.dtype == PA_DTYPE_F32    ? pick_select<float>(c.head_size)
                   : c.dtype == PA_DTYPE_BF16 ? pick_select<__nv_bfloat16>(c.head_size)
                                              : pick_select<__half>(c.head_size);
  return host_launch(fn, (unsigned)(items * p.chunks), 1, kSelThreads, smem, c.stream, args,
                     "launch select kernel");
}

}  // namespace
}  // namespace pa

extern "C" {

size_t pa_sparse_workspace_bytes(int num_rows, int num_heads, int num_kv_heads, int head_size,
                                 int block_size, int max_seq_len, int num_selected,
                                 int partition_size) {
  pa::SparseLayout lay;
  if (!pa::sparse_layout(num_rows, num_heads, num_kv_heads, head_size, block_size, max_seq_len,
                         num_selected, partition_size, &lay))
    return 0;
  return lay.total;
}

pa_status_t pa_select_blocks(int32_t *selected, const void *query, const void *key_bounds,
                             const int32_t *block_tables, const int32_t *seq_lens,
                             const int32_t *q_start, int num_seqs, int num_rows, int num_heads,
                             int num_kv_heads, int head_size, int num_blocks, int block_size,
                             int max_blocks_per_seq, int max_seq_len, int num_selected,
                             int sink_blocks, int recent_blocks, int partition_size, int dtype,
                             void *workspace, size_t workspace_bytes, void *stream) {
  using namespace pa;
  SparseCall c{selected,     nullptr,      query,        key_bounds,  block_tables,
               seq_lens,     q_start,      num_seqs,     num_rows,    num_heads,
               num_kv_heads, head_size,    num_blocks,   block_size,  max_blocks_per_seq,
               max_seq_len,  num_selected, sink_blocks,  recent_blocks, partition_size,
               dtype,        workspace,    workspace_bytes, stream};
  if (!selected || !query || !key_bounds) return PA_ERR_INVALID_ARG;
  SparseLayout lay;
  pa_status_t st = check_sparse(c, &lay);
  if (st != PA_OK || num_rows == 0) return st;
  return run_select(c, lay, false);
}

pa_status_t pa_sparse_forward(void *out, int32_t *selected, const void *query,
                              const void *key_cache, const void *value_cache,
                              const void *key_bounds, const int32_t *block_tables,
                              const int32_t *seq_lens, const int32_t *q_start, int num_seqs,
                              int num_rows, int num_heads, int num_kv_heads, int head_size,
                              int num_blocks, int block_size, int max_blocks_per_seq,
                              int max_seq_len, int num_selected, int sink_blocks,
                              int recent_blocks, float scale, int partition_size, int dtype,
                              void *workspace, size_t workspace_bytes, void *stream) {
  using namespace pa;
  const bool given = key_bounds == nullptr;
  SparseCall c{given ? nullptr : selected, given ? selected : nullptr, query, key_bounds,
               block_tables, seq_lens,     q_start,      num_seqs,     num_rows,   num_heads,
               num_kv_heads, head_size,    num_blocks,   block_size,   max_blocks_per_seq,
               max_seq_len,  num_selected, sink_blocks,  recent_blocks, partition_size,
               dtype,        workspace,    workspace_bytes, stream};
  if (!out || !query || !key_cache || !value_cache || (given && !selected))
    return PA_ERR_INVALID_ARG;
  if (!host_aligned(out, 16) || !host_aligned(key_cache, 16) || !host_aligned(value_cache, 16))
    return PA_ERR_INVALID_ARG;
  if (!(scale - scale == 0.f)) return PA_ERR_INVALID_ARG;  // not finite
  SparseLayout lay;
  pa_status_t st = check_sparse(c, &lay);
  if (st != PA_OK || num_rows == 0) return st;
  // The attention's own limits, before anything is enqueued: the view's items
  // fit its 31-bit counts.
  const long long items = (long long)num_rows * num_kv_heads;
  const long long parts = (lay.view_len + partition_size - 1) / partition_size;
  if (items * (parts > 0 ? parts : 1) >= (1ll << 31) || parts > (1 << 20))
    return PA_ERR_UNSUPPORTED;
  st = run_select(c, lay, true);
  if (st != PA_OK) return st;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  return pa_forward(out, query, key_cache, value_cache,
                    reinterpret_cast<const int32_t *>(ws + lay.table),
                    reinterpret_cast<const int32_t *>(ws + lay.lens), (int)items,
                    num_heads / num_kv_heads, 1, head_size, num_blocks * num_kv_heads, block_size,
                    num_selected, lay.view_len, scale, partition_size, dtype, workspace,
                    lay.table, stream, nullptr);
}

}  // extern "C"
