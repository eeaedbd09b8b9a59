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
// one that exact scores give (ties to the lower page).  A score in fp32 is
// within eps = gamma 2^-24 sum |Q| |bound| of the exact one: gamma counts the
// G - 1 additions in Q (all of one sign), a lane's chain of products, the
// warp's 5 additions and 3 for the sum of magnitudes itself, which is taken
// as the sum over lanes of the largest a lane saw on any page.  Where the
// scores on the two sides of the cut are more than 2 eps apart, the cut is
// the exact one.  Else the pages within 2 eps of the last one in are scored
// again in pairs of fp32 numbers: sums and products with their exact rounding
// errors carried along (the two-sum and two-product of T. J. Dekker, "A
// floating-point technique for extending the available precision", 1971), 45
// bits and more of the sum of magnitudes.  (fp64 instructions run at a
// sixty-fourth of fp32's rate on GB300: the same in fp64 took a warp 10 us at
// D 128, 20 us at D 256.)
//
// Layout of the work: an item is one (row, KV head).  Enough items: one CTA
// scores an item's pages and selects.  Few: the pages are cut into chunks, one
// CTA each, so that a single long sequence fills the GPU, and a second launch
// selects, one CTA an item (no counters to keep at zero between calls, whose
// shapes may change).  The selected pages come out in
// page order with the last page last, as a block table of the view in which
// every (row, KV head) is a sequence of one KV head: the attention kernels
// then need nothing new.
//
// Bound: the bytes of the key bounds (2 D numbers a page and KV head), with
// many items; with few, the chain of launches.  Measured on GB300 (32/4 heads,
// D 128, bf16, pages of 16; a whole pa_sparse_forward, one call after another):
//   256 sequences of 512 to 3584 tokens, 32 blocks each: 73 us, of which the
//     selection 22 (67 MB of bounds; 25 alone with a cold L2, 2.7 TB/s: every
//     item is resident, so that all score first and all select after) and the
//     attention 51 (268 MB, 5.2 TB/s);
//   one sequence of 100,000 tokens, 256 blocks: 23.5 us in four launches that
//     wait for one another (scores, selection, partitions, Phase 2), each some
//     3 us of start and dependent loads; the selection from 6250 scores is 5.
#include <math_constants.h>

#include <type_traits>

#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_ops.h"

namespace pa {
namespace {

constexpr int kSelMaxWarps = 8;     // of a CTA
constexpr int kSelList = 256;       // pages listed in shared memory
constexpr int kSelWarpPages = 256;  // candidates that one warp selects from, eight a lane
constexpr int kSelSmemPages = 8192; // keys kept in shared memory

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

// The item's row: its sequence and the keys it sees (0: none, or bad input).  By
// a warp.
__device__ __forceinline__ void locate(const SelectParams &p, int row, int &seq, int &vis) {
  seq = row;
  vis = 0;
  int before = 0, n = 1;  // the row's index in its chunk, the chunk's rows
  if (p.q_start) {
    check_starts(p.q_start, p.num_seqs, row, p.num_rows, p.status);
    const int lo = first_above(p.q_start, p.num_seqs + 1, row);
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
    if (q0 < 0 || before < 0 || before >= n || n > p.num_rows - q0) {
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

// An order-preserving map of floats (no NaN) to unsigned integers and back.
__device__ __forceinline__ uint32_t order32(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unorder32(uint32_t u) {
  return __uint_as_float((u >> 31) ? u ^ 0x80000000u : ~u);
}

// Marks of pages whose order the second scoring decided, outside the range of any float.
constexpr uint32_t kKeyIn = 0xffffffffu, kKeyOut = 0u;

struct SelShared {
  float w[512];           // Q+ then Q-, 2 D numbers
  float wide[2][512];     // the same in pairs, where needed
  uint64_t fine[kSelList];
  int list[kSelList];
  uint32_t mark[kSelList];
  int counts[32 * kSelMaxWarps];
  int red_i[2][kSelMaxWarps];
  uint32_t red_u[2][kSelMaxWarps];
  float red_f[kSelMaxWarps];
  int flag, count;
};

// Sum over the CTA, for every thread.  `turn` alternates between calls, so
// that one barrier a call suffices.
template <int WARPS>
__device__ __forceinline__ int block_sum(int v, SelShared &sh, int &turn) {
  v = __reduce_add_sync(0xffffffffu, v);
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) sh.red_i[turn][threadIdx.x >> 5] = v;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int i = 0; i < WARPS; ++i) t += sh.red_i[turn][i];
  return t;
}
// The smallest lo and the largest hi over the CTA, for every thread.
template <int WARPS>
__device__ __forceinline__ void block_min_max(uint32_t &lo, uint32_t &hi, SelShared &sh) {
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    sh.red_u[0][threadIdx.x >> 5] = lo;
    sh.red_u[1][threadIdx.x >> 5] = hi;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < WARPS; ++i) {
    lo = min(lo, sh.red_u[0][i]);
    hi = max(hi, sh.red_u[1][i]);
  }
}
template <int WARPS>
__device__ __forceinline__ float block_max(float v, SelShared &sh) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sh.red_f[threadIdx.x >> 5] = v;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < WARPS; ++i) v = fmaxf(v, sh.red_f[i]);
  return v;
}

// A sum and the rounding errors of its additions.
struct PairSum {
  float s = 0.f, c = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float t = __fadd_rn(s, x), z = __fsub_rn(t, s);
    c += __fadd_rn(__fsub_rn(s, __fsub_rn(t, z)), __fsub_rn(x, z));
    s = t;
  }
  // renormalised, as an integer of the same order (NaN lowest)
  __device__ __forceinline__ uint64_t key() const {
    float h = __fadd_rn(s, c), l = __fsub_rn(c, __fsub_rn(h, s));
    if (!(fabsf(s) <= 3.402823466e38f)) {  // beyond fp32: infinite, or NaN
      h = s != s ? -CUDART_INF_F : s;
      l = 0.f;
    }
    return (uint64_t)order32(h) << 32 | order32(l);
  }
};

// Q+ and Q- in pairs, for rescoring, by the threads from `start` in steps of
// `step`; the caller synchronises.  (What few items reach is kept in short
// loops: there, code costs its fetch.)
template <typename T, int D>
__device__ __forceinline__ void wide_weights(const T *q, int G, SelShared &sh, int start, int step) {
#pragma unroll 1
  for (int d = start; d < D; d += step) {
    PairSum qp, qn;
#pragma unroll 4
    for (int g = 0; g < G; ++g) {
      const float f = to_float(q[(size_t)g * D + d]);
      qp.add(fmaxf(f, 0.f));
      qn.add(fminf(f, 0.f));
    }
    sh.wide[0][d] = qp.s;
    sh.wide[1][d] = qp.c;
    sh.wide[0][D + d] = qn.s;
    sh.wide[1][D + d] = qn.c;
  }
}
// A page's score in pairs, by a warp (every lane gets its key).
template <typename T, int D>
__device__ __forceinline__ uint64_t fine_score(const SelectParams &p, int blk, int h, const SelShared &sh) {
  PairSum a;
  if ((unsigned)blk >= (unsigned)p.num_blocks) {
    a.s = -CUDART_INF_F;
    return a.key();
  }
  const T *b = static_cast<const T *>(p.key_bounds) + ((size_t)blk * p.num_kv_heads + h) * 2 * D;
#pragma unroll 4
  for (int d = threadIdx.x & 31; d < 2 * D; d += 32) {
    const float f = to_float(b[d]), w = sh.wide[0][d];
    const float prod = __fmul_rn(w, f);
    a.add(prod);
    a.c += fmaf(sh.wide[1][d], f, fmaf(w, f, -prod));
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const float s2 = __shfl_xor_sync(0xffffffffu, a.s, d);
    const float c2 = __shfl_xor_sync(0xffffffffu, a.c, d);
    a.c = __fadd_rn(a.c, c2);
    a.add(s2);
  }
  return a.key();
}
// The m pages listed in sh.list scored in pairs and the `more` best of them (ties
// to the lower page) marked, kKeyIn or kKeyOut, in sh.mark.
template <typename T, int D, int WARPS>
__device__ __forceinline__ void rescore_list(const SelectParams &p, const T *q, const int32_t *bt, int h,
                                             int G, int m, int more, SelShared &sh) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  wide_weights<T, D>(q, G, sh, tid, WARPS * 32);
  __syncthreads();  // (also publishes the list)
#pragma unroll 1
  for (int j = warp; j < m; j += WARPS) {
    const uint64_t s = fine_score<T, D>(p, __ldg(bt + sh.list[j]), h, sh);
    if (lane == 0) sh.fine[j] = s;
  }
  __syncthreads();
  for (int j0 = tid; j0 < m; j0 += WARPS * 32) {
    const uint64_t s = sh.fine[j0];
    const int i = sh.list[j0];
    int rank = 0;
    for (int j = 0; j < m; ++j) {
      const uint64_t t = sh.fine[j];
      rank += t > s || (t == s && sh.list[j] < i);
    }
    sh.mark[j0] = rank < more ? kKeyIn : kKeyOut;
  }
  __syncthreads();
}

// The highest bit in which keys between lo and hi can differ (-1: none) and
// the bits above it, where the search for a cut starts.
__device__ __forceinline__ int first_bit(uint32_t lo, uint32_t hi, uint32_t &cut) {
  const int bit = lo == hi ? -1 : 31 - __clz(lo ^ hi);
  cut = bit < 0 ? lo : bit == 31 ? 0u : (hi >> (bit + 1)) << (bit + 1);
  return bit;
}

// The need best of the cand pages from `first` on, by the whole CTA with up to
// REGS keys a thread in registers, listed in page order.  False (nothing
// listed) if more pages than the list holds are too close to call.
template <typename T, int D, int WARPS, int REGS>
__device__ __forceinline__ bool select_in_registers(const SelectParams &p, const T *q, const int32_t *bt,
                                                    const uint32_t *kc, int32_t *list, int h, int G,
                                                    int first, int cand, int need, float eps,
                                                    SelShared &sh) {
  constexpr int THREADS = WARPS * 32;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // one barrier a bit
  int turn = 0;
  uint32_t key[REGS];
  uint32_t klo = 0xffffffffu, khi = 0u;
  // (no early ends in these loops: a missing page's key is below every
  // score and cut, and a branch a round would cost more than the round)
#pragma unroll
  for (int v = 0; v < REGS; ++v) {
    const int i = tid + v * THREADS;
    key[v] = i < cand ? kc[first + i] : kKeyOut;
  }
#pragma unroll
  for (int v = 0; v < REGS; ++v) {
    klo = min(klo, key[v] == kKeyOut ? 0xffffffffu : key[v]);
    khi = max(khi, key[v]);
  }
  block_min_max<WARPS>(klo, khi, sh);
  uint32_t cut;
  int have = cand;
  for (int bit = first_bit(klo, khi, cut); bit >= 0 && have != need; --bit) {
    const uint32_t mid = cut | (1u << bit);
    int c = 0;
#pragma unroll
    for (int v = 0; v < REGS; ++v) {
      c += key[v] >= mid;
    }
    c = block_sum<WARPS>(c, sh, turn);
    if (c >= need) {
      cut = mid;
      have = c;
    }
  }
  uint32_t ka = 0xffffffffu, kb = 0u;
#pragma unroll
  for (int v = 0; v < REGS; ++v) {
    if (key[v] >= cut)
      ka = min(ka, key[v]);
    else
      kb = max(kb, key[v]);
  }
  block_min_max<WARPS>(ka, kb, sh);
  const float tau = unorder32(ka);
  bool done = have == need && tau - unorder32(kb) > 2.f * eps;
  if (!done) {
    const float fhi = tau + 2.f * eps, flo = tau - 2.f * eps;
    const uint32_t hi = fhi == fhi ? order32(fhi) : kKeyIn - 1;
    const uint32_t lo = flo == flo ? order32(flo) : kKeyOut + 1;
    int c = 0, m = 0;
#pragma unroll
    for (int v = 0; v < REGS; ++v) {
      c += key[v] > hi;
      m += key[v] >= lo && key[v] <= hi;
    }
    if (tid == 0) sh.count = 0;
    const int more = need - block_sum<WARPS>(c, sh, turn);
    m = block_sum<WARPS>(m, sh, turn);
    if (m <= kSelList) {
#pragma unroll
      for (int v = 0; v < REGS; ++v) {
        if (key[v] >= lo && key[v] <= hi)
          sh.list[atomicAdd(&sh.count, 1)] = first + tid + v * THREADS;
      }
      rescore_list<T, D, WARPS>(p, q, bt, h, G, m, more, sh);
#pragma unroll
      for (int v = 0; v < REGS; ++v) {
        if (key[v] >= lo && key[v] <= hi)
          for (int j = 0; j < m; ++j)
            if (sh.list[j] == first + tid + v * THREADS) {
              key[v] = sh.mark[j];
              break;
            }
      }
      cut = hi + 1;
      done = true;
      __syncthreads();  // the list is free for the pages chosen
    }
  }
  if (done) {
    // in page order: round v before round v + 1, warp by warp in each
#pragma unroll
    for (int v = 0; v < REGS; ++v) {
      const unsigned m = __ballot_sync(0xffffffffu, key[v] >= cut);
      if (lane == 0) sh.counts[v * WARPS + warp] = __popc(m);
    }
    __syncthreads();
    if (warp == 0) {  // running sums, a few a lane
      constexpr int PER = REGS * WARPS / 32;
      int c[PER], sum = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        c[i] = sh.counts[lane * PER + i];
        sum += c[i];
      }
      int run = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, run, d);
        if (lane >= d) run += t;
      }
      run -= sum;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        sh.counts[lane * PER + i] = run;
        run += c[i];
      }
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < REGS; ++v) {
      const unsigned m = __ballot_sync(0xffffffffu, key[v] >= cut);
      if (key[v] >= cut)
        list[sh.counts[v * WARPS + warp] + __popc(m & ((1u << lane) - 1u))] =
            first + tid + v * THREADS;
    }
  }
  __syncthreads();
  return done;
}

}  // namespace

// Dynamic shared memory: the keys (order32 of the scores) of p.smem_pages
// pages.
template <typename T, int D, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, WARPS == 4 ? 8 : 3)
    pa_select_kernel(const __grid_constant__ SelectParams p) {
  // (at most 64 registers a thread with four warps, whose items should all be
  // resident; 80 with eight, which hold more keys: 61 against 65 us a call for
  // 64 sequences of up to 4096 pages at D 256)
  constexpr int THREADS = WARPS * 32;
  constexpr int N = 16 / (int)sizeof(T);       // elements of a 16-byte piece
  constexpr int PIECES = 2 * D / N;            // of a page's bounds
  constexpr int LPP = PIECES < 32 ? PIECES : 32;  // lanes of a page
  constexpr int VPL = PIECES / LPP;            // pieces a lane
  constexpr int PPW = 32 / LPP;                // pages of a warp side by side
  constexpr int SEG = VPL <= 1 ? 8 : 8 / VPL;  // pages of a warp at a time: 32 registers' worth
  __shared__ SelShared sh;
  extern __shared__ __align__(16) uint32_t s_keys[];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int parts = p.mode == kSelPick ? 1 : p.chunks;
  const int item = blockIdx.x / parts, chunk = blockIdx.x % parts;
  const int row = item / p.num_kv_heads, h = item % p.num_kv_heads;
  const int G = p.num_heads / p.num_kv_heads;

  // the row's queries and (one row a sequence) its table, on their way to L2
  // while the kernel before this one ends
  const T *q = static_cast<const T *>(p.query) + ((size_t)row * p.num_heads + h * G) * D;
  for (int i = tid * 128; i < G * D * (int)sizeof(T); i += THREADS * 128)
    prefetch_l2(reinterpret_cast<const char *>(q) + i);
  if (tid == 0) prefetch_l2(p.seq_lens + (p.q_start ? 0 : row));
  if (!p.q_start && tid * 32 < p.chunk_pages)
    prefetch_l2(p.block_tables + (size_t)row * p.max_blocks_per_seq +
                min(chunk * p.chunk_pages + tid * 32, p.max_blocks_per_seq - 1));
  pdl_wait_primary();
  pdl_launch_dependents();
  int seq, vis;
  locate(p, row, seq, vis);
  const int n = (vis + p.block_size - 1) >> p.log2_block_size;  // pages the row sees
  const int32_t *bt = p.block_tables + (size_t)seq * p.max_blocks_per_seq;
  const int k = p.num_selected;
  const bool all = n <= k;
  const int nch = (n + p.chunk_pages - 1) / p.chunk_pages;
  if (p.mode == kSelScore && (all || chunk >= nch)) return;
  const int first = p.sinks, last = n - p.recent;  // pages [first, last) go by their score
  const int need = k - p.sinks - p.recent;         // of them
  // the keys: in shared memory if the CTA scores them all and they fit
  uint32_t *kc = p.mode == kSelBoth && n <= p.smem_pages ? s_keys : p.keys + (size_t)item * p.max_pages;
  int32_t *selected = p.selected ? p.selected + (size_t)item * k : nullptr;
  int32_t *table = p.table ? p.table + (size_t)item * k : nullptr;
  // where the chosen candidates' pages are listed, in page order
  int32_t *list = need <= kSelList ? sh.list : (table ? table : selected) + p.sinks;

  float size = 0.f;  // the largest sum |Q| |bound| of a page
  if (!all && p.mode != kSelPick) {
    // ---- Q+ and Q-: the group's loads all in flight ----
    for (int d = tid; d < D; d += THREADS) {
      float qp = 0.f, qn = 0.f;
#pragma unroll
      for (int g = 0; g < 16; ++g) {
        const float f = g < G ? to_float(q[(size_t)g * D + d]) : 0.f;
        qp += fmaxf(f, 0.f);
        qn += fminf(f, 0.f);
      }
      sh.w[d] = qp;
      sh.w[D + d] = qn;
    }
    __syncthreads();

    // ---- scores of the chunk's pages ----
    float w[VPL][N];
    const int lp = lane % LPP;
#pragma unroll
    for (int v = 0; v < VPL; ++v)
#pragma unroll
      for (int e = 0; e < N; ++e) w[v][e] = sh.w[(v * LPP + lp) * N + e];
    const int c_end = min(n, (chunk + 1) * p.chunk_pages);
    constexpr int STEPS = SEG / PPW;
    // the page whose score this lane ends up with (below), of the warp's SEG
    constexpr int SPLIT = STEPS == 8 ? 3 : STEPS == 4 ? 2 : STEPS == 2 ? 1 : 0;
    const int my_page = (lp >> (LPP == 32 ? 5 - SPLIT : 4 - SPLIT)) * PPW + lane / LPP;
    const bool my_turn = (lp & ((LPP >> SPLIT) - 1)) == 0;
    auto entry = [&](int p0) -> int {  // -1 past the chunk: those lanes load nothing
      return lane < SEG && p0 + lane < c_end ? __ldg(bt + p0 + lane) : -1;
    };
    const int p_first = chunk * p.chunk_pages + warp * SEG;
    int next = entry(p_first);
    for (int p0 = p_first; p0 < c_end; p0 += WARPS * SEG) {
      int blk = next;
      next = entry(p0 + WARPS * SEG);
      if ((unsigned)blk >= (unsigned)p.num_blocks) {
        if (lane < SEG && p0 + lane < c_end) report(p.status, kStatusBadInput);
        blk = -1;
      }
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
        float mag = 0.f;
#pragma unroll
        for (int v = 0; v < VPL; ++v) {
          float f[N];
          widen<T>(x[j][v], f);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            acc[j] = fmaf(w[v][e], f[e], acc[j]);
            mag = fmaf(fabsf(w[v][e]), fabsf(f[e]), mag);
          }
        }
        size = fmaxf(size, mag);
      }
      // The sums over a page's lanes, the STEPS pages' together: halves of the
      // lanes exchange halves of the pages until each holds one.
      int off = LPP / 2;
#pragma unroll
      for (int c = STEPS / 2; c > 0; c >>= 1) {
        const bool up = (lane & off) != 0;
#pragma unroll
        for (int j = 0; j < c; ++j) {
          const float give = up ? acc[j] : acc[j + c];
          acc[j] = (up ? acc[j + c] : acc[j]) + __shfl_xor_sync(0xffffffffu, give, off);
        }
        off >>= 1;
      }
#pragma unroll
      for (int d = LPP >> (SPLIT + 1); d > 0; d >>= 1) acc[0] += __shfl_xor_sync(0xffffffffu, acc[0], d);
      const int b = __shfl_sync(0xffffffffu, blk, my_page);
      if (my_turn && p0 + my_page < c_end)
        kc[p0 + my_page] = order32(b < 0 || acc[0] != acc[0] ? -CUDART_INF_F : acc[0]);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) size += __shfl_xor_sync(0xffffffffu, size, d);
    size = block_max<WARPS>(size, sh);  // (its barriers also publish the keys)
    if (p.mode == kSelScore) {
      if (tid == 0) p.sizes[(size_t)item * p.chunks + chunk] = size;
      return;
    }
  }
  if (!all) {
    if (p.mode == kSelPick) {
      for (int c = tid; c < nch; c += THREADS)
        size = fmaxf(size, p.sizes[(size_t)item * p.chunks + c]);
      size = block_max<WARPS>(size, sh);
    }
    const float eps = (float)(G + VPL * N + 7) * 5.9604644775390625e-8f * size + 1e-36f;

    // ---- the need best of pages [first, last) ----
    // A cut with exactly need keys at or above it, by bisection on the keys'
    // bits from the highest in which any two differ.  It is exact if the
    // scores on its two sides are more than 2 eps apart.
    const int cand = last - first;  // more than need
    bool done = need == 0;
    if (!done && cand <= kSelWarpPages) {
      // one warp, the keys in registers, no barriers
      if (warp == 0) {
        uint32_t key[kSelWarpPages / 32];
        uint32_t klo = 0xffffffffu, khi = 0u;
#pragma unroll
        for (int v = 0; v < kSelWarpPages / 32; ++v) {
          const int i = lane + 32 * v;
          key[v] = i < cand ? kc[first + i] : kKeyOut;  // below every score
          klo = min(klo, i < cand ? key[v] : 0xffffffffu);
          khi = max(khi, key[v]);
        }
        klo = __reduce_min_sync(0xffffffffu, klo);
        khi = __reduce_max_sync(0xffffffffu, khi);
        uint32_t cut;
        int have = cand;
        for (int bit = first_bit(klo, khi, cut); bit >= 0 && have != need; --bit) {
          const uint32_t mid = cut | (1u << bit);
          int c = 0;
#pragma unroll
          for (int v = 0; v < kSelWarpPages / 32; ++v) c += key[v] >= mid;
          c = __reduce_add_sync(0xffffffffu, c);
          if (c >= need) {
            cut = mid;
            have = c;
          }
        }
        uint32_t ka = 0xffffffffu, kb = 0u;
#pragma unroll
        for (int v = 0; v < kSelWarpPages / 32; ++v) {
          if (key[v] >= cut)
            ka = min(ka, key[v]);
          else
            kb = max(kb, key[v]);
        }
        ka = __reduce_min_sync(0xffffffffu, ka);
        kb = __reduce_max_sync(0xffffffffu, kb);
        const float tau = unorder32(ka);
        bool exact = have == need && tau - unorder32(kb) > 2.f * eps;
        if (!exact) {
          // up to 32 pages between: scored again here, one lane each to keep
          const float fhi = tau + 2.f * eps, flo = tau - 2.f * eps;
          const uint32_t hi = fhi == fhi ? order32(fhi) : kKeyIn - 1;
          const uint32_t lo = flo == flo ? order32(flo) : kKeyOut + 1;
          int c = 0, m = 0, mine = -1;
#pragma unroll
          for (int v = 0; v < kSelWarpPages / 32; ++v) {
            c += key[v] > hi;
            const bool in = key[v] >= lo && key[v] <= hi;
            const unsigned b = __ballot_sync(0xffffffffu, in);
            // lane m + r takes the r-th of them
            const int r = lane - m;
            if (r >= 0 && r < __popc(b)) mine = 32 * v + __fns(b, 0, r + 1);
            m += __popc(b);
          }
          const int more = need - __reduce_add_sync(0xffffffffu, c);
          if (m <= 32) {
            wide_weights<T, D>(q, G, sh, lane, 32);
            __syncwarp();
            uint64_t score = 0;
#pragma unroll 1
            for (int j = 0; j < m; ++j) {
              const uint64_t t =
                  fine_score<T, D>(p, __ldg(bt + first + __shfl_sync(0xffffffffu, mine, j)), h, sh);
              if (lane == j) score = t;
            }
            int rank = 0;
#pragma unroll 1
            for (int j = 0; j < m; ++j) {
              const uint64_t t = __shfl_sync(0xffffffffu, score, j);
              rank += t > score || (t == score && j < lane);  // in page order already
            }
#pragma unroll 1
            for (int j = 0; j < m; ++j) {
              const int i = __shfl_sync(0xffffffffu, mine, j);
              const uint32_t mark = __shfl_sync(0xffffffffu, rank, j) < more ? kKeyIn : kKeyOut;
#pragma unroll
              for (int v = 0; v < kSelWarpPages / 32; ++v)
                if (i == lane + 32 * v) key[v] = mark;
            }
            cut = hi + 1;
            exact = true;
          }
        }
        if (exact) {
          int at = 0;
#pragma unroll
          for (int v = 0; v < kSelWarpPages / 32; ++v) {
            const unsigned m = __ballot_sync(0xffffffffu, key[v] >= cut);
            if (key[v] >= cut) list[at + __popc(m & ((1u << lane) - 1u))] = first + lane + 32 * v;
            at += __popc(m);
          }
        }
        if (lane == 0) sh.flag = exact;
      }
      __syncthreads();
      done = sh.flag;
    } else if (!done && cand <= 8 * THREADS) {
      done = select_in_registers<T, D, WARPS, 8>(p, q, bt, kc, list, h, G, first, cand, need, eps, sh);
    } else if (WARPS == 8 && !done && cand <= 32 * THREADS) {
      done = select_in_registers<T, D, WARPS, 32>(p, q, bt, kc, list, h, G, first, cand, need, eps, sh);
    }
    if (!done) {
      int turn = 0;
      uint32_t klo = 0xffffffffu, khi = 0u;
#pragma unroll 4
      for (int i = first + tid; i < last; i += THREADS) {
        const uint32_t u = kc[i];
        klo = min(klo, u);
        khi = max(khi, u);
      }
      block_min_max<WARPS>(klo, khi, sh);
      uint32_t cut;
      int have = cand;
      for (int bit = first_bit(klo, khi, cut); bit >= 0 && have != need; --bit) {
        const uint32_t mid = cut | (1u << bit);
        int c = 0;
#pragma unroll 8
        for (int i = first + tid; i < last; i += THREADS) c += kc[i] >= mid;
        c = block_sum<WARPS>(c, sh, turn);
        if (c >= need) {
          cut = mid;
          have = c;
        }
      }
      // tau, the need-th largest score, is the lowest above the cut
      uint32_t ka = 0xffffffffu, kb = 0u;
#pragma unroll 4
      for (int i = first + tid; i < last; i += THREADS) {
        const uint32_t u = kc[i];
        if (u >= cut)
          ka = min(ka, u);
        else
          kb = max(kb, u);
      }
      block_min_max<WARPS>(ka, kb, sh);
      const float tau = unorder32(ka);
      if (!(have == need && tau - unorder32(kb) > 2.f * eps)) {
        // Pages above hi are in, pages below lo out; those between (all of
        // them, if eps is not finite) are scored again in pairs.
        const float fhi = tau + 2.f * eps, flo = tau - 2.f * eps;
        const uint32_t hi = fhi == fhi ? order32(fhi) : kKeyIn - 1;
        const uint32_t lo = flo == flo ? order32(flo) : kKeyOut + 1;
        int c = 0, m = 0;
        for (int i = first + tid; i < last; i += THREADS) {
          c += kc[i] > hi;
          m += kc[i] >= lo && kc[i] <= hi;
        }
        const int more = need - block_sum<WARPS>(c, sh, turn);  // of the m in between
        m = block_sum<WARPS>(m, sh, turn);
        if (tid == 0) sh.count = 0;
        __syncthreads();
        if (m <= kSelList) {
          for (int i = first + tid; i < last; i += THREADS)
            if (kc[i] >= lo && kc[i] <= hi) sh.list[atomicAdd(&sh.count, 1)] = i;
          rescore_list<T, D, WARPS>(p, q, bt, h, G, m, more, sh);
          for (int j = tid; j < m; j += THREADS) kc[sh.list[j]] = sh.mark[j];
        } else {
          uint64_t *gfine = p.fine + (size_t)item * p.max_pages;
          wide_weights<T, D>(q, G, sh, tid, THREADS);
          __syncthreads();
          for (int i = first + warp; i < last; i += WARPS) {
            if (kc[i] > hi || kc[i] < lo) continue;
            const uint64_t s = fine_score<T, D>(p, __ldg(bt + i), h, sh);
            if (lane == 0) gfine[i] = s;
          }
          __syncthreads();
          // the more-th largest by bisection, then its ties in page order
          uint64_t t = 0;
          for (int b = 63; b >= 0; --b) {
            const uint64_t mid = t | (1ull << b);
            int cnt = 0;
            for (int i = first + tid; i < last; i += THREADS)
              if (kc[i] >= lo && kc[i] <= hi) cnt += gfine[i] >= mid;
            if (block_sum<WARPS>(cnt, sh, turn) >= more) t = mid;
          }
          int cnt = 0;
          for (int i = first + tid; i < last; i += THREADS)
            if (kc[i] >= lo && kc[i] <= hi) cnt += gfine[i] > t;
          int ties = more - block_sum<WARPS>(cnt, sh, turn);
          if (warp == 0) {
            for (int i0 = first; i0 < last; i0 += 32) {
              const int i = i0 + lane;
              const bool in = i < last && kc[i] >= lo && kc[i] <= hi;
              const uint64_t u = in ? gfine[i] : 0;
              const unsigned eq = __ballot_sync(0xffffffffu, in && u == t);
              const bool keep = in && (u > t || (u == t && __popc(eq & ((1u << lane) - 1u)) < ties));
              ties = max(0, ties - __popc(eq));
              if (in) kc[i] = keep ? kKeyIn : kKeyOut;
            }
          }
        }
        __syncthreads();
        cut = hi + 1;  // those above and the marks
      }
      // the chosen candidates in page order, a segment a warp
      const int seg = ((cand + WARPS - 1) / WARPS + 31) / 32 * 32;
      const int s0 = first + min(cand, warp * seg), s1 = min(last, s0 + seg);
      int cnt = 0;
#pragma unroll 4
      for (int i = s0 + lane; i < s1; i += 32) cnt += kc[i] >= cut;
      cnt = __reduce_add_sync(0xffffffffu, cnt);
      turn ^= 1;
      if (lane == 0) sh.red_i[turn][warp] = cnt;
      __syncthreads();
      int at = 0;
      for (int i = 0; i < warp; ++i) at += sh.red_i[turn][i];
#pragma unroll 4
      for (int i0 = s0; i0 < s1; i0 += 32) {
        const int i = i0 + lane;
        const bool in = i < s1 && kc[i] >= cut;
        const unsigned m = __ballot_sync(0xffffffffu, in);
        const int o = at + __popc(m & ((1u << lane) - 1u));
        if (in && o < need) list[o] = i;
        at += __popc(m);
      }
      __syncthreads();
    }
  }
  // ---- the selected pages, in page order ----
  for (int o = tid; o < k; o += THREADS) {
    const int i = all ? (o < n ? o : -1)
                  : o < p.sinks       ? o
                  : o < k - p.recent  ? list[o - p.sinks]
                                      : n - (k - o);
    if (selected) selected[o] = i;
    if (table) table[o] = i >= 0 ? view_block(__ldg(bt + i), h, p.num_kv_heads, p.num_blocks) : -1;
  }
  if (tid == 0 && p.lens)
    p.lens[item] = all ? vis : (k - 1) * p.block_size + vis - (n - 1) * p.block_size;
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

template <typename T, int WARPS>
const void *pick_select(int head_size) {
  switch (head_size) {
    case 64: return reinterpret_cast<const void *>(&pa_select_kernel<T, 64, WARPS>);
    case 128: return reinterpret_cast<const void *>(&pa_select_kernel<T, 128, WARPS>);
    case 256: return reinterpret_cast<const void *>(&pa_select_kernel<T, 256, WARPS>);
  }
  return nullptr;
}
template <typename T>
const void *pick_select(int head_size, int warps) {
  return warps == 4 ? pick_select<T, 4>(head_size) : pick_select<T, 8>(head_size);
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// The workspace: the attention's over the view, then table, lengths
// and what the selection keeps a page.
struct SparseLayout {
  size_t table, lens, sizes, keys, fine, total;
  int max_pages, view_len;
  int partition;  // of the view's attention
};
constexpr int kSelMaxChunks = 1024;  // of an item
constexpr int kViewItems = 4 * 152;  // of the attention, four an SM

// The partition of the view's attention: the caller's, halved while that still
// gives at most four items an SM (32 rows of 4 KV heads, 48 blocks of 16: 29.9 us
// a call in partitions of 256, 34.5 in 512, 31.0 in 128).
int view_partition(long long items, int view_len, int partition_size, int block_size) {
  int p = partition_size;
  while (p % 2 == 0 && (p / 2) % 64 == 0 && (p / 2) % block_size == 0 && p / 2 < view_len &&
         items * ((view_len + p / 2 - 1) / (p / 2)) <= kViewItems)
    p /= 2;
  return p;
}

bool sparse_layout(int num_rows, int num_heads, int num_kv_heads, int head_size, int block_size,
                   int max_seq_len, int num_selected, int partition_size, SparseLayout *o) {
  if (num_rows < 0 || num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads ||
      head_size < 1 || block_size < 1 || max_seq_len < 0 || num_selected < 1 || partition_size < 1)
    return false;
  const long long items = (long long)num_rows * num_kv_heads;
  const long long cap = (long long)num_selected * block_size;
  if (items > 0x7fffffffll || cap > 0x7fffffffll || max_seq_len > kMaxTokens) return false;
  o->max_pages = (int)(((long long)max_seq_len + block_size - 1) / block_size);
  o->view_len = (int)(cap < max_seq_len ? cap : max_seq_len);
  o->partition = view_partition(items, o->view_len, partition_size, block_size);
  const int group = num_heads / num_kv_heads;
  size_t attn = pa_workspace_bytes((int)items, group, head_size, o->view_len, o->partition);
  if (attn == 0) return false;
  // never less than what a call with fewer rows, in smaller partitions, needs
  const size_t few = pa_workspace_bytes(kViewItems, group, head_size, 1, 64);
  if (attn < few) attn = few;
  o->table = align256(attn);
  o->lens = o->table + align256((size_t)items * num_selected * 4);
  o->sizes = o->lens + align256((size_t)items * 4);
  const int chunks = (o->max_pages + 63) / 64;
  o->keys = o->sizes + align256((size_t)items * (chunks < kSelMaxChunks ? chunks : kSelMaxChunks) * 4);
  o->fine = o->keys + align256((size_t)items * o->max_pages * 4);
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
  if (c.num_rows == 0) return PA_OK;  // (empty tensors have no address)
  if (!c.query || !c.block_tables || !c.seq_lens || !c.workspace) return PA_ERR_INVALID_ARG;
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
  p.sizes = reinterpret_cast<float *>(ws + lay.sizes);
  p.keys = reinterpret_cast<uint32_t *>(ws + lay.keys);
  p.fine = reinterpret_cast<uint64_t *>(ws + lay.fine);
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
  // One CTA an item if that gives every SM four.  Otherwise chunks, towards 32
  // CTAs an SM: with lengths of all kinds in a batch, a long sequence's chunks
  // are what the last SMs wait for (64 sequences of up to 4096 pages, D 256, a
  // call: 77 us at eight an SM, 65 at 16, 63 at 32, 67 at 64).  A chunk is at
  // least two rounds of the CTA's warps (128 pages; 32 rows of up to 512 pages:
  // 29.3 us a call, 30.9 in chunks of one round), or one where that leaves SMs
  // with less than two CTAs (one row of 6250 pages: 23.5 us, 24.1 with two).
  p.chunks = 1;
  p.chunk_pages = lay.max_pages > 0 ? lay.max_pages : 1;
  if (items < 4ll * sms) {
    const int least = items * ((lay.max_pages + 127) / 128) >= 2ll * sms ? 128 : 64;
    long long want = (32ll * sms + items - 1) / items;
    const long long most = (lay.max_pages + least - 1) / least;
    if (want > most) want = most;
    if (want > kSelMaxChunks) want = kSelMaxChunks;
    if (want > 1) {
      p.chunk_pages = (int)(((lay.max_pages + want - 1) / want + least - 1) / least * least);
      p.chunks = (lay.max_pages + p.chunk_pages - 1) / p.chunk_pages;
    }
  }
  if (items * p.chunks > 0x7fffffffll) return PA_ERR_UNSUPPORTED;
  p.smem_pages = p.chunks > 1 ? 0 : lay.max_pages < kSelSmemPages ? lay.max_pages : kSelSmemPages;
  const size_t smem = (size_t)p.smem_pages * 4;
  // Whole items: four warps, so that the items of a decode batch are all
  // resident at once (1024 items: one wave, where eight warps took two).
  // Chunks: eight, for the launch that selects from all of an item's pages.
  const int warps = p.chunks == 1 ? 4 : 8;
  const void *fn = c.dtype == PA_DTYPE_F32    ? pick_select<float>(c.head_size, warps)
                   : c.dtype == PA_DTYPE_BF16 ? pick_select<__nv_bfloat16>(c.head_size, warps)
                                              : pick_select<__half>(c.head_size, warps);
  p.mode = p.chunks == 1 ? kSelBoth : kSelScore;
  st = host_launch(fn, (unsigned)(items * p.chunks), 1, warps * 32, smem, c.stream, args,
                   "launch select kernel");
  if (st != PA_OK || p.chunks == 1) return st;
  p.mode = kSelPick;
  return host_launch(fn, (unsigned)items, 1, warps * 32, 0, c.stream, args, "launch select kernel");
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
  SparseLayout lay;
  pa_status_t st = check_sparse(c, &lay);
  if (st != PA_OK || num_rows == 0) return st;
  if (!selected || !key_bounds) return PA_ERR_INVALID_ARG;
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
  if (!(scale - scale == 0.f)) return PA_ERR_INVALID_ARG;  // not finite
  SparseLayout lay;
  pa_status_t st = check_sparse(c, &lay);
  if (st != PA_OK || num_rows == 0) return st;
  if (!out || !key_cache || !value_cache || (given && !selected)) return PA_ERR_INVALID_ARG;
  if (!host_aligned(out, 16) || !host_aligned(key_cache, 16) || !host_aligned(value_cache, 16))
    return PA_ERR_INVALID_ARG;
  // The attention's own limits, before anything is enqueued: the view's items
  // fit its 31-bit counts.
  const long long items = (long long)num_rows * num_kv_heads;
  const long long parts = (lay.view_len + lay.partition - 1) / lay.partition;
  if (items * (parts > 0 ? parts : 1) >= (1ll << 31) || parts > (1 << 20))
    return PA_ERR_UNSUPPORTED;
  st = run_select(c, lay, true);
  if (st != PA_OK) return st;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  return pa_forward(out, query, key_cache, value_cache,
                    reinterpret_cast<const int32_t *>(ws + lay.table),
                    reinterpret_cast<const int32_t *>(ws + lay.lens), (int)items,
                    num_heads / num_kv_heads, 1, head_size, num_blocks * num_kv_heads, block_size,
                    num_selected, lay.view_len, scale, lay.partition, dtype, workspace,
                    lay.table, stream, nullptr);
}

}  // extern "C"
