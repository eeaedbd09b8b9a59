// Decode attention over a prefix that a group of sequences shares: Phase 1 of
// pa_prefix_forward, on the 5th-generation tensor cores (tcgen05, sm_103a).
//
// For the rows (sequence, head) of a group and one KV head, and one split of
// the prefix's keys,
//   S = Q K^T,  m = max_k S,  l = sum_k exp(S - m),  O = exp(S - m) V / l,
// the three going to the workspace as one more partition of every row's own
// (Phase 2 merges them with the log-sum-exp rule).  The prefix's keys and
// values are read once for all the rows of an item, so with many rows this is
// a matrix product and bound by the tensor cores, with few by the read of the
// prefix.
//
// An item is up to NT x 128 rows of a (group, KV head) and one split.  The CTA
// holds the rows' queries in shared memory and streams the split through a
// ring of slots (TMA, whole pages): K of stage j, V of stage j, K of stage
// j + 1, ...  One thread issues the MMAs.  S lives in tensor memory, fp32, one
// row a lane; a softmax thread owns a row: its maximum and sum need no
// shuffles.  P goes back over S's columns, rounded to the input type (a weight
// is off by 2^-8 of itself at most in bf16; in f16 by 2^-11, or 2^-32 of the
// split's largest weight where that is more), and is the PV product's A operand
// straight from tensor memory.  The sum adds the rounded weights, so that those
// that V is multiplied with sum to one.
//   D 64, 128: two row tiles (NT 2) share every stage of 128 keys; while the
//     softmax of one runs, the tensor cores work on the other:
//     PV_0(j) S_0(j+1) PV_1(j) S_1(j+1) ...
//     Tensor memory: S_0 S_1 (128 columns each), O_0 O_1 (D each).
//   D 256: O takes 256 columns, so one tile (NT 1), stages of 64 keys and two
//     S buffers: S(j+1) is issued before PV(j).
// MMAs of one thread execute in order, so a PV has read its P before the next
// S of that buffer overwrites it, and a commit behind an S also covers the PV
// before it.  The running maximum is raised lazily: O is rescaled only when a
// stage's exceeds it by more than 2^8, or when the key would outweigh half of all
// before it: the weight of the running maximum itself is 1 and exact, any other's
// is rounded, which shows where few keys carry the result.  (Raised beyond 2^8
// only, one of 7e5 results left the parity bar with logits of standard deviation
// 6, the worst by 1.4; with half, the worst is at 0.74 of it, and at 0.63 if every
// new maximum is taken.  256 behind 8192 tokens 62.0 -> 61.2 us, 8 behind 100,000
// 49.0 -> 50.5 us.)
//
// Measured on GB300 (a whole call, one after another; 32/4 heads, bf16, D 128):
//   256 sequences behind 8192 tokens, 16 to 512 of their own: 61.0 us (96
//     items of 22 stages; the own tokens' Phase 1 runs beside them).  First
//     scores at 6 us, the items' ends at 41 to 48, the own tokens' last item at
//     55, Phase 2 from 57 to 61.  In the steady state a stage of both tiles
//     takes 3000 clocks (3400 where O is rescaled, the first stages as a rule)
//     against 2048 of its MMAs: a tile's chain S, softmax, PV is what bounds it,
//     with the tensor pipe 0.68 busy.
//   8 sequences behind 100,000 tokens (205 MB): 50.5 us, 4.1 TB/s; a stage takes
//     2740 clocks (3100 where O is rescaled), what its bytes take at the copy
//     rate, and the rest is start, epilogue and Phase 2.
// Two softmax threads a row were slower (3200 clocks a stage and more: the
// exchange of their maxima joins the chain), an epilogue in full lines through
// shared memory the same.
#include <math_constants.h>

#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_ops.h"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr int kTileRows = 128;      // the MMA's M
// The running maximum is raised when a stage's is above it by more than this, in
// log2 units, or by so much that the key would weigh more than 2^-kLazyShare of
// all keys before it together.
constexpr float kLazyMargin = 8.f, kLazyShare = 1.f;
// Weights are 2^(s - m + this): a weight below f16's normal range loses bits
// and below 2^-25 becomes zero, so f16's start 2^7 higher (with the margin
// 2^15, below its largest number).  The sum takes the factor out again.
template <typename T>
constexpr float kWeightShift = std::is_same<T, __half>::value ? 7.f : 0.f;

template <int D>
struct PrefixShape {
  static constexpr int NT = D == 256 ? 1 : 2;       // row tiles of an item
  static constexpr int KEYS = D == 256 ? 64 : 128;  // keys of a stage
  static constexpr int SLOTS = D == 64 ? 10 : 5;    // K or V of a stage each
  static constexpr int PANELS = D * 2 / 128;        // 128-byte panels of a row
  static constexpr int GROUP = PANELS * 1024;       // bytes of 8 keys
  static constexpr int SLOT = KEYS / 8 * GROUP;
  static constexpr int QPANEL = kTileRows * 128;
  static constexpr int QTILE = PANELS * QPANEL;
  static constexpr int SOFTMAX_WARPS = 4 * NT;
  // K's producer, the MMA warp, V's producer.  NT 2: a whole third warpgroup
  // (one idle warp) whose registers the softmax warps take over: a row's 128
  // scores stay in registers
  static constexpr int THREADS = (SOFTMAX_WARPS + (NT == 2 ? 4 : 3)) * 32;
  // full and empty of each slot, Q ready a tile, S, P and (NT 2) half of P
  // ready a buffer, O done a tile, PV done (NT 1), drain, never
  static constexpr int BARS = 2 * SLOTS + 2 + 2 + 2 + 2 + 2 + 3;
  static constexpr size_t SMEM = (size_t)NT * QTILE + (size_t)SLOTS * SLOT + BARS * 8 + 16;
};

// pairs of floats, one instruction for both
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// lo += the low half of x (two numbers of type T), hi += the high half, in fp32
template <typename T>
__device__ __forceinline__ void add_halves(uint32_t x, float &lo, float &hi) {
  if constexpr (std::is_same<T, __half>::value)
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n add.rn.f32.f16 %0, l, %0;\n"
        " add.rn.f32.f16 %1, h, %1;\n}"
        : "+f"(lo), "+f"(hi)
        : "r"(x));
  else
    asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n add.rn.f32.bf16 %0, l, %0;\n"
        " add.rn.f32.bf16 %1, h, %1;\n}"
        : "+f"(lo), "+f"(hi)
        : "r"(x));
}
// eight floats in one store (32-byte aligned)
__device__ __forceinline__ void store8(float *dst, const float (&v)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// One item: rows [row0, row0 + rows) of group [seq0, ...), one KV head, one
// split of the prefix.
struct PrefixItem {
  int group, seq0, rows, row0, kvh, split, tok0, tok1;
};

// Group g's first sequence, sequences and prefix length, clamped to what the
// buffers hold; false if its starts were out of order or range.
__device__ __forceinline__ bool prefix_group(const PrefixParams &p, int g, int &seq0, int &n,
                                             int &len) {
  seq0 = __ldg(p.prefix_start + g);
  int end = __ldg(p.prefix_start + g + 1);
  len = __ldg(p.prefix_lens + g);
  const bool ok = seq0 >= 0 && end >= seq0 && end <= p.num_seqs;
  if (!ok || len < 0 || len > p.max_prefix_len) {
    report(p.status, kStatusBadInput);
    seq0 = max(0, min(seq0, p.num_seqs));
    end = max(seq0, min(end, p.num_seqs));
    len = max(0, min(len, p.max_prefix_len));
  }
  n = end - seq0;
  return ok;
}

// Walks the item list in order (the same list in every role): find() must be
// called by a whole warp with non-decreasing indices.  The list ends before the
// first 32 groups with a start out of order or range, so groups never overlap
// and the items are never more than the sequences allow.
template <int ROWS>
struct ItemWalk {
  int base = 0, first_group = 0;      // items before, and first of, the 32 groups held
  int cnt, incl, seq0, n, len;        // this lane's group
  bool loaded = false;

  __device__ __forceinline__ bool find(const PrefixParams &p, int item, PrefixItem &it) {
    const int lane = threadIdx.x & 31;
    while (true) {
      if (!loaded) {
        cnt = seq0 = n = len = 0;
        const int g = first_group + lane;
        bool ok = true;
        if (g < p.num_prefixes) {
          ok = prefix_group(p, g, seq0, n, len);
          const int tiles = (n * p.group + ROWS - 1) / ROWS;
          const int splits = (len + p.split_tokens - 1) / p.split_tokens;
          cnt = tiles * splits * p.num_kv_heads;
        }
        if (!__all_sync(0xffffffffu, ok)) return false;
        incl = cnt;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const int t = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += t;
        }
        loaded = true;
      }
      const int total = __shfl_sync(0xffffffffu, incl, 31);
      if (item < base + total) {
        const unsigned hit = __ballot_sync(0xffffffffu, base + incl > item);
        const int l = __ffs(hit) - 1;
        int rem = item - base - __shfl_sync(0xffffffffu, incl - cnt, l);
        it.group = first_group + l;
        it.seq0 = __shfl_sync(0xffffffffu, seq0, l);
        const int rows = __shfl_sync(0xffffffffu, n, l) * p.group;
        const int plen = __shfl_sync(0xffffffffu, len, l);
        // row tiles fastest: the CTAs of one wave share their keys in L2
        const int tiles = (rows + ROWS - 1) / ROWS;
        const int tile = rem % tiles;
        rem /= tiles;
        it.kvh = rem % p.num_kv_heads;
        it.split = rem / p.num_kv_heads;
        it.row0 = tile * ROWS;
        it.rows = min(ROWS, rows - it.row0);
        it.tok0 = it.split * p.split_tokens;
        it.tok1 = min(it.tok0 + p.split_tokens, plen);
        return true;
      }
      if (first_group + 32 >= p.num_prefixes) return false;
      first_group += 32;
      base += total;
      loaded = false;
    }
  }
};

// Partitions of a sequence's own keys (its partials come before the prefix's).
__device__ __forceinline__ int own_parts(const PrefixParams &p, int seq) {
  const int L = max(0, min(__ldg(p.seq_lens + seq), p.max_seq_len));
  return (L + p.partition_size - 1) / p.partition_size;
}

}  // namespace

template <typename T, int D>
__global__ void __launch_bounds__(PrefixShape<D>::THREADS, 1)
    pa_prefix_kernel(const __grid_constant__ PrefixParams p, const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v) {
  using Z = PrefixShape<D>;
  constexpr int NT = Z::NT, KEYS = Z::KEYS, NS = Z::SLOTS;
  constexpr uint32_t kIdescS = instr_desc<T>(kTileRows, KEYS, false);
  constexpr uint32_t kIdescPV = instr_desc<T>(kTileRows, D, true);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // 1024-byte aligned as the swizzle needs it: dynamic shared memory starts
  // right after the 1 KB that the system reserves (checked)
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *qbuf = smem_raw;                       // NT x [panel][128 rows][128 B]
  uint8_t *ring = qbuf + NT * Z::QTILE;           // NS x [8-key group][panel][8 keys][128 B]
  uint64_t *bars = reinterpret_cast<uint64_t *>(ring + NS * Z::SLOT);
  volatile int *flags = reinterpret_cast<volatile int *>(bars + Z::BARS);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + Z::BARS) + 1;
  const uint32_t q_u32 = smem_u32(qbuf), ring_u32 = smem_u32(ring);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * NS, q_full = empty0 + 8 * NS,
                 s_full = q_full + 16, p_full = s_full + 16, o_done = p_full + 16,
                 p_half = o_done + 16,
                 pv_done = p_half + 16, drain = pv_done + 8, never = drain + 8;
  const uint64_t limit = p.wait_limit_ns;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full + 8 * i, 4);
      mbar_init(s_full + 8 * i, 1);
      mbar_init(p_full + 8 * i, 4);
      mbar_init(p_half + 8 * i, 4);
      mbar_init(o_done + 8 * i, 1);
    }
    mbar_init(pv_done, 1);
    mbar_init(drain, 1);
    mbar_init(never, 1);
    flags[0] = 0;
    fence_mbar_init();
  }
  // What the items' first loads need (the lists, tables and queries, as if one
  // line of them a thread), on its way to L2 while the kernel before this one
  // ends
  {
    const long long i = (long long)blockIdx.x * Z::THREADS + threadIdx.x;
    const auto fetch = [&](const void *base, long long bytes) {
      if (i * 128 < bytes) prefetch_l2(static_cast<const char *>(base) + i * 128);
    };
    fetch(p.prefix_start, 4ll * (p.num_prefixes + 1));
    fetch(p.prefix_lens, 4ll * p.num_prefixes);
    fetch(p.seq_lens, 4ll * p.num_seqs);
    fetch(p.prefix_tables, 4ll * p.num_prefixes * p.max_prefix_blocks);
    fetch(p.query, (long long)p.num_seqs * p.num_heads * D * 2);
  }
  // wait for the kernel before in the stream, also before taking tensor
  // memory that a CTA of it may still hold; every CTA does before it lets the
  // own tokens' Phase 1 start, which then waits for the hand-over alone (by the
  // last warp, ahead of the copies, which its fence would wait for)
  pdl_wait_primary();
  pdl_launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == Z::THREADS - 32 && p.sched) hand_over(p.sched, kReadyBit);
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) report(p.status, kStatusBadInput);
    return;
  }
  if (warp == Z::SOFTMAX_WARPS + 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tmem_o = tmem + 256;  // S (and P) buffers at columns 0 and 128
  ItemWalk<NT * kTileRows> walk;
  PrefixItem it;

  // NT 2: 3 warpgroups at 168 registers, 2 x 208 + 80 <= 3 x 168
  if (warp >= Z::SOFTMAX_WARPS) {
    if constexpr (NT == 2) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == Z::SOFTMAX_WARPS || warp == Z::SOFTMAX_WARPS + 2) {
      // ======================= producer warps =======================
      // One for K, one for V: a warp's copies of pages leave one after another,
      // some 50 ns each, and a stage has 32 of them with pages of 8 (D 64, two
      // sequences behind 60,000 tokens: 50.1 us a call with one warp, 40.7 with
      // two; 8 behind 100,000, D 128, pages of 16: 49.5, 48.2).
      const int kv = warp == Z::SOFTMAX_WARPS ? 0 : 1;
      const CUtensorMap *tmap = kv == 0 ? &tmap_k : &tmap_v;
      if (lane == 0) prefetch_tmap(tmap);
      bool ok = true;
      int op = kv;  // the next copy: K and V of each stage, in turn
      const int U = p.block_size;
      for (int item = blockIdx.x; ok && walk.find(p, item, it); item += gridDim.x) {
        const int32_t *bt = p.prefix_tables + (size_t)it.group * p.max_prefix_blocks;
        const int stages = (it.tok1 - it.tok0 + KEYS - 1) / KEYS;
        // lane's page of a stage; the next stage's entries load while this one waits
        auto entry = [&](int j) -> int {
          const int tok = it.tok0 + j * KEYS + lane * U;
          return j < stages && lane < KEYS / U && tok < it.tok1 ? __ldg(bt + (tok >> p.log2_block_size)) : -1;
        };
        int blk = entry(0);
        for (int j = 0; ok && j < stages; ++j) {
          const int next = entry(j + 1);
          const int tok = it.tok0 + j * KEYS + lane * U;
          int y = -1;
          if (lane < KEYS / U && tok < it.tok1) {
            if ((unsigned)blk >= (unsigned)p.num_blocks)
              report(p.status, kStatusBadInput);
            else
              y = (blk * p.num_kv_heads + it.kvh) * U;
          }
          blk = next;
          const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, y >= 0)) * U * D * 2u;
          const int sl = op % NS;
          if (op >= NS) {
            bool w = true;
            if (lane == 0) w = mbar_wait(empty0 + 8 * sl, ((op / NS) - 1) & 1, limit, flags);
            ok = __shfl_sync(0xffffffffu, w, 0);
            if (!ok) break;
          }
          if (lane == 0) mbar_arrive_expect_tx(full0 + 8 * sl, bytes);
          __syncwarp();
          if (y >= 0)
            tma_load_4d(ring_u32 + (uint32_t)sl * Z::SLOT + (uint32_t)(lane * U / 8) * Z::GROUP, tmap,
                        0, 0, 0, y >> 3, full0 + 8 * sl);
          op += 2;
        }
      }
      // the partitions of every row, for Phase 2: its own, then its prefix's
      for (int s = blockIdx.x * 32 + lane; kv == 0 && s < p.num_seqs; s += gridDim.x * 32) {
        int lo = 0, hi = p.num_prefixes + 1;  // the first start above s
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (__ldg(p.prefix_start + mid) > s)
            hi = mid;
          else
            lo = mid + 1;
        }
        int splits = 0;
        if (lo == 0 || lo > p.num_prefixes) {  // in no group
          report(p.status, kStatusBadInput);
        } else {
          int s0, n, len;
          prefix_group(p, lo - 1, s0, n, len);
          splits = (len + p.split_tokens - 1) / p.split_tokens;
        }
        p.row_limit[s] = (own_parts(p, s) + splits) * p.partition_size;
      }
      if (!ok && lane == 0) {
        report(p.status, kStatusTimeout);
        flags[0] = 1;
      }
      if (lane == 0) flags[2 + kv] = op;
      __syncwarp();
    } else if (warp == Z::SOFTMAX_WARPS + 1) {
      // ======================= MMA warp =======================
      // The whole warp runs the loop, so that descriptors and control stay in
      // uniform registers; one elected lane issues.
      const uint32_t leader = elect_one();
      bool ok = true;
      int sk = 0, par = 0;        // ring slot of the next stage's K, its phase
      int items[2] = {0, 0};      // items of each tile
      int done[2] = {0, 0};       // stages of each tile (NT 1: [0], over both buffers)
      // The tile and ring descriptors' constant parts; a k-step adds to the
      // address field (16-byte units) only.
      const uint64_t q_desc = smem_desc(q_u32, 16, 1024);
      const uint64_t k_desc = smem_desc(ring_u32, 16, Z::GROUP);
      const uint64_t v_desc = smem_desc(ring_u32, 1024, Z::GROUP);
      auto wait_slot = [&](int sl, int ph) -> bool {
        return mbar_wait(full0 + 8 * sl, (uint32_t)ph, limit, flags);
      };
      auto advance = [&](int &sl, int &ph) {
        if (++sl == NS) {
          sl = 0;
          ph ^= 1;
        }
      };
      // S = Q K^T: D / 16 k-steps of 32 bytes inside a panel
      auto issue_s = [&](int sl, int t, int buf) {
        const uint64_t db0 = k_desc + (uint32_t)sl * (uint32_t)(Z::SLOT >> 4);
        const uint64_t da0 = q_desc + (uint32_t)t * (uint32_t)(Z::QTILE >> 4);
  #pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc_mma_if(leader, tmem + 128u * (uint32_t)buf,
                    da0 + (uint32_t)(((ks >> 2) * Z::QPANEL + (ks & 3) * 32) >> 4),
                    db0 + (uint32_t)(((ks >> 2) * 1024 + (ks & 3) * 32) >> 4), kIdescS, ks > 0 ? 1u : 0u);
        tc_commit_if(leader, s_full + 8u * (uint32_t)buf);
      };
      // O += P V: k-steps of 16 keys; P two keys a column, V MN-major
      auto issue_pv = [&](int sl, int t, int buf, bool first, int k0, int k1) {
        const uint64_t db0 = v_desc + (uint32_t)sl * (uint32_t)(Z::SLOT >> 4);
  #pragma unroll
        for (int kk = k0; kk < k1; ++kk)
          tc_mma_ts_if(leader, tmem_o + (uint32_t)(t * D), tmem + 128u * (uint32_t)buf + 8u * (uint32_t)kk,
                       db0 + (uint32_t)((kk * 2 * Z::GROUP) >> 4), kIdescPV, first && kk == 0 ? 0u : 1u);
      };
      for (int item = blockIdx.x; ok && walk.find(p, item, it); item += gridDim.x) {
        const int stages = (it.tok1 - it.tok0 + KEYS - 1) / KEYS;
        const int nt = (it.rows + kTileRows - 1) / kTileRows;
  #pragma unroll
        for (int t = 0; t < NT; ++t)
          if (ok && t < nt) ok = mbar_wait(q_full + 8 * t, items[t] & 1, limit, flags);
        if (ok) ok = wait_slot(sk, par);
        if (ok) {
          tc_fence_after();
          if constexpr (NT == 2) {
            issue_s(sk, 0, 0);
            if (nt == 2) issue_s(sk, 1, 1);
          } else {
            issue_s(sk, 0, done[0] & 1);
          }
          tc_commit_if(leader, empty0 + 8 * sk);
        }
        for (int j = 0; ok && j < stages; ++j) {
          const bool more = j + 1 < stages;
          int sv = sk, pv = par;  // V's slot, then the next K's
          advance(sv, pv);
          int sn = sv, pn = pv;
          advance(sn, pn);
          sk = sn;
          par = pn;
          if constexpr (NT == 2) {
            // this V and the next K are in long before P, as a rule: awaited
            // first, they cost nothing between P and its MMAs
            ok = wait_slot(sv, pv) && (!more || wait_slot(sn, pn));
            if (!ok) break;
  #pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (t >= nt) break;
              ok = mbar_wait(p_half + 8 * t, done[t] & 1, limit, flags);
              if (!ok) break;
              tc_fence_after();
              issue_pv(sv, t, t, j == 0, 0, KEYS / 32);
              ok = mbar_wait(p_full + 8 * t, done[t] & 1, limit, flags);
              if (!ok) break;
              tc_fence_after();
              issue_pv(sv, t, t, false, KEYS / 32, KEYS / 16);
              if (t == nt - 1) tc_commit_if(leader, empty0 + 8 * sv);
              if (more) {
                issue_s(sn, t, t);
                if (t == nt - 1) tc_commit_if(leader, empty0 + 8 * sn);
              } else {
                tc_commit_if(leader, o_done + 8 * t);
              }
              ++done[t];
            }
          } else {
            const int b = done[0] & 1;
            if (more) {
              ok = wait_slot(sn, pn);
              if (!ok) break;
              tc_fence_after();
              issue_s(sn, 0, b ^ 1);
              tc_commit_if(leader, empty0 + 8 * sn);
            }
            ok = mbar_wait(p_full + 8 * b, (done[0] >> 1) & 1, limit, flags) && wait_slot(sv, pv);
            if (!ok) break;
            tc_fence_after();
            issue_pv(sv, 0, b, j == 0, 0, KEYS / 16);
            tc_commit_if(leader, empty0 + 8 * sv);
            tc_commit_if(leader, pv_done);
            if (!more) tc_commit_if(leader, o_done);
            ++done[0];
          }
        }
  #pragma unroll
        for (int t = 0; t < NT; ++t) items[t] += t < nt;
        ok = __all_sync(0xffffffffu, ok);
      }
      // nothing may still run when the memory is freed
      tc_commit_if(leader, drain);
      mbar_wait(drain, 0, kDrainLimitNs, nullptr);
      if (!ok && lane == 0) {
        report(p.status, kStatusTimeout);
        flags[0] = 1;
      }
      __syncwarp();
    }
  } else {
    // ======================= softmax warps: thread = row =======================
    if constexpr (NT == 2) asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int t = warp >> 2;               // the tile
    const int r = threadIdx.x & 127;       // row of the tile, and tensor-memory lane
    const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t my_o = tmem_o + (uint32_t)(t * D) + lane_off;
    uint8_t *qt = qbuf + t * Z::QTILE;
    // a negative scale's sign goes into the queries, and a zero scale is zero
    // queries, so that the largest product is always the largest logit and a
    // masked product of -inf always a weight of zero
    const float sc = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
    const uint32_t q_flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
    const uint32_t q_keep = p.scale_log2 == 0.f ? 0u : 0xffffffffu;
    bool ok = true;
    int done = 0, items = 0, ops = 0;
    if (p.debug_flags & kPrefixDebugStall) {
      // wait on a barrier that nothing releases: the bound must end it
      ok = mbar_wait(never, 0, limit, flags);
      ok = __all_sync(0xffffffffu, ok);
    }
    for (int item = blockIdx.x; ok && walk.find(p, item, it); item += gridDim.x) {
      const int stages = (it.tok1 - it.tok0 + KEYS - 1) / KEYS;
      const int rows = it.rows - t * kTileRows;  // of this tile
      if (rows <= 0) {
        ops += 2 * stages;
        continue;
      }
      const int gr = it.row0 + t * kTileRows + r;  // row of the group
      const bool live = r < rows;
      const bool warp_live = 32 * (warp & 3) < rows;
      const int sq = (int)(((uint64_t)(uint32_t)gr * p.group_magic) >> 36);  // gr / group
      const int seq = it.seq0 + (live ? sq : 0);
      const int head = it.kvh * p.group + (live ? gr - sq * p.group : 0);
      const size_t orow = (size_t)seq * p.num_heads + head;
      {  // the warp's 32 queries into the swizzled tile (zeros past the item's
         // rows), lanes along a row
        constexpr int CPR = D / 8;        // 16-byte pieces of a row
        constexpr int RPI = CPR < 32 ? 32 / CPR : 1;
        const int c = lane % CPR;
        const uint4 *src = static_cast<const uint4 *>(p.query) + c;
        // eight loads in flight a lane, in a short loop: code that runs once
        // an item costs its fetch
#pragma unroll 1
        for (int i0 = 0; i0 < 32; i0 += 8 * RPI) {
          uint4 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = 32 * (warp & 3) + i0 + i * RPI + lane / CPR;  // row of the tile
            const int g = it.row0 + t * kTileRows + rr;
            const int sq = (int)(((uint64_t)(uint32_t)g * p.group_magic) >> 36);  // g / group
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (rr < rows)
              v[i] = __ldg(src + ((size_t)(it.seq0 + sq) * p.num_heads + it.kvh * p.group +
                                  (g - sq * p.group)) * CPR);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = 32 * (warp & 3) + i0 + i * RPI + lane / CPR;
            v[i] = make_uint4((v[i].x ^ q_flip) & q_keep, (v[i].y ^ q_flip) & q_keep,
                              (v[i].z ^ q_flip) & q_keep, (v[i].w ^ q_flip) & q_keep);
            *reinterpret_cast<uint4 *>(qt + (c >> 3) * Z::QPANEL + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) =
                v[i];
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full + 8 * t);
      }
      float m_run = -CUDART_INF_F, l = 0.f;
      float raise_at = -CUDART_INF_F;  // a stage's maximum above it becomes the running one
      for (int j = 0; ok && j < stages; ++j) {
        const int buf = NT == 2 ? t : done & 1;
        const uint32_t par = NT == 2 ? (uint32_t)done & 1u : ((uint32_t)done >> 1) & 1u;
        const uint32_t sbuf = tmem + 128u * (uint32_t)buf + lane_off;
        ok = __all_sync(0xffffffffu, mbar_wait(s_full + 8 * buf, par, limit, flags));
        if (!ok) break;
        tc_fence_after();
        const int valid = min(KEYS, it.tok1 - it.tok0 - j * KEYS);
        if (valid < KEYS && t == 0) {
          // V rows past the range may hold anything (0 x NaN would reach O):
          // zeros.  Tile 0's P is awaited before either tile's PV.
          const int ov = ops + 2 * j + 1;
          ok = __all_sync(0xffffffffu, mbar_wait(full0 + 8 * (ov % NS), (ov / NS) & 1, limit, flags));
          if (!ok) break;
          uint8_t *vst = ring + (size_t)(ov % NS) * Z::SLOT;
          for (int i = r; i < (KEYS - valid) * (D / 8); i += 128) {
            const int row = valid + i / (D / 8), c = i % (D / 8);
            *reinterpret_cast<uint4 *>(vst + (row >> 3) * Z::GROUP + (c >> 3) * 1024 + (row & 7) * 128 +
                                       (((c & 7) ^ (row & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        if (warp_live) {
          // the scores, the second half in flight behind the first's maximum
          uint32_t s[KEYS / 32][32];
          auto x = [&](int k) -> float { return __uint_as_float(s[k >> 5][k & 31]); };
          float m8[8];
          auto row_max = [&](int c) {
            if (valid < KEYS) {
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (32 * c + k >= valid) s[c][k] = 0xff800000u;  // -inf
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int k = 32 * c + i;
              m8[i] = c == 0 ? fmaxf(fmax3(x(k), x(k + 8), x(k + 16)), x(k + 24))
                             : fmax3(fmax3(m8[i], x(k), x(k + 8)), x(k + 16), x(k + 24));
            }
          };
          tmem_ld32(sbuf, s[0]);
          tmem_ld32(sbuf + 32, s[1]);
          tmem_ld_wait(s[0]);
          tmem_ld_wait(s[1]);
          if constexpr (KEYS == 128) {
            tmem_ld32(sbuf + 64, s[2]);
            tmem_ld32(sbuf + 96, s[3]);
          }
          row_max(0);
          row_max(1);
          if constexpr (KEYS == 128) {
            tmem_ld_wait(s[2]);
            tmem_ld_wait(s[3]);
            row_max(2);
            row_max(3);
          }
          const float mt = sc * fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]),
                                      fmaxf(m8[6], m8[7]));
          const bool raise = mt > raise_at;
          const float alpha = raise ? exp2f(m_run - mt) : 1.f;
          if (raise) m_run = mt;
          if (j > 0 && __any_sync(0xffffffffu, raise)) {
            // rescale the rows' O, once the PV of the stage before is done (NT
            // 2: this S was issued behind it)
            if constexpr (NT == 1) {
              ok = __all_sync(0xffffffffu, mbar_wait(pv_done, (uint32_t)(done - 1) & 1u, limit, flags));
              if (!ok) break;
              tc_fence_after();
            }
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
              uint32_t o[32];
              tmem_ld32(my_o + 32 * c, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * alpha);
              tmem_st32(my_o + 32 * c, o);
            }
            tmem_st_wait();
          }
          const float mb = m_run == -CUDART_INF_F ? 0.f : kWeightShift<T> - m_run;
          const uint64_t sc2 = pair(sc, sc), mb2 = pair(mb, mb);
          float ls[4] = {0.f, 0.f, 0.f, 0.f};
          // P over the scores' own registers (word e holds keys 2e, 2e + 1), so
          // that no register waits for a store in flight
          auto weights = [&](int h, int e0, int e1) {
#pragma unroll
            for (int e = e0; e < e1; ++e) {
              const int k = 64 * h + 2 * e;
              const float2 y = unpair(fma2(pair(x(k), x(k + 1)), sc2, mb2));
              s[h][e] = MmaOp<T>::pack(ex2(y.x), ex2(y.y));
              add_halves<T>(s[h][e], ls[2 * (e & 1)], ls[2 * (e & 1) + 1]);
            }
          };
          weights(0, 0, 32);
          tmem_st32(sbuf, s[0]);
          if constexpr (KEYS == 128) {
            // the first 64 keys' PV may begin; by now their store has landed
            weights(1, 0, 8);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_half + 8 * buf);
            weights(1, 8, 32);
            tmem_st32(sbuf + 32, s[1]);
          }
          l = fmaf(l, alpha, (ls[0] + ls[2]) + (ls[1] + ls[3]));
          tmem_st_wait();
        } else if (NT == 2) {
          if (lane == 0) mbar_arrive(p_half + 8 * buf);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 8 * buf);
        raise_at = m_run + fmaxf(fminf(lg2(l) - kWeightShift<T> - kLazyShare, kLazyMargin), 0.f);
        ++done;
      }
      ops += 2 * stages;
      if (!ok) break;
      ok = __all_sync(0xffffffffu, mbar_wait(o_done + 8 * t, items & 1, limit, flags));
      if (!ok) break;
      ++items;
      tc_fence_after();
      if (warp_live) {
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const size_t slot = orow * p.max_parts + own_parts(p, seq) + it.split;
        float *dst = p.tmp_out + slot * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(my_o + 32 * c, o);
          tmem_ld_wait(o);
          if (!live) continue;
#pragma unroll
          for (int k = 0; k < 32; k += 8) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(o[k + e]) * inv;
            store8(dst + 32 * c + k, v);
          }
        }
        if (live) {
          // what the weights are relative to, in natural-log units
          p.max_logits[slot] = (m_run - kWeightShift<T>) * 0.69314718055994530942f;
          p.exp_sums[slot] = l;
        }
      }
      tc_fence_before();
    }
    if (!ok && lane == 0) {
      report(p.status, kStatusTimeout);
      flags[0] = 1;
    }
  }
  // every role is done with the tensor memory: free it
  tc_fence_before();
  __syncthreads();
  if (warp == Z::SOFTMAX_WARPS + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (flags[0] && warp == Z::SOFTMAX_WARPS && lane < NS) {
    // given up midway: every copy lands before the CTA retires (else the MMA
    // warp has awaited them all).  Lane: the last copy into its slot
    const int k_end = flags[2], v_end = flags[3], end = max(k_end, v_end);
    for (int i = end - 1; i >= 0 && i > end - 1 - 2 * NS; --i)
      if (i % NS == lane && i < ((i & 1) ? v_end : k_end)) {
        mbar_wait(full0 + 8 * lane, (i / NS) & 1, kDrainLimitNs, nullptr);
        break;
      }
  }
}

namespace {
template <typename T>
PrefixKernelInfo pick(int head_size) {
  switch (head_size) {
    case 64:
      return {reinterpret_cast<const void *>(&pa_prefix_kernel<T, 64>), PrefixShape<64>::THREADS,
              PrefixShape<64>::SMEM, PrefixShape<64>::NT * kTileRows, PrefixShape<64>::KEYS};
    case 128:
      return {reinterpret_cast<const void *>(&pa_prefix_kernel<T, 128>), PrefixShape<128>::THREADS,
              PrefixShape<128>::SMEM, PrefixShape<128>::NT * kTileRows, PrefixShape<128>::KEYS};
    case 256:
      return {reinterpret_cast<const void *>(&pa_prefix_kernel<T, 256>), PrefixShape<256>::THREADS,
              PrefixShape<256>::SMEM, PrefixShape<256>::NT * kTileRows, PrefixShape<256>::KEYS};
  }
  return {};
}
}  // namespace

PrefixKernelInfo prefix_kernel(int dtype_bf16, int head_size) {
  return dtype_bf16 ? pick<__nv_bfloat16>(head_size) : pick<__half>(head_size);
}

// Splits of the prefix, at most most_splits, from a model of the call's time in
// microseconds (coefficients measured on GB300; the sizes of the groups are not
// known on the host, so a row tile is counted as half empty a group, and own
// lengths as half their bound; times of one build):
//   - the prefix kernel: waves of items on 152 SMs, each an item's stages at
//     the tensor cores' pace or that of the keys' bytes, plus 10 us an item
//     (start, queries, epilogue);
//   - the own tokens run on the SMs left free meanwhile, 50 GB/s each (57
//     with items of 512 tokens; what a single SM's copies of pages reach);
//     what is left then takes as long on those, or 3 us and 5.7 TB/s on all
//     of them.  So it pays to leave SMs free (256 sequences behind 8192 tokens
//     with 264 of their own: 3 splits, 96 items, 61.6 us, against 4 splits,
//     128 items, 64.5 us and 2 splits, 64 items, 68.4 us; D 256, 64 behind two
//     of 12,000 with 455 of their own: 9 splits, 90 items, 40.9 us, against 8
//     splits, 43.7 us, 11 splits, 43.9 us and 12 splits, 51.0 us), unless
//     there is little else to do (8 behind 100,000: 37 splits, 148 items, 48.8
//     us, 38 splits, 152 items, 48.7 us, 34 splits, 49.9 us);
//   - Phase 2: every split is another partial of every row.
void prefix_plan(int num_seqs, int num_prefixes, int num_heads, int num_kv_heads, int head_size,
                 int max_seq_len, int max_prefix_len, int partition_size, int most_splits,
                 int *split_tokens, int *max_splits) {
  const PrefixKernelInfo k = prefix_kernel(1, head_size);
  const double rows = (double)num_seqs * (num_heads / num_kv_heads);
  const int groups = num_prefixes < num_seqs ? num_prefixes : (num_seqs > 0 ? num_seqs : 1);
  const long long packed = (long long)((rows + k.tile_rows - 1) / k.tile_rows);
  long long tiles = packed + (groups > 1 ? groups / 2 : 0);
  if (tiles < groups) tiles = groups;
  if (tiles < 1) tiles = 1;
  const long long heads = tiles * num_kv_heads;
  const int stages = (max_prefix_len + k.stage_keys - 1) / k.stage_keys;
  const double pace = head_size == 64 ? 0.9 : head_size == 128 ? 1.5 : 0.87;
  // of its bytes alone; several prefixes are taken as 0.8 of the bound on average
  const double stage_us = (groups > 1 ? 0.8 : 1.) * k.stage_keys * head_size * 4. / 6.3e6;
  const double own_mb = (double)num_seqs * max_seq_len * 0.5 * num_kv_heads * head_size * 4e-6;
  const double own_parts = 0.7 * ((max_seq_len + partition_size - 1) / partition_size);
  int best = 1;
  double best_cost = 0.;
  for (int n = 1; n <= most_splits && (n == 1 || n <= stages); ++n) {
    const int per = (stages + n - 1) / n;
    const long long items = heads * (per > 0 ? (stages + per - 1) / per : 1);
    const long long waves = (items + kPrefixSms - 1) / kPrefixSms;
    const long long active = items < kPrefixSms ? items : kPrefixSms;
    const double bytes_pace = (double)active * groups / tiles * stage_us;
    const double t = waves * (per * (bytes_pace > pace ? bytes_pace : pace) + 10.);
    const double beside = waves == 1 ? (kPrefixSms - active) * 0.05 : 0.;  // MB a us
    const double left_mb = own_mb - t * beside;
    double after = left_mb > 0. ? 3. + left_mb / 5.7 : 0.;
    if (left_mb > 0. && left_mb < after * beside) after = left_mb / beside;
    const double cost = t + after +
                        (double)num_seqs * num_heads * (n + own_parts) * head_size * 4. / 3e6;
    if (n == 1 || cost < best_cost) {
      best = n;
      best_cost = cost;
    }
  }
  const int per = (stages + best - 1) / best;
  *split_tokens = (per > 0 ? per : 1) * k.stage_keys;
  *max_splits = (max_prefix_len + *split_tokens - 1) / *split_tokens;
}

}  // namespace pa
