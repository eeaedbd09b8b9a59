// pa_latent_forward: decode attention (and chunks of query tokens) in the
// absorbed form of latent attention: a token's cache row is one latent vector
// and a rotated key part, [latent_dim | 64], shared by all heads, the keys of
// every head are the row and the values its latent part.
//
//   S[64 rows][64 keys] = Q[64][W] . K^T                 (W = latent_dim + 64)
//   O^T[128 of latent_dim][64 rows] += C^T[128][64 keys] . P^T
// on the 5th-generation tensor cores, fp32 accumulators in tensor memory: S in
// two buffers of 64 columns, O^T in latent_dim / 128 tiles of 64.  Rows are
// (token, head) pairs, which stand one behind the other in the query, so 64 of
// them are one box for TMA whatever the number of heads.  The cache's bytes
// cross into shared memory once: the tile that S read as keys is, read along
// the other axis, the values of O^T.
//
// Bound: a row of 576 elements is 1152 bytes and 2 (576 + 512) flops a head.
// To 64 heads HBM bounds it.  128 heads are two groups of rows, taken by two
// CTAs that walk the same keys at the same time; there the MMAs are next to the
// limit: S has M = 64, which takes the time of 128.  More rows a CTA do not fit:
// 64 rows of queries are 72 KB, a tile of 64 keys 72 KB, and two tiles have to be
// there for copies to run beside MMAs.
//
// Measured on GB300: one sequence of 100000 keys, 16 heads: 40 us (17 at the
// bytes' rate; 13 of them the start, the epilogue and the join); 64 sequences of
// 1024 to 8192 keys, 128 heads: 146 us, 2.5 TB/s and 580 TFLOP/s.  There a tile takes
// 3700 cycles, 2550 of them MMAs: with two tiles in the ring its copy (2300
// cycles; 1000 when an SM's own side of L2 has it), S, the softmax (900) and O^T
// stand behind one another.  Slower were: tiles in parts that are copied, used
// and given back by themselves (162), tiles sent to L2 ahead of their copies
// (146), waits that look all the time (162).
//
// A softmax warp has eight rows, four threads a row (16 keys each, as the MMA
// fragments have them), so a row's maximum and sum are its own.  The maximum in
// use is raised only when a score passes it by 2^8, or by so much that the key
// would outweigh half of all before it: the weight of the maximum itself is exact,
// any other's is rounded, which shows where few keys carry a row (raised beyond
// 2^8 only, single results of ten million left the parity bar by up to 1.4).
// Weights are rounded to the
// input type (the MMA takes nothing wider): off by half a step, 2^-8 of themselves
// at most in bf16; in f16 by 2^-11, or 2^-32 of the piece's largest where that is
// more, as f16's start 2^7 above the maximum in use, which the sum takes out (a
// weight below 2^-25 of it was lost, and the sum with it: 63 keys at 2^-26 with
// values of 57344 gave 0 instead of 0.043).  The sum takes them as rounded.  A
// warp that raises goes on with the new one and leaves word with its weights;
// the MMA warp then holds O^T's MMAs back until all warps, each of which has
// every row in its lanes of O^T, have brought O^T down to it.
//
// Warps: 0-7 softmax and output (two to a quarter of the lanes), 8 producer (the
// walk over the shares, TMA), 9 MMA issuer.  One CTA an SM; work is cut in shares
// (pa_share.cuh), a CTA's each; every wait is bounded.
// Loops that issue MMAs are rolled and stand once: an SM fetches code that it
// has not run at some 250 cycles an MMA (the first tile took 13,000 cycles with
// three unrolled copies).
#include <math.h>
#include <math_constants.h>

#include <type_traits>

#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_ops.h"
#include "pa_share.cuh"
#include "pa_tcgen05.cuh"

namespace pa {
namespace {

constexpr int kLatentRows = 64;   // query rows of a unit
constexpr int kLatentKeys = 64;   // keys of a step
constexpr int kLatentHead = 2;     // tiles' time that a piece's beginning and end take
constexpr int kLatentSoftmax = 8;  // warps
constexpr int kLatentThreads = 32 * (kLatentSoftmax + 2);
constexpr int kLatentMaxCtas = 152;
constexpr int kLatentShares = 192;  // that a workspace has places for: a CTA's each
constexpr float kLatentNone = -3.402823466e38f;  // the maximum of no keys
// The maximum in use is raised when a score is above it by more than this, in log2
// units, or by so much that the key would weigh more than 2^-kLatentHalf of all
// before it together.
constexpr float kLatentMargin = 8.f, kLatentHalf = 1.f;
// Weights are 2^(x - maximum in use + this): with the margin 2^15, below f16's largest
template <typename T>
constexpr float kLatentShift = std::is_same<T, __half>::value ? 7.f : 0.f;

constexpr int kLatentFirst = 1, kLatentLast = 2, kLatentEnd = 4;
constexpr int kLatentDebugStall = 1;  // PA_DEBUG_STALL_CONSUMERS

struct LatentParams {
  void *out;                 // [rows][H][latent_dim]
  const int32_t *block_tables, *seq_lens, *q_start;
  int *status;
  int num_seqs, num_rows, num_heads, num_blocks;
  int block_size, log2_block_size, unit_rows, max_blocks_per_seq, max_seq_len;
  int side;  // CTAs that take the row groups of a unit side by side (1 or 2)
  int debug_flags;
  float scale_log2;
  uint64_t wait_limit_ns;
};

struct alignas(16) LatentStage {
  int flags, valid, tok0;  // keys of the stage in range, its first key
  int lim_base;            // row r sees keys below lim_base + (flat0 + r) / H + 1
  int flat0, rows;         // the rows' place in the sequence's chunk, how many
  int row0;                // and in the output (in heads)
  int place;               // -1: the unit is whole
};

template <int LAT>
struct LatentShape {
  static constexpr int NP = LAT / 64 + 1;       // 128-byte panels of a row
  static constexpr int GROUP = NP * 1024;       // 8 rows
  static constexpr int SLOT = 8 * GROUP;        // 64 keys
  static constexpr int SLOTS = LAT == 512 ? 2 : 4;
  static constexpr int QBYTES = NP * 8192;      // [panel][64 rows][128 B]
  static constexpr int PBYTES = 8192;           // [64 rows][64 keys]
  static constexpr int NT = LAT / 128;          // O^T tiles
  static constexpr int TMEM = LAT == 512 ? 512 : 256;
  static constexpr int NBARS = 2 * SLOTS + 10;
};

template <int LAT>
struct LatentShared {
  using Z = LatentShape<LAT>;
  uint8_t q[Z::QBYTES];
  uint8_t ring[Z::SLOTS][Z::SLOT];
  uint8_t p[Z::PBYTES];
  float alpha[kLatentRows];   // factors of rows whose maximum was raised
  float sum[2][kLatentRows];  // (pieces in turn) the rows' sums
  LatentStage info[Z::SLOTS];
  alignas(8) uint8_t raised[2][kLatentSoftmax];  // (tiles in turn) whether a warp raised any
  uint64_t bars[Z::NBARS];
  int flags[2];
  uint32_t tmem;
  int pad;
  ShareScan<128, 64> scan;
};

struct LatentBatch {
  const LatentParams &p;
  int num_seqs;
  bool tell;  // report what is bad
  __device__ __forceinline__ int4 read(int s) const {
    int4 r = make_int4(__ldg(p.seq_lens + s), s, 1, 0);
    bool bad = r.x < 0 || r.x > p.max_seq_len;
    if (p.q_start) {
      r.y = __ldg(p.q_start + s);
      const int e = __ldg(p.q_start + s + 1);
      bad = bad || r.y < 0 || e < r.y || e > p.num_rows || e - r.y > r.x;
      if (tell && s == 0 && r.y > 0) report(p.status, kStatusBadInput);  // rows that are nobody's
      r.z = e - r.y;
    }
    if (bad) {
      if (tell) report(p.status, kStatusBadInput);
      r.x = r.z = 0;
    }
    return r;
  }
  __device__ __forceinline__ ShareSeq seq(const int4 &r) const {
    ShareSeq q{r.x, r.y, r.z, 0, 0, kLatentHead};
    q.steps = (r.x + kLatentKeys - 1) / kLatentKeys;
    if (q.steps > 0) {
      const int groups = (int)(((long long)r.z * p.num_heads + kLatentRows - 1) / kLatentRows);
      q.units = (groups + p.side - 1) / p.side;
    }
    return q;
  }
};

// 16 lanes by 64 columns of tensor memory, as MMA fragments: thread t has rows
// t / 4 and t / 4 + 8, columns 8 j + 2 (t % 4) + {0, 1}: words 4 j + {0, 1} and + {2, 3}
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
               : "r"(taddr));
}
// 8 columns of this warp's 32 lanes (lane = thread), the load with its wait
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
               "tcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ bool any_raised(const uint8_t *r) {
  static_assert(kLatentSoftmax == 8, "eight flags in a word");
  return *reinterpret_cast<const volatile unsigned long long *>(r) != 0;
}

}  // namespace

template <typename T, int LAT>
__global__ void __launch_bounds__(kLatentThreads, 1)
    pa_latent_kernel(const __grid_constant__ LatentParams p, const __grid_constant__ ShareSpace space,
                     const __grid_constant__ CUtensorMap tmap_c, const __grid_constant__ CUtensorMap tmap_q) {
  using Z = LatentShape<LAT>;
  using Shared = LatentShared<LAT>;
  constexpr int NP = Z::NP, NS = Z::SLOTS;
  constexpr uint32_t kIdescS = instr_desc<T>(kLatentRows, kLatentKeys, false, false);
  constexpr uint32_t kIdescO = instr_desc<T>(128, kLatentRows, false, true);
  constexpr float kShift = kLatentShift<T>;

  // The 128-byte swizzle needs every tile 1024-byte aligned; the dynamic shared
  // memory starts so (there is no static part), which is checked.
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if ((smem_u32(smem_raw) & 1023u) != 0) {
    if (threadIdx.x == 0) report(p.status, kStatusBadInput);
    return;
  }
  Shared &sh = *reinterpret_cast<Shared *>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int *flags = sh.flags;
  const uint32_t full = smem_u32(sh.bars), empty = full + 8 * NS, q_full = empty + 8 * NS, q_empty = q_full + 8,
                 s_full = q_empty + 8, p_full = s_full + 16, pv_done = p_full + 8, o_done = pv_done + 8,
                 rescaled = o_done + 8, drain = rescaled + 8, never = drain + 8;
  const uint32_t q_u32 = smem_u32(sh.q), ring_u32 = smem_u32(sh.ring), p_u32 = smem_u32(sh.p);
  const uint64_t limit = p.wait_limit_ns;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, kLatentSoftmax + 1);  // the O^T MMAs' commit and each softmax warp's header read
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(s_full, 1);
    mbar_init(s_full + 8, 1);
    mbar_init(p_full, kLatentSoftmax);
    mbar_init(pv_done, 1);
    mbar_init(o_done, 1);
    mbar_init(rescaled, kLatentSoftmax);
    mbar_init(drain, 1);
    mbar_init(never, 1);
    sh.flags[0] = 0;
    fence_mbar_init();
  }
  if (warp == kLatentSoftmax && lane == 0) {
    prefetch_tmap(&tmap_c);
    prefetch_tmap(&tmap_q);
  }
  // Launched with programmatic dependent launch: wait for the previous kernel
  // in the stream before the tensor memory is taken and before any global
  // access.
  pdl_wait_primary();
  if (warp == kLatentSoftmax + 1) {
    tmem_alloc(smem_u32(&sh.tmem), Z::TMEM);
    tmem_relinquish();
  }
  LatentBatch batch{p, p.num_seqs, blockIdx.x == 0};
  share_scan(batch, sh.scan);
  batch.tell = false;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_o = sh.tmem, tmem_s = sh.tmem + 64 * Z::NT;

  if (warp == kLatentSoftmax) {
    // ======================= producer warp =======================
    const int U = p.unit_rows;
    SharePlan plan;
    // (large shares alone: a piece's rows are up to 128 KB, and more pieces took more
    // than they evened out: 168 -> 160 us for 64 sequences with 128 heads)
    plan.make(sh.scan.cum[128], (int)gridDim.x / p.side, true);
    // an item: a share, for one of the row groups that stand side by side
    const int item = blockIdx.x, share = item / p.side;
    ShareWalk walk{};
    walk.begin(batch, sh.scan, plan.begin(share), share < plan.big ? plan.begin(share + 1) : 0);
    // the tile whose table entries are on their way
    LatentStage f{};
    int f_left = 0, f_end = 0, ent = -1;
    const int32_t *table = p.block_tables;
    auto fetch = [&]() {
      if (f_left == 0) {
        while (true) {
          if (walk.left <= 0) {
            f.flags = kLatentEnd;
            return;
          }
          // the piece's row group of this CTA; a unit's last may have none beside
          const int group = walk.unit * p.side + item % p.side;
          const int n = walk.steps(), step = walk.first();
          const int flat0 = group * kLatentRows, all = walk.q.n * p.num_heads;
          if (flat0 < all) {
            f.flat0 = flat0;
            f.rows = min(kLatentRows, all - flat0);
            f.row0 = walk.q.row0 * p.num_heads + flat0;
            f.lim_base = walk.q.len - walk.q.n;
            f_end = f.lim_base + (flat0 + f.rows - 1) / p.num_heads + 1;
            const bool begins = step == 0, ends = step + n == walk.q.steps;
            f.place = begins && ends ? -1 : 2 * item + (begins ? 1 : 0);
            if (begins && !ends && lane == 0) {
              ShareJoin j{};
              j.share = item;
              j.parts = plan.of(walk.last()) - share + 1;
              j.by = p.side;
              j.rows = f.rows;
              j.group = j.stride = 1;
              j.out_row = f.row0;
              share_join(space, j);
            }
            table = p.block_tables + (size_t)walk.s * p.max_blocks_per_seq;
            f.tok0 = step * kLatentKeys;
            f.flags = kLatentFirst;
            f_left = n;
          }
          walk.next(batch, sh.scan);
          if (f_left > 0) break;
        }
      } else {
        f.tok0 += kLatentKeys;
        f.flags = 0;
      }
      if (--f_left == 0) f.flags |= kLatentLast;
      f.valid = max(min(f_end - f.tok0, kLatentKeys), 0);
      ent = lane * U < f.valid ? __ldg(table + ((f.tok0 + lane * U) >> p.log2_block_size)) : -1;
    };
    fetch();
    bool ok = true;
    int i = 0, nq = 0;
    while (true) {
      const int sl = i % NS;
      if (i >= NS) {
        bool w = true;
        if (lane == 0) w = mbar_wait(empty + 8 * sl, ((i / NS) - 1) & 1, limit, flags);
        ok = __shfl_sync(0xffffffffu, w, 0);
        if (!ok) break;
      }
      if (f.flags & kLatentEnd) {
        if (lane == 0) {
          sh.info[sl] = f;
          mbar_arrive(full + 8 * sl);
        }
        ++i;
        break;
      }
      // rows of pages: unit_rows of them a copy, each panel of 8 rows one swizzle atom
      const int tok = f.tok0 + lane * U;
      int y = -1;
      if (lane * U < f.valid) {
        if ((unsigned)ent >= (unsigned)p.num_blocks)
          report(p.status, kStatusBadInput);
        else
          y = ent * p.block_size + (tok & (p.block_size - 1));
      }
      const unsigned on = __ballot_sync(0xffffffffu, y >= 0);
      if (lane == 0) {
        sh.info[sl] = f;
        mbar_arrive_expect_tx(full + 8 * sl, (uint32_t)__popc(on) * U * 128u * NP);
      }
      __syncwarp();
      if (y >= 0)
        tma_load_4d(ring_u32 + (uint32_t)sl * Z::SLOT + (uint32_t)(lane * U / 8) * Z::GROUP, &tmap_c, 0, 0, 0,
                    y >> 3, full + 8 * sl);
      const bool first = f.flags & kLatentFirst;
      const int row0 = f.row0;
      ++i;
      fetch();
      if (first) {  // the piece's queries, once the last one's have been read
        if (nq >= 1) {
          bool w = true;
          if (lane == 0) w = mbar_wait(q_empty, (nq - 1) & 1, limit, flags);
          ok = __shfl_sync(0xffffffffu, w, 0);
          if (!ok) break;
        }
        if (lane == 0) mbar_arrive_expect_tx(q_full, (uint32_t)Z::QBYTES);
        __syncwarp();
        if (lane < NP) tma_load_2d(q_u32 + lane * 8192u, &tmap_q, lane * 64, row0, q_full);
        ++nq;
      }
    }
    if (!ok && lane == 0) {
      report(p.status, kStatusTimeout);
      flags[0] = 1;
    }
    if (lane == 0) {  // every copy of this CTA lands before it retires
      for (int j = i > NS ? i - NS : 0; j < i; ++j)
        mbar_wait(full + 8 * (j % NS), (j / NS) & 1, kDrainLimitNs, nullptr);
      if (nq > 0) mbar_wait(q_full, (nq - 1) & 1, kDrainLimitNs, nullptr);
    }
    __syncwarp();
  } else if (warp == kLatentSoftmax + 1) {
    // ======================= MMA warp =======================
    // The whole warp runs the loop, so that descriptors and control stay in
    // uniform registers; one elected lane issues.
    const uint32_t leader = elect_one();
    bool ok = true;
    int nq = 0, nr = 0;  // pieces whose queries S has taken, rescales
    const uint64_t q_desc = smem_desc(q_u32, 16, 1024), k_desc = smem_desc(ring_u32, 16, Z::GROUP);
    const uint64_t v_desc = smem_desc(ring_u32, 1024, Z::GROUP), p_desc = smem_desc(p_u32, 16, 1024);
    auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
      const bool w = mbar_wait(bar, parity, limit, flags);
      ok = __all_sync(0xffffffffu, w);
      return ok;
    };
    int issued = 0, fl = 0, fl_next = 0;  // tiles whose S is issued; the flags of tile i, of the last issued
    for (int i = 0; ok; ++i) {
      // S of this tile if it is not yet issued; then of the next, before O^T of
      // this one, if its keys (and queries) are here
      bool end = false;
#pragma unroll 1
      for (int a = issued - i; a < 2; ++a) {
        const int sl = issued % NS;
        const uint32_t bar = full + 8 * sl, par = (issued / NS) & 1;
        if (a == 0 ? !wait(bar, par) : !__all_sync(0xffffffffu, mbar_test(bar, par))) break;
        const int f = sh.info[sl].flags;
        if (f & kLatentEnd) {
          end = a == 0;
          break;
        }
        if (f & kLatentFirst) {
          if (a == 0 ? !wait(q_full, nq & 1) : !__all_sync(0xffffffffu, mbar_test(q_full, nq & 1))) break;
          ++nq;
        }
        tc_fence_after();
        const uint32_t d = tmem_s + 64u * (uint32_t)(issued & 1);
        const uint64_t db = k_desc + (uint32_t)sl * (uint32_t)(Z::SLOT >> 4);
#pragma unroll 1
        for (int pn = 0; pn < NP; ++pn)
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            tc_mma_if(leader, d, q_desc + (uint32_t)(pn * 512 + ks * 2), db + (uint32_t)(pn * 64 + ks * 2), kIdescS,
                      pn + ks > 0 ? 1u : 0u);
        tc_commit_if(leader, s_full + 8u * (uint32_t)(issued & 1));
        if (f & kLatentLast) tc_commit_if(leader, q_empty);
        fl = a == 0 ? f : fl;
        fl_next = f;
        ++issued;
      }
      if (!ok || end) break;
      if (!wait(p_full, i & 1)) break;
      if (any_raised(sh.raised[i & 1]) && !wait(rescaled, nr++ & 1)) break;
      tc_fence_after();
      const uint64_t da = v_desc + (uint32_t)(i % NS) * (uint32_t)(Z::SLOT >> 4);
#pragma unroll 1
      for (int kk = 0; kk < kLatentKeys / 16; ++kk)
#pragma unroll
        for (int j = 0; j < Z::NT; ++j)
          tc_mma_if(leader, tmem_o + 64u * (uint32_t)j, da + (uint32_t)(kk * (2 * Z::GROUP >> 4) + j * 128),
                    p_desc + (uint32_t)(kk * 2), kIdescO, (fl & kLatentFirst) && kk == 0 ? 0u : 1u);
      tc_commit_if(leader, pv_done);
      tc_commit_if(leader, empty + 8 * (i % NS));
      if (fl & kLatentLast) tc_commit_if(leader, o_done);
      fl = fl_next;
    }
    // nothing may still run when the memory is freed
    tc_commit_if(leader, drain);
    mbar_wait(drain, 0, kDrainLimitNs, nullptr);
    if (!ok && lane == 0) {
      report(p.status, kStatusTimeout);
      flags[0] = 1;
    }
    __syncwarp();
  } else {
    // ======================= softmax warps =======================
    // thread: row 16 quarter + 8 half + lane / 4, keys 8 j + 2 (lane % 4) + {0, 1}
    const int quarter = warp & 3, half = warp >> 2;
    const int t = threadIdx.x, q4 = lane & 3, row = 16 * quarter + 8 * half + (lane >> 2);
    const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
    float m = kLatentNone, l = 0.f;  // m: 2^kShift below the maximum in use
    float raise_at = kLatentNone;    // a score above it becomes the maximum in use
    int lim = 0, pieces = 0;
    bool ok = true;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      const bool w = mbar_wait(bar, parity, limit, flags);
      ok = __all_sync(0xffffffffu, w);
      return ok;
    };
    if (p.debug_flags & kLatentDebugStall) wait(never, 0);  // ends by its bound
    for (int i = 0; ok; ++i) {
      const int sl = i % NS;
      if (!wait(full + 8 * sl, (i / NS) & 1)) break;
      const LatentStage h = sh.info[sl];
      __syncwarp();
      if (h.flags & kLatentEnd) break;
      if (lane == 0) mbar_arrive(empty + 8 * sl);  // done with the header
      if (h.flags & kLatentFirst) {
        lim = row < h.rows ? h.lim_base + (h.flat0 + row) / p.num_heads + 1 : 0;
        m = raise_at = kLatentNone;
        l = 0.f;
      }
      if (!wait(s_full + 8 * (i & 1), (i >> 1) & 1)) break;
      tc_fence_after();
      uint32_t sr[32];
      tmem_ld_frag(tmem_s + 64u * (uint32_t)(i & 1) + lane_off, sr);
      tmem_ld_wait(sr);
      float x[16], top = kLatentNone, al = 1.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int j = 4 * (k >> 1) + (k & 1);
        x[k] = __uint_as_float(half ? sr[j + 2] : sr[j]) * p.scale_log2;
      }
      if (h.valid < kLatentKeys || h.tok0 + kLatentKeys > lim) {
        const int end = min(h.valid, lim - h.tok0) - 2 * q4;
#pragma unroll
        for (int k = 0; k < 16; ++k)
          if (8 * (k >> 1) + (k & 1) >= end) x[k] = -CUDART_INF_F;
      }
#pragma unroll
      for (int k = 0; k < 16; k += 2) top = fmax3(top, x[k], x[k + 1]);
      const bool raise = __any_sync(0xffffffffu, top > raise_at);
      if (raise) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        top = fmaxf(__fsub_ru(top, kShift), m);
        al = ex2(m - top);
        m = top;
        l *= al;
      }
      // weights, rounded to the input type; the sums take them as rounded
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 16; k += 2) {
        w[k / 2] = MmaOp<T>::pack(ex2(x[k] - m), ex2(x[k + 1] - m));
        const float2 r = MmaOp<T>::unpack(w[k / 2]);
        l += r.x + r.y;
      }
      // into P's tile, which the MMAs of the tile before have read
      if (i >= 1 && !wait(pv_done, (i - 1) & 1)) break;
      if (raise && q4 == 0) sh.alpha[row] = al;  // (those of the tile before have been used)
#pragma unroll
      for (int k = 0; k < 8; ++k)  // 16-byte piece k: eight keys
        *reinterpret_cast<uint32_t *>(sh.p + row * 128 + ((k ^ (row & 7)) << 4) + 4 * q4) = w[k];
      // rows of keys that are not the item's may hold anything (0 x NaN would reach O^T)
      if (h.valid < kLatentKeys) {
        uint8_t *v = sh.ring[sl];
        constexpr int kPieces = LAT / 8;  // 16-byte pieces of a key's latent part
        for (int e = t; e < (kLatentKeys - h.valid) * kPieces; e += 32 * kLatentSoftmax) {
          const int r = h.valid + e / kPieces, c = e % kPieces;
          *reinterpret_cast<uint4 *>(v + (r >> 3) * Z::GROUP + (c >> 3) * 1024 + (r & 7) * 128 +
                                     (((c & 7) ^ (r & 7)) << 4)) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
      if (h.flags & kLatentLast) {
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (q4 == 0) {
          sh.sum[pieces & 1][row] = l;
          if (h.place >= 0 && row < h.rows)
            space.ml[(size_t)h.place * kLatentRows + row] = make_float2(m, l);
        }
      }
      if (lane == 0) sh.raised[i & 1][warp] = raise && !(h.flags & kLatentFirst);
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_full);
      // (of the row's whole sum; rounded down, and the next reference up: no weight
      // above 2^15 however far the scores are)
      float all = l + __shfl_xor_sync(0xffffffffu, l, 1);
      all += __shfl_xor_sync(0xffffffffu, all, 2);
      raise_at = __fadd_rd(m, kShift + fmaxf(fminf(lg2(all) - kShift - kLatentHalf, kLatentMargin), 0.f));
      // what the other warps left with their weights
      if (!wait(p_full, i & 1)) break;
      if (any_raised(sh.raised[i & 1])) {
        // O^T (its MMAs of the tile before are done, those of this one wait): this
        // warp's lanes, half of the rows, eight rows of a warp that raised at a time
        tc_fence_after();
#pragma unroll 1
        for (int g = 4 * half; g < 4 * half + 4; ++g) {
          if (!*const_cast<volatile uint8_t *>(&sh.raised[i & 1][(g >> 1) + 4 * (g & 1)])) continue;
          const float4 a0 = *reinterpret_cast<const float4 *>(sh.alpha + 8 * g);
          const float4 a1 = *reinterpret_cast<const float4 *>(sh.alpha + 8 * g + 4);
          const float al[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll 1
          for (int j = 0; j < Z::NT; ++j) {
            const uint32_t at = tmem_o + 64u * (uint32_t)j + 8u * (uint32_t)g + lane_off;
            uint32_t o[8];
            tmem_ld8(at, o);
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * al[k]);
            tmem_st8(at, o);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(rescaled);
      }
      if (h.flags & kLatentLast) {
        if (!wait(o_done, pieces & 1)) break;
        tc_fence_after();
        const int r0 = 32 * half;
        if (r0 < h.rows) {
          const float sum = sh.sum[pieces & 1][r0 + lane];  // (lane: a row)
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll 1
          for (int j = 0; j < Z::NT; ++j) {
            const int d = 128 * j + 32 * quarter + lane;
            uint32_t o[32];
            tmem_ld32(tmem_o + 64u * (uint32_t)j + 32u * (uint32_t)half + lane_off, o);
            tmem_ld_wait(o);
            if (h.place >= 0) {
              float *dst = space.o + ((size_t)h.place * kLatentRows + r0) * LAT + d;
#pragma unroll
              for (int k = 0; k < 32; ++k)
                if (r0 + k < h.rows) dst[(size_t)k * LAT] = __uint_as_float(o[k]);
            } else {
              T *dst = static_cast<T *>(p.out) + ((size_t)h.row0 + r0) * LAT + d;
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                const float f = __shfl_sync(0xffffffffu, inv, k);
                if (r0 + k < h.rows) dst[(size_t)k * LAT] = from_float<T>(__uint_as_float(o[k]) * f);
              }
            }
          }
        }
        ++pieces;
        tc_fence_before();  // (before this warp's next weights let O^T be written)
      }
    }
    if (!ok && lane == 0) {
      report(p.status, kStatusTimeout);
      flags[0] = 1;
    }
    // outputs of empty sequences
    if (!p.q_start)
      for (int s = blockIdx.x; s < p.num_seqs; s += gridDim.x)
        if (share_seq(batch, sh.scan, s).len == 0) {
          uint4 *z = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + (size_t)s * p.num_heads * LAT);
          for (int e = t; e < p.num_heads * LAT / 8; e += 32 * kLatentSoftmax) z[e] = make_uint4(0u, 0u, 0u, 0u);
        }
  }

  // every role is done with the tensor memory: free it
  tc_fence_before();
  __syncthreads();
  if (warp == kLatentSoftmax + 1) {
    tc_fence_after();
    tmem_dealloc(sh.tmem, Z::TMEM);
  }
  pdl_launch_dependents();
}

namespace {

template <typename T>
const void *latent_pick(int latent_dim, int *smem) {
  if (latent_dim == 512) {
    *smem = (int)sizeof(LatentShared<512>);
    return reinterpret_cast<const void *>(&pa_latent_kernel<T, 512>);
  }
  *smem = (int)sizeof(LatentShared<256>);
  return reinterpret_cast<const void *>(&pa_latent_kernel<T, 256>);
}
static_assert(sizeof(LatentShared<512>) <= 232448 && sizeof(LatentShared<256>) <= 232448, "shared memory of an SM");

}  // namespace
}  // namespace pa

extern "C" {

size_t pa_latent_workspace_bytes(int latent_dim) {
  if (latent_dim != 256 && latent_dim != 512) return 0;
  return pa::share_bytes(pa::kLatentShares, pa::kLatentRows, latent_dim, nullptr, nullptr);
}

pa_status_t pa_latent_forward(void *out, const void *query, const void *cache, const int32_t *block_tables,
                              const int32_t *seq_lens, const int32_t *q_start, int num_seqs, int num_rows,
                              int num_heads, int latent_dim, int rope_dim, int num_blocks, int block_size,
                              int max_blocks_per_seq, int max_seq_len, float scale, int dtype, void *workspace,
                              size_t workspace_bytes, void *stream, const pa_options_t *opts) {
  using namespace pa;
  pa_options_t opt{};
  if (opts) opt = *opts;
  pa_status_t st = latent_check_cache(dtype, num_heads, latent_dim, rope_dim, num_blocks, block_size,
                                      max_blocks_per_seq, max_seq_len);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || num_rows < 0 || (!q_start && num_rows != num_seqs)) return PA_ERR_INVALID_ARG;
  if (!isfinite(scale)) return PA_ERR_INVALID_ARG;
  if (max_seq_len > kMaxTokens || (long long)num_rows * num_heads >= (1ll << 31)) return PA_ERR_UNSUPPORTED;
  if (num_rows == 0 || num_seqs == 0) return PA_OK;  // (empty tensors have no address)
  if (!out || !query || !cache || !block_tables || !seq_lens || !workspace) return PA_ERR_INVALID_ARG;
  const void *wide[] = {out, query, cache};
  for (const void *q : wide)
    if (!host_aligned(q, 16)) return PA_ERR_INVALID_ARG;
  const void *ints[] = {block_tables, seq_lens, q_start};
  for (const void *q : ints)
    if (!host_aligned(q, 4)) return PA_ERR_INVALID_ARG;
  if (!host_aligned(workspace, 256)) return PA_ERR_INVALID_ARG;
  if (workspace_bytes < pa_latent_workspace_bytes(latent_dim)) return PA_ERR_WORKSPACE_TOO_SMALL;

  LatentParams p{};
  p.out = out;
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
  p.unit_rows = block_size < kLatentKeys ? block_size : kLatentKeys;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_seq_len = max_seq_len;
  p.side = num_heads > kLatentRows ? 2 : 1;
  p.debug_flags = opt.debug_flags;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wait_limit_ns = opt.wait_limit_ns ? opt.wait_limit_ns : kDefaultWaitLimitNs;

  CUtensorMap tmap_c, tmap_q;
  st = host_cache_map(&tmap_c, cache, dtype, latent_dim + rope_dim, (long long)num_blocks * block_size, p.unit_rows);
  if (st != PA_OK) return st;
  st = host_rows_map(&tmap_q, query, dtype, latent_dim + rope_dim, (long long)num_rows * num_heads, kLatentRows);
  if (st != PA_OK) return st;
  int sms = 0, smem = 0;
  st = host_sm_count(&sms);
  if (st != PA_OK) return st;
  const void *fn = dtype == PA_DTYPE_BF16 ? latent_pick<__nv_bfloat16>(latent_dim, &smem)
                                          : latent_pick<__half>(latent_dim, &smem);
  st = host_ensure_smem(fn, smem);
  if (st != PA_OK) return st;
  int ctas = sms < kLatentMaxCtas ? sms : kLatentMaxCtas;
  ctas -= ctas % p.side;
  if (ctas < p.side) ctas = p.side;
  ShareSpace space;
  share_bytes(kLatentShares, kLatentRows, latent_dim, workspace, &space);
  void *args[4] = {&p, &space, &tmap_c, &tmap_q};
  st = host_launch(fn, (unsigned)ctas, 1, kLatentThreads, smem, stream, args, "launch latent attention kernel");
  if (st != PA_OK) return st;
  JoinParams j{};
  j.space = space;
  j.out = out;
  j.max_rows = kLatentRows;
  j.item_rows = q_start || num_heads > kLatentRows ? kLatentRows : num_heads;
  j.width = latent_dim;
  return share_launch_join(j, dtype == PA_DTYPE_BF16, sms, stream);
}

}  // extern "C"
