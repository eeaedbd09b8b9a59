// pa_q4_forward: decode attention (and chunks of query tokens) over a cache
// whose keys and values are held in 4 bits (pa_q4.h).
//
// With codes c, lowest values lo and steps st, group by group of 64 elements,
//   q . K_t       = sum_g st_tg (q_g . c_tg) + lo_tg sum(q_g)
//   sum_t p_t V_t = sum_t (p_t st_t) c_t + sum_t p_t lo_t      (of each group)
// so the codes go into the matrix products as they are, and the steps and
// lowest values meet scores and weights instead of elements.  What a code costs
// on its way there is what bounds this kernel next to the bytes (logic and shifts
// run at half an instruction a cycle), so both products take codes in a form
// that masking alone makes: four bits at the bottom of an f16 are c 2^-24, the
// next four c 2^-20, as f16's lowest numbers are evenly spaced (and exact in
// the MMA): five operations for eight codes.  Keys' powers of two are
// made up for in the queries: a head is scaled by a power of two so that its
// largest element is below 2^15 (or 2^11, against the larger codes), which f16
// holds to the last bit of a bf16 or an f16 down to 2^-17 of it.  Values' come
// off in the end.
//
// Weights: the product takes w = p st in f16, so it must neither overflow nor
// vanish with st: with S the larger of a token's |st|, the running maximum is
// that of x + log2 S (x: score in log2 units), p' = 2^(x + log2 S - m), and a
// group's w = p' st / S.  The normaliser sum(p' / S) is summed in fp32.  The
// reference m is 2^7 below the maximum in use, which the sums take out: w is off
// by up to 2^-11 of itself, or 2^-32 of the piece's largest where that is more,
// f16 having no more numbers there.  (With weights from 1 down, those of a group
// whose steps are 2^-23.4 of its head's largest were off by a third.)  That must
// not meet codes of 0 to 15 (a value is what is left of lo and them, so its error
// would be three times that of weights against values), but codes about their
// middle: with w' the rounded weights,
//   sum_t p_t V_t = sum_t w'_t c_t - 7.5 sum_t w'_t + sum_t (p' / S) (lo + 7.5 st)
// the last in fp32, sum(w') by one more MMA a group, against - 7.5 in row 0.
// (Without it f16 outputs were off by 0.00056 of themselves, 0.00021 being their
// own rounding's part; it costs 2 %.)
//
// Layout: S^T[16 tokens][8 heads] = K Q^T and O^T[D][8 heads] += V^T P^T
// (mma.sync m16n8k16, f16), a warp 16 tokens at a time.
// Which element of a head is which k of the first product is free, and so is
// which element of V is which row of O^T: ldmatrix hands a lane words of eight
// codes of a key, and (transposed) units of four codes of two tokens' values,
// and both are used as they come.  (Measured on GB300, cycles of a quarter of an
// SM: 8.1 an f16 MMA, 2 a logic operation or byte move, 4 a movmatrix.  8-bit
// MMAs of this kind are made of f16 ones and conversions there: slower.)
//
// A warp takes shares of the work (pa_share.cuh) by itself, its tokens copied by
// cp.async into its own ring of shared memory: no warp waits for another, and
// what a warp has of a unit leaves from its registers.  (Four warps that shared
// a unit's tokens and merged at its end spent 4 us on each piece of a unit.)
//
// Measured on GB300, bf16: 256 sequences of 512 to 3584 tokens, 32/4 heads, D 128:
// 77 us (293 MB: 3.8 TB/s; 44 at the copy rate), one of 100,000 25 us (9), 64 of 16 to
// 32,768, 16/2 heads, D 256, 41 us (16).  Nothing is full: half of the issue slots are
// used (a third at D 256), half of DRAM's rate, a fifth of the tensor pipe, and hardly
// a stall is memory's.  Each warp copies, scores, exponentiates and sums one tile
// behind another, and three warps a scheduler (two at D 256) are what the registers
// hold.  Beginning and join are 10, 8 and 12 us of these.
// A unit has 16 rows, so long chunks read and unmask the keys once for every 16 / group
// tokens: 8 sequences of 8192 with 1, 5, 16, 64 and 256 tokens each take 40, 62, 126,
// 388 and 1430 us (193 TFLOP/s), over 16-bit keys and values 44, 56, 66, 167 and 365.
#include <cuda_runtime.h>
#include <math.h>
#include <math_constants.h>

#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_ops.h"
#include "pa_q4.h"
#include "pa_share.cuh"

namespace pa {
namespace {

constexpr int kQ4Warps = 4;
constexpr int kQ4Threads = kQ4Warps * 32;
constexpr int kQ4MaxCtas = 4 * 152;                       // of a grid
constexpr int kQ4Shares = (1 + kShareSmall) * kQ4MaxCtas * kQ4Warps;  // that a workspace has places for
constexpr float kQ4Margin = 8.f;           // log2 units
constexpr float kQ4Shift = 7.f;            // weights are 2^(x + log2 S - maximum in use + this): up to 2^15
constexpr float kQ4LeastStep = 0x1p-24f;   // f16's smallest: stands in for a step of 0
constexpr float kQ4None = -3.402823466e38f;  // the maximum of no keys

enum { kQ4Whole = 0, kQ4Place0 = 1, kQ4Place1 = 2, kQ4End = 3 };

// A piece of a unit, as the walk hands it from a warp's copies to its products.
struct alignas(16) Q4Piece {
  int tok, end;       // the warp's first token, the end of the unit's tokens
  int steps, dest;
  int rows, row0;     // columns of the unit, its first query row
  int kvh, lim_base;  // column c sees the tokens below lim_base + c / group + 1
  int share, parts;   // parts: the shares that the unit lies in, with its first piece
  int pad[2];
};
constexpr int kQ4Head = 3;         // tiles' time that a piece's beginning and end take
// (a small share always has steps: a warp that is given none takes no more)
static_assert(kShareTwo * kShareSmallPct / (100 * kShareSmall) > kQ4Head, "small shares longer than a head");
constexpr float kMiddle = 7.5f;       // of the codes
constexpr int kQ4Pieces = 8;  // handed over and not yet taken: at most stages + 1

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float log2f_fast(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// The scales of a token's groups.
template <int NG>
__device__ __forceinline__ void load_scales(const uint8_t *at, float2 (&z)[NG]) {
  uint32_t w[NG];
  if constexpr (NG == 1) {
    w[0] = *reinterpret_cast<const uint32_t *>(at);
  } else if constexpr (NG == 2) {
    const uint2 v = *reinterpret_cast<const uint2 *>(at);
    w[0] = v.x, w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4 *>(at);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
#pragma unroll
  for (int i = 0; i < NG; ++i) z[i] = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
}
template <int D, int NT>
struct Q4Shape {
  static constexpr int NG = D / kQ4Group;   // groups of a head
  static constexpr int RB = D / 2;          // bytes of a row's codes
  static constexpr int CPR = RB / 16;       // 16-byte pieces (32 codes) of a row
  static constexpr int GM = 8 * NT;         // columns of a unit
  // tiles of 16 tokens that a warp takes at once: two give the MMAs of one
  // something to run beside, where registers allow (D 64, 16 columns: 68.5 -> 57.8 us)
  static constexpr int TT = D <= 128 ? 2 : 1;
  static constexpr int TOKENS = 16 * TT;  // of a step
  static constexpr int QREGS = CPR * NT * 4;
  static constexpr bool QSMEM = QREGS > 32;  // query fragments in shared memory
  static constexpr int KEYS = 0, VALUES = TOKENS * RB, KSC = 2 * TOKENS * RB, VSC = KSC + TOKENS * 4 * NG,
                       STAGE = VSC + TOKENS * 4 * NG;
  // CTAs an SM by registers (with a third that spilled a few, D 256 took 122 us
  // instead of 79, 16 columns at D 128 178 instead of 117), and the ring that
  // their shared memory leaves
  static constexpr int CTAS = NT == 1 ? (D == 64 ? 4 : D == 128 ? 3 : 2) : (D == 64 ? 3 : 2);
  static constexpr int STAGES = D == 256 || (D == 128 && NT == 1) ? 3 : 4;
  static constexpr int CACHE = D == 256 && NT == 1 ? 64 : 384;  // sequences of the plan kept by
  static constexpr int QBUF = QSMEM ? QREGS * 128 : 0;  // a warp's
  static constexpr int SMEM = kQ4Warps * (STAGES * STAGE + QBUF);
  // where piece c of row r stands: eight rows' pieces c in eight 16-byte columns
  __device__ static __forceinline__ int at(int r, int c) {
    return r * RB + ((c ^ (CPR == 2 ? (r >> 2) & 1 : CPR == 4 ? (r >> 1) & 3 : r & 7)) << 4);
  }
};

struct Q4Batch {
  const Q4Params &p;
  int num_seqs, step;  // step: tokens
  bool tell;           // report what is bad
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
    ShareSeq q{r.x, r.y, r.z, 0, 0, kQ4Head};
    q.steps = (r.x + step - 1) / step;  // (at most 2^30 keys)
    if (q.steps > 0)
      q.units = p.q_start ? p.num_kv_heads * ((r.z + p.chunk_tokens - 1) / p.chunk_tokens) : p.num_kv_heads;
    return q;
  }
};

}  // namespace

template <typename T, int D, int NT, bool CHUNK>
__global__ void __launch_bounds__(kQ4Threads, Q4Shape<D, NT>::CTAS)
    pa_q4_kernel(const __grid_constant__ Q4Params p, const __grid_constant__ ShareSpace space) {
  using Z = Q4Shape<D, NT>;
  constexpr int NG = Z::NG, RB = Z::RB, CPR = Z::CPR, GM = Z::GM, NST = Z::STAGES, TT = Z::TT;
  extern __shared__ __align__(128) uint8_t smem_q4[];
  __shared__ ShareScan<kQ4Threads, Z::CACHE> s_scan;
  __shared__ Q4Piece s_piece[kQ4Warps][kQ4Pieces];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t *ring = smem_q4 + warp * (NST * Z::STAGE);
  const uint32_t ring_u32 = smem_u32(ring);
  uint4 *qbuf = reinterpret_cast<uint4 *>(smem_q4 + kQ4Warps * NST * Z::STAGE + warp * Z::QBUF);

  pdl_wait_primary();
  Q4Batch batch{p, p.num_seqs, Z::TOKENS, blockIdx.x == 0};
  share_scan(batch, s_scan);
  batch.tell = false;
  SharePlan plan;
  plan.make(s_scan.cum[kQ4Threads], (int)gridDim.x * kQ4Warps);

  // the row of the query (and output) that is column c of a unit
  auto query_row = [&](int row0, int kvh, int c) -> size_t {
    const int tok = CHUNK ? c / p.group : 0;
    return (size_t)(row0 + tok) * p.num_heads + (size_t)(kvh * p.group + c - tok * p.group);
  };

  // ---- the walk over the share, a tile ahead of the copies
  ShareWalk walk{};
  int share = (int)blockIdx.x * kQ4Warps + warp;  // the one that is walked
  walk.begin(batch, s_scan, plan.begin(share), share < plan.big ? plan.begin(share + 1) : 0);
  int handed = 0;                                  // pieces
  int ahead = -1;                                  // (lane 0) a small share taken before it is needed
  int f_left = 0, f_tok = 0, f_end = 0, f_at = 0;  // tiles left of the piece, their next token, its KV head's place
  const int32_t *table = p.block_tables;
  const int hbs = p.num_kv_heads * p.block_size;
  auto next_piece = [&]() {
    if (walk.left <= 0 && plan.small > 0) {
      if (lane == 0 && ahead < 0) ahead = atomicAdd(space.counters + kShareTaken, 1) & 0x7fffffff;
      const int k = __shfl_sync(0xffffffffu, ahead, 0);
      ahead = -1;
      share = plan.big + k;
      if (k < plan.small) walk.begin(batch, s_scan, plan.begin(share), plan.begin(share + 1));
    }
    Q4Piece u{};
    u.dest = kQ4End;
    if (walk.left > 0) {
      const int n = walk.steps(), step = walk.first();
      u.kvh = walk.unit;
      u.rows = p.group;
      u.row0 = walk.s;
      u.lim_base = walk.q.len - 1;
      u.end = walk.q.len;
      if (CHUNK) {
        const int nrg = (walk.q.n + p.chunk_tokens - 1) / p.chunk_tokens;
        u.kvh = walk.unit / nrg;
        const int t0 = (walk.unit - u.kvh * nrg) * p.chunk_tokens, nt = min(p.chunk_tokens, walk.q.n - t0);
        u.rows = nt * p.group;
        u.row0 = walk.q.row0 + t0;
        u.lim_base = walk.q.len - walk.q.n + t0;
        u.end = u.lim_base + nt;
      }
      u.dest = step > 0 ? kQ4Place0 : step + n == walk.q.steps ? kQ4Whole : kQ4Place1;
      u.steps = n;
      u.share = share;
      u.tok = step * Z::TOKENS;
      if (u.dest == kQ4Place1) u.parts = plan.of(walk.last()) - share + 1;
      // (its queries on their way to L2)
#pragma unroll
      for (int i = lane; i < GM * (D / 64); i += 32) {
        const int c = i / (D / 64);
        if (c < u.rows)
          prefetch_l2(static_cast<const T *>(p.query) + query_row(u.row0, u.kvh, c) * D + i % (D / 64) * 64);
      }
      table = p.block_tables + (size_t)walk.s * p.max_blocks_per_seq;
      f_left = n;
      f_tok = u.tok;
      f_end = u.end;
      f_at = u.kvh * p.block_size;
      walk.next(batch, s_scan);
    }
    if (lane == 0) s_piece[warp][handed & (kQ4Pieces - 1)] = u;
    ++handed;
  };
  // the table entries of the next tiles, of 16 tokens each (of pages of 8 tokens: looked
  // up with the copies)
  int e[TT];
#pragma unroll
  for (int h = 0; h < TT; ++h) e[h] = -1;
  auto look_up = [&]() {
#pragma unroll
    for (int h = 0; h < TT; ++h)
      if (f_left > 0 && f_tok + 16 * h < f_end) e[h] = __ldg(table + ((f_tok + 16 * h) >> p.log2_block_size));
  };
  next_piece();
  look_up();

  // ---- one stage of copies
  const uint32_t lane_dst = ring_u32 + (uint32_t)Z::at(lane / CPR, lane % CPR);
  const uint8_t *const keys = p.key_codes + lane * 16, *const values = p.value_codes + lane * 16;
  const uint8_t *const key_scales = static_cast<const uint8_t *>(p.key_scales), *const value_scales = static_cast<const uint8_t *>(p.value_scales);
  auto issue = [&](uint32_t slot) {  // (a slot is its offset in the ring)
    if (f_left > 0) {
      bool whole = f_end - f_tok >= Z::TOKENS && p.block_size != 8;
#pragma unroll
      for (int h = 0; h < TT; ++h) whole = whole && (unsigned)e[h] < (unsigned)p.num_blocks;
      if (whole) {
#pragma unroll
        for (int h = 0; h < TT; ++h) {  // sixteen rows one behind the other
          const uint32_t row = (uint32_t)e[h] * hbs + (f_at + ((f_tok + 16 * h) & (p.block_size - 1)));
          const uint8_t *k = keys + (size_t)row * RB, *v = values + (size_t)row * RB;
          const uint32_t dst = lane_dst + slot + 16u * RB * h;
#pragma unroll
          for (int j = 0; j < CPR / 2; ++j) {
            // rows 32 j / CPR on: eight (or sixteen) rows swap pieces alike, four rows
            // (CPR 8) on the other side
            const uint32_t to = (CPR == 8 && (j & 1) ? dst ^ 64u : dst) + 512u * j;
            cp_async16(to + Z::KEYS, k + 512 * j, 16);
            cp_async16(to + Z::VALUES, v + 512 * j, 16);
          }
          const size_t sc = (size_t)(row + (lane & 15)) * (4 * NG);
          cp_async_small<4 * NG>(ring_u32 + slot + (lane < 16 ? Z::KSC : Z::VSC) + (16 * h + (lane & 15)) * 4 * NG,
                                 (lane < 16 ? key_scales : value_scales) + sc, 4 * NG);
        }
      } else if (f_end > f_tok) {
        // the last tokens, pages of 8, bad entries: row by row; rows out of range are zeros
        auto place = [&](int r, bool &on) -> size_t {
          on = f_tok + r < f_end;
          const int blk = on ? __ldg(table + ((f_tok + r) >> p.log2_block_size)) : 0;
          if ((unsigned)blk >= (unsigned)p.num_blocks) {
            report(p.status, kStatusBadInput);
            on = false;
          }
          return on ? (size_t)(uint32_t)(blk * hbs + f_at + ((f_tok + r) & (p.block_size - 1))) : 0;
        };
#pragma unroll
        for (int j = 0; j < TT * CPR / 2; ++j) {
          const int i = lane + 32 * j, r = i / CPR, c = i % CPR;
          const uint32_t to = ring_u32 + slot + (uint32_t)Z::at(r, c);
          bool on;
          size_t src = place(r, on) * RB;
          src += on ? c * 16 : 0;
          cp_async16(to + Z::KEYS, p.key_codes + src, on ? 16 : 0);
          cp_async16(to + Z::VALUES, p.value_codes + src, on ? 16 : 0);
        }
#pragma unroll
        for (int h = 0; h < TT; ++h) {
          const int r = 16 * h + (lane & 15);
          bool on;
          const size_t src = place(r, on) * (4 * NG);
          cp_async_small<4 * NG>(ring_u32 + slot + (lane < 16 ? Z::KSC : Z::VSC) + r * 4 * NG,
                                 (lane < 16 ? key_scales : value_scales) + src, on ? 4 * NG : 0);
        }
      }
      f_tok += Z::TOKENS;
      if (--f_left == 0) next_piece();
      if (f_left == 2 && walk.left <= 0 && plan.small > 0 && lane == 0 && ahead < 0)
        ahead = atomicAdd(space.counters + kShareTaken, 1) & 0x7fffffff;
      look_up();
    }
    cp_async_commit();
  };

#pragma unroll
  for (int i = 0; i < NST - 1; ++i) issue((uint32_t)(i * Z::STAGE));

  const uint32_t middle = g == 0 ? 0xc780c780u : 0u;  // (f16) -kMiddle
  // ---- the tiles
  uint4 qf[Z::QSMEM ? 1 : NT][Z::QSMEM ? 1 : CPR];  // Q^T fragments of two k-steps
  float qsum[NT][NG][2];  // scale x the sum of the group's q, of this lane's columns
  float qmul[NT][2];      // what the columns' products are worth
  float o[NT][2 * CPR][4];  // O^T: row pairs (g, g + 8), columns 2t, 2t + 1
  float sl[NT][2], sb[NT][NG][2], m[NT][2];  // m: 2^kQ4Shift below the maximum in use
  int lim[CHUNK ? NT : 1][2];
  int rows = 0, row0 = 0, kvh = 0, dest = 0, at_share = 0, parts = 0, left = 0, tok = 0, end = 0, taken = 0;

  // (slots: of this tile, and of the one to copy, whose last tile is done with)
  for (uint32_t slot = 0, copy = (NST - 1) * Z::STAGE;; copy = slot, slot = slot + Z::STAGE == NST * Z::STAGE ? 0 : slot + Z::STAGE) {
    cp_async_wait<NST - 2>();
    __syncwarp();
    const uint8_t *stage = ring + slot;
    const uint32_t stage_u32 = ring_u32 + slot;
    if (left == 0) {
      const Q4Piece u = s_piece[warp][taken++ & (kQ4Pieces - 1)];
      if (u.dest == kQ4End) break;
      rows = u.rows, row0 = u.row0, kvh = u.kvh, dest = u.dest, at_share = u.share, parts = u.parts;
      left = u.steps, tok = u.tok, end = u.end;
      // queries: lane (g, t) has elements 8 t .. 8 t + 7 of each 32 of column g
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int c = nt * 8 + g;
        const bool live = c < rows;
        const uint4 *src =
            reinterpret_cast<const uint4 *>(static_cast<const T *>(p.query) + (live ? query_row(row0, kvh, c) : 0) * D) + t;
        float top = 0.f, sum[NG];
#pragma unroll
        for (int i = 0; i < NG; ++i) sum[i] = 0.f;
#pragma unroll
        for (int ch = 0; ch < CPR; ++ch) {
          const uint4 a = live ? __ldg(src + 4 * ch) : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 f = MmaOp<T>::unpack(w[i]);
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
            sum[ch >> 1] += f.x + f.y;
          }
        }
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
          sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // the head times 2^(14 - e), e the exponent of its largest: below 2^15
        const int e = max((int)(__float_as_uint(top) >> 23) - 127, -100);
        const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
        // (scores come in units of 2^(e - 14) 2^-24)
        const float down = top < CUDART_INF_F ? __uint_as_float((uint32_t)(127 + e) << 23) * 0x1p10f : CUDART_NAN_F;
#pragma unroll
        for (int ch = 0; ch < CPR; ++ch) {
          const uint4 a = live ? __ldg(src + 4 * ch) : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t w[4] = {a.x, a.y, a.z, a.w};
          float f[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 v = MmaOp<T>::unpack(w[i]);
            f[2 * i] = v.x * up, f[2 * i + 1] = v.y * (up * 0.0625f);
          }
          // elements 0, 4 | 2, 6 against the codes 2^-24, then 1, 5 | 3, 7 against 2^-20
          using H = MmaOp<__half>;
          const uint4 q = make_uint4(H::pack(f[0], f[4]), H::pack(f[2], f[6]), H::pack(f[1], f[5]), H::pack(f[3], f[7]));
          if constexpr (Z::QSMEM)
            qbuf[(nt * CPR + ch) * 32 + lane] = q;
          else
            qf[nt][ch] = q;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          qmul[nt][i] = __shfl_sync(0xffffffffu, down, 8 * t + 4 * i) * p.scale_log2;
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            qsum[nt][gr][i] = __shfl_sync(0xffffffffu, sum[gr], 8 * t + 4 * i) * p.scale_log2;
            sb[nt][gr][i] = 0.f;
          }
          sl[nt][i] = 0.f;
          m[nt][i] = kQ4None;
          if (CHUNK) lim[nt][i] = u.lim_base + (nt * 8 + 2 * t + i) / p.group + 1;
        }
#pragma unroll
        for (int i = 0; i < 2 * CPR; ++i)
#pragma unroll
          for (int e2 = 0; e2 < 4; ++e2) o[nt][i][e2] = 0.f;
      }
      if (Z::QSMEM) __syncwarp();
    }
    issue(copy);

    const int valid = end - tok;
    if (valid > 0) {
      // ---- scores of tokens g, g + 8 (of each tile) and columns 2t, 2t + 1
      constexpr uint32_t kLow = 0x000f000fu, kHigh = 0x00f000f0u;
      const int r = lane & 15, c1 = lane >> 4;
      float x[TT][NT][4];
#pragma unroll
      for (int h = 0; h < TT; ++h) {
        const uint32_t krow = stage_u32 + Z::KEYS + 16 * RB * h;
        float y[NT][4];
        float2 ka[NG], kb[NG];  // scales of tokens g and g + 8
        load_scales<NG>(stage + Z::KSC + (16 * h + g) * NG * 4, ka);
        load_scales<NG>(stage + Z::KSC + (16 * h + g + 8) * NG * 4, kb);
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          uint32_t w0, w1, w2, w3;  // rows g and g + 8, pieces 2 gr and 2 gr + 1
          ldsm_x4(krow + (uint32_t)Z::at(r, 2 * gr + c1), w0, w1, w2, w3);
          float acc[NT][4];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t a = c ? w2 : w0, b = c ? w3 : w1, a8 = a >> 8, b8 = b >> 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint4 q;
              if constexpr (Z::QSMEM)
                q = qbuf[(nt * CPR + 2 * gr + c) * 32 + lane];
              else
                q = qf[nt][2 * gr + c];
              if (c == 0)
                mma_first(acc[nt], a & kLow, b & kLow, a8 & kLow, b8 & kLow, q.x, q.y);
              else
                MmaOp<__half>::run(acc[nt], a & kLow, b & kLow, a8 & kLow, b8 & kLow, q.x, q.y);
              MmaOp<__half>::run(acc[nt], a & kHigh, b & kHigh, a8 & kHigh, b8 & kHigh, q.z, q.w);
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float2 z = i < 2 ? ka[gr] : kb[gr];
              y[nt][i] = gr ? fmaf(z.y, acc[nt][i], y[nt][i]) : z.y * acc[nt][i];
              x[h][nt][i] = gr ? fmaf(z.x, qsum[nt][gr][i & 1], x[h][nt][i]) : z.x * qsum[nt][gr][i & 1];
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) x[h][nt][i] = fmaf(qmul[nt][i & 1], y[nt][i], x[h][nt][i]);
      }
      // ---- values' scales of tokens g and g + 8, and the larger steps S (by magnitude:
      // codes may count downwards)
      float2 va[TT][NG], vb[TT][NG];
      float inv_a[TT], inv_b[TT];
      bool raise = false;
#pragma unroll
      for (int h = 0; h < TT; ++h) {
        load_scales<NG>(stage + Z::VSC + (16 * h + g) * NG * 4, va[h]);
        load_scales<NG>(stage + Z::VSC + (16 * h + g + 8) * NG * 4, vb[h]);
        float top_a = kQ4LeastStep, top_b = kQ4LeastStep;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) top_a = fmaxf(top_a, fabsf(va[h][gr].y)), top_b = fmaxf(top_b, fabsf(vb[h][gr].y));
        const float lg_a = log2f_fast(top_a), lg_b = log2f_fast(top_b);
        inv_a[h] = rcp(top_a), inv_b[h] = rcp(top_b);
        // the maximum in use is raised when x + log2 S is 8 above it: any reference
        // serves the sums as long as nothing overflows (rounded down here and up
        // there, so that no weight passes 2^15 however far the scores are)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          x[h][nt][0] += lg_a, x[h][nt][1] += lg_a, x[h][nt][2] += lg_b, x[h][nt][3] += lg_b;
          if (valid < Z::TOKENS) {
            if (16 * h + g >= valid) x[h][nt][0] = x[h][nt][1] = -CUDART_INF_F;
            if (16 * h + g + 8 >= valid) x[h][nt][2] = x[h][nt][3] = -CUDART_INF_F;
          }
          if (CHUNK) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (tok + 16 * h + g + 4 * (i & 2) >= lim[nt][i & 1]) x[h][nt][i] = -CUDART_INF_F;
          }
          raise = raise || fmaxf(x[h][nt][0], x[h][nt][2]) > __fadd_rd(m[nt][0], kQ4Margin + kQ4Shift) ||
                  fmaxf(x[h][nt][1], x[h][nt][3]) > __fadd_rd(m[nt][1], kQ4Margin + kQ4Shift);
        }
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float top = -CUDART_INF_F;
#pragma unroll
            for (int h = 0; h < TT; ++h) top = fmaxf(top, fmaxf(x[h][nt][i], x[h][nt][i + 2]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            top = fmaxf(__fsub_ru(top, kQ4Shift), m[nt][i]);
            const float f = ex2f(m[nt][i] - top);
            m[nt][i] = top;
#pragma unroll
            for (int c = 0; c < 2 * CPR; ++c) o[nt][c][i] *= f, o[nt][c][i + 2] *= f;
            sl[nt][i] *= f;
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) sb[nt][gr][i] *= f;
          }
      }
#pragma unroll
      for (int h = 0; h < TT; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int i = 0; i < 4; ++i) x[h][nt][i] = ex2f(x[h][nt][i] - m[nt][i & 1]);
          sl[nt][0] = fmaf(x[h][nt][0], inv_a[h], fmaf(x[h][nt][2], inv_b[h], sl[nt][0]));
          sl[nt][1] = fmaf(x[h][nt][1], inv_a[h], fmaf(x[h][nt][3], inv_b[h], sl[nt][1]));
        }
      // ---- O^T += V^T P^T, group by group
#pragma unroll
      for (int h = 0; h < TT; ++h) {
        const uint32_t vrow = stage_u32 + Z::VALUES + 16 * RB * h;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          const float wa = va[h][gr].y * inv_a[h], wb = vb[h][gr].y * inv_b[h];
          float la = va[h][gr].x * inv_a[h], lb = vb[h][gr].x * inv_b[h];
          la = fmaf(kMiddle, wa, la), lb = fmaf(kMiddle, wb, lb);
          uint32_t pf[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float *y = x[h][nt];
            sb[nt][gr][0] = fmaf(y[0], la, fmaf(y[2], lb, sb[nt][gr][0]));
            sb[nt][gr][1] = fmaf(y[1], la, fmaf(y[3], lb, sb[nt][gr][1]));
            pf[nt][0] = movmatrix_trans(MmaOp<__half>::pack(y[0] * wa, y[1] * wa));
            pf[nt][1] = movmatrix_trans(MmaOp<__half>::pack(y[2] * wb, y[3] * wb));
            // - 7.5 sum(w), to the lanes of row 0
            float d[4] = {sb[nt][gr][0], sb[nt][gr][1], 0.f, 0.f};
            MmaOp<__half>::run(d, middle, 0u, middle, 0u, pf[nt][0], pf[nt][1]);
            sb[nt][gr][0] = d[0], sb[nt][gr][1] = d[1];
          }
          // units of four codes: tokens 2t, 2t + 1 | the eight behind, pieces 2 gr, 2 gr + 1
          uint32_t w[4];
          ldsm_x4_trans(vrow + (uint32_t)Z::at(r, 2 * gr + c1), w[0], w[1], w[2], w[3]);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t a = w[2 * c], b = w[2 * c + 1], a8 = a >> 8, b8 = b >> 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              // codes 0 and 2 of a unit (2^-24 each), then 1 and 3 (2^-20)
              MmaOp<__half>::run(o[nt][2 * (2 * gr + c)], a & kLow, a8 & kLow, b & kLow, b8 & kLow, pf[nt][0], pf[nt][1]);
              MmaOp<__half>::run(o[nt][2 * (2 * gr + c) + 1], a & kHigh, a8 & kHigh, b & kHigh, b8 & kHigh, pf[nt][0],
                                 pf[nt][1]);
            }
          }
        }
      }
    }

    tok += Z::TOKENS;
    if (--left == 0) {
      // ---- the piece's sums: out, or into its place
      if (dest == kQ4Place1 && lane == 0) {
        ShareJoin j{};
        j.share = at_share;
        j.parts = parts;
        j.by = 1;
        j.rows = rows;
        j.group = p.group;
        j.stride = p.num_heads;
        j.out_row = (long long)row0 * p.num_heads + kvh * p.group;
        share_join(space, j);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e2 = 0; e2 < 2; ++e2) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            sl[nt][e2] += __shfl_xor_sync(0xffffffffu, sl[nt][e2], d);
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) sb[nt][gr][e2] += __shfl_xor_sync(0xffffffffu, sb[nt][gr][e2], d);
          }
          const int c = nt * 8 + 2 * t + e2;
          if (c < rows) {
            const float inv = dest != kQ4Whole ? 1.f : sl[nt][e2] == 0.f ? 0.f : 1.f / sl[nt][e2];
            const float fa = inv * 0x1p24f, fb = inv * 0x1p20f;
            const size_t place = (2 * (size_t)at_share + (dest == kQ4Place1 ? 1 : 0)) * GM + c;
            if (dest != kQ4Whole && g == 0) space.ml[place] = make_float2(m[nt][e2], sl[nt][e2]);
            T *out = static_cast<T *>(p.out) + query_row(row0, kvh, c) * D + 4 * g;
            float *part = space.o + place * D + 4 * g;
#pragma unroll
            for (int ch = 0; ch < CPR; ++ch) {
              // rows 32 ch + 4 g + 0 .. 3
              const float b = sb[nt][ch >> 1][e2] * inv;
              const float r0 = fmaf(o[nt][2 * ch][e2], fa, b), r1 = fmaf(o[nt][2 * ch + 1][e2], fb, b);
              const float r2 = fmaf(o[nt][2 * ch][e2 + 2], fa, b), r3 = fmaf(o[nt][2 * ch + 1][e2 + 2], fb, b);
              if (dest == kQ4Whole)
                store4(out + 32 * ch, r0, r1, r2, r3);
              else
                store4(part + 32 * ch, r0, r1, r2, r3);
            }
          }
        }
    }
  }
  // (earlier, the join's CTAs would wait beside this grid's: 76 -> 92 us)
  pdl_launch_dependents();
  // outputs of empty sequences
  if (!CHUNK)
    for (int q = blockIdx.x; q < p.num_seqs; q += gridDim.x)
      if (share_seq(batch, s_scan, q).len == 0) {
        uint4 *z = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + (size_t)q * p.num_heads * D);
        for (int i = threadIdx.x; i < p.num_heads * D / 8; i += kQ4Threads) z[i] = make_uint4(0u, 0u, 0u, 0u);
      }
}

namespace {

struct Q4Kernel {
  const void *fn;
  int ctas, smem;
};
template <typename T, int D, int NT>
Q4Kernel q4_pick2(bool chunk) {
  using Z = Q4Shape<D, NT>;
  if (NT == 1 && !chunk) return {reinterpret_cast<const void *>(&pa_q4_kernel<T, D, NT, false>), Z::CTAS, Z::SMEM};
  if (NT == 2)
    return {chunk ? reinterpret_cast<const void *>(&pa_q4_kernel<T, D, 2, true>)
                  : reinterpret_cast<const void *>(&pa_q4_kernel<T, D, 2, false>),
            Z::CTAS, Z::SMEM};
  return {};
}
template <typename T>
Q4Kernel q4_pick(int head_size, int nt, bool chunk) {
  switch (head_size * 10 + nt) {
    case 641: return q4_pick2<T, 64, 1>(chunk);
    case 642: return q4_pick2<T, 64, 2>(chunk);
    case 1281: return q4_pick2<T, 128, 1>(chunk);
    case 1282: return q4_pick2<T, 128, 2>(chunk);
    case 2561: return q4_pick2<T, 256, 1>(chunk);
    case 2562: return q4_pick2<T, 256, 2>(chunk);
  }
  return {};
}

}  // namespace
}  // namespace pa

extern "C" {

size_t pa_q4_workspace_bytes(int head_size) {
  if (head_size != 64 && head_size != 128 && head_size != 256) return 0;
  return pa::share_bytes(pa::kQ4Shares, 16, head_size, nullptr, nullptr);
}

pa_status_t pa_q4_forward(void *out, const void *query, const void *key_cache, const void *value_cache,
                          const void *key_scales, const void *value_scales, const int32_t *block_tables,
                          const int32_t *seq_lens, const int32_t *q_start, int num_seqs, int num_rows,
                          int num_heads, int num_kv_heads, int head_size, int num_blocks, int block_size,
                          int max_blocks_per_seq, int max_seq_len, float scale, int dtype, void *workspace,
                          size_t workspace_bytes, void *stream) {
  using namespace pa;
  pa_status_t st = host_check_cache(dtype, num_heads, num_kv_heads, head_size, num_blocks, block_size,
                                    max_blocks_per_seq, max_seq_len);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || num_rows < 0 || (!q_start && num_rows != num_seqs)) return PA_ERR_INVALID_ARG;
  if (!isfinite(scale)) return PA_ERR_INVALID_ARG;
  if (dtype == PA_DTYPE_F32) return PA_ERR_UNSUPPORTED;  // tensor path only
  if (max_seq_len > kMaxTokens) return PA_ERR_UNSUPPORTED;
  if (num_rows == 0 || num_seqs == 0) return PA_OK;  // (empty tensors have no address)
  if (!out || !query || !key_cache || !value_cache || !key_scales || !value_scales || !block_tables ||
      !seq_lens || !workspace)
    return PA_ERR_INVALID_ARG;
  const void *wide[] = {out, query, key_cache, value_cache, key_scales, value_scales};
  for (const void *q : wide)
    if (!host_aligned(q, 16)) return PA_ERR_INVALID_ARG;
  const void *ints[] = {block_tables, seq_lens, q_start};
  for (const void *q : ints)
    if (!host_aligned(q, 4)) return PA_ERR_INVALID_ARG;
  if (!host_aligned(workspace, 256)) return PA_ERR_INVALID_ARG;
  if (workspace_bytes < pa_q4_workspace_bytes(head_size)) return PA_ERR_WORKSPACE_TOO_SMALL;

  Q4Params p{};
  p.key_codes = static_cast<const uint8_t *>(key_cache);
  p.value_codes = static_cast<const uint8_t *>(value_cache);
  p.key_scales = key_scales;
  p.value_scales = value_scales;
  p.query = query;
  p.out = out;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.q_start = q_start;
  p.status = static_cast<int *>(workspace);
  p.num_seqs = num_seqs;
  p.num_rows = num_rows;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = num_heads / num_kv_heads;
  p.num_blocks = num_blocks;
  p.block_size = block_size;
  while ((1 << p.log2_block_size) < block_size) ++p.log2_block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_seq_len = max_seq_len;
  p.scale_log2 = scale * 1.4426950408889634f;
  const int nt = q_start || p.group > 8 ? 2 : 1;
  p.chunk_tokens = 16 / p.group;

  int sms = 0;
  st = host_sm_count(&sms);
  if (st != PA_OK) return st;
  const Q4Kernel k = dtype == PA_DTYPE_BF16 ? q4_pick<__nv_bfloat16>(head_size, nt, q_start != nullptr)
                                            : q4_pick<__half>(head_size, nt, q_start != nullptr);
  st = host_ensure_smem(k.fn, (size_t)k.smem + 16 * 1024);  // (the kernel's static part counts against the same limit)
  if (st != PA_OK) return st;
  const int ctas = sms * k.ctas < kQ4MaxCtas ? sms * k.ctas : kQ4MaxCtas;
  ShareSpace space;
  share_bytes(kQ4Shares, 16, head_size, workspace, &space);
  void *args[2] = {&p, &space};
  st = host_launch(k.fn, (unsigned)ctas, 1, kQ4Threads, k.smem, stream, args, "launch 4-bit attention kernel");
  if (st != PA_OK) return st;
  JoinParams j{};
  j.space = space;
  j.out = out;
  j.max_rows = 8 * nt;
  j.item_rows = q_start ? p.chunk_tokens * p.group : p.group;
  j.width = head_size;
  return share_launch_join(j, dtype == PA_DTYPE_BF16, sms, stream);
}

}  // extern "C"
