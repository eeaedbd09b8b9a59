// pa_q4_forward: decode attention (and chunks of query tokens) over a cache
// whose keys and values are held in 4 bits (pa_q4.h).
//
// With codes c, lowest values lo and steps st, group by group of 64 elements,
//   q . K_t      = sum_g st_tg (q_g . c_tg) + lo_tg sum(q_g)
//   sum_t p_t V_t = sum_t (p_t st_t) c_t + sum_t p_t lo_t      (of each group)
// so the codes go into the matrix products as they are, and the steps and
// lowest values meet scores and weights instead of elements.  A code becomes
// an element of the MMA by a shift and one logic operation for two of them:
// its four bits are the top of the mantissa of 16, which makes 16 + c.  The
// 16s come off again with lo: lo' = lo - 16 st.
//
// Weights: w = p st is rounded to bf16 for the product, and the sums take what
// the product took: with a = 1 / st and b = lo' / st,
//   out = (sum_t w_t (16 + c_t) + sum_t w_t b_t) / sum_t w_t a_t,
// so that rounding w is rounding the softmax's weight, no more (the 16s and
// lo would else be weighed differently from the codes).
//
// Layout: S^T[16 tokens][8 heads] = K Q^T and O^T[D][8 heads] += V^T P^T by
// mma.sync m16n8k16, a warp 16 tokens at a time.  Which element of a head is
// which k of the product is free, and so is which element of V is which row of
// O^T; both are chosen so that a lane's codes are whole words of a token's
// row: words 4 t + .. (t = lane % 4) of a key's group, word g (g = lane / 4) of
// a value's.  Rows sit in shared memory in an order (and with their 32-byte
// groups swapped) that keeps those reads free of bank conflicts.
//
// A CTA has four warps; of every 64 tokens each takes 16, copied by cp.async
// into its own ring, so no warp waits for another until the end of a piece of
// a unit, where the four merge.  Work is split in equal shares (pa_share.cuh).
#include <cuda_runtime.h>
#include <limits.h>
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
constexpr float kQ4Margin = 8.f;           // log2 units
constexpr float kQ4LeastStep = 0x1p-24f;   // f16's smallest: stands in for a step of 0

constexpr int kQ4First = 1, kQ4Last = 2, kQ4End = 4;
enum { kQ4Whole = 0, kQ4Place0 = 1, kQ4Place1 = 2 };

// What a warp's ring stage holds, written with its copies.
struct alignas(16) Q4Head {
  int flags, valid;   // tokens of the stage in range
  int tok0;           // the first of them
  int lim_base;       // column c sees the tokens below lim_base + c / group + 1
  int rows, row0;     // columns of the unit, its first query row
  int kvh, dest;
};

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
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  return __byte_perm(a, b, sel);
}

// Codes i and i + 4 of a word as the pair 16 + c_i, 16 + c_(i+4) of T: the code
// at the top of the mantissa of 16.0.
template <typename T, int I>
__device__ __forceinline__ uint32_t code_pair(uint32_t w) {
  constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
  constexpr int at = bf ? 3 : 6;  // lowest bit of the mantissa's top four
  constexpr uint32_t mask = (0xfu << at) * 0x10001u, base = bf ? 0x41804180u : 0x4c004c00u;
  const uint32_t x = 4 * I >= at ? w >> (4 * I - at) : w << (at - 4 * I);
  return (x & mask) | base;
}

template <int D, int NT>
struct Q4Shape {
  static constexpr int NG = D / kQ4Group;   // groups of a head
  static constexpr int RB = D / 2;          // bytes of a row's codes
  static constexpr int CPR = RB / 16;       // 16-byte pieces of a row
  static constexpr int GM = 8 * NT;         // columns of a unit
  static constexpr int KEYS = 0, VALUES = 16 * RB, KSC = 32 * RB, VSC = KSC + 64 * NG,
                       HEAD = VSC + 64 * NG, STAGE = (HEAD + (int)sizeof(Q4Head) + 127) / 128 * 128;
  // CTAs an SM by registers, and the ring that their shared memory leaves
  static constexpr int CTAS = NT == 1 ? (D == 256 ? 3 : 4) : (D == 256 ? 2 : 3);
  static constexpr int STAGES = D == 256 ? (NT == 1 ? 3 : 4) : 4;
  static constexpr int OROW = D + 4;        // floats between rows of the merge
  static constexpr int OBUF = 2 * GM * OROW * 4;
  static constexpr int SMEM = kQ4Warps * STAGES * STAGE + OBUF;
  // place of a token's row in a stage: the even ones of eight first, so that
  // the four tokens 2t that a warp reads at once are neighbours
  __device__ static __forceinline__ int place(int r) { return (r & 8) | ((r & 1) << 2) | ((r & 7) >> 1); }
  // which 32-byte group of a row stands where
  __device__ static __forceinline__ int swap(int pl) {
    return NG == 1 ? 0 : NG == 2 ? ((pl >> 1) ^ (pl >> 2)) & 1 : (pl & 3) ^ ((pl >> 1) & 2);
  }
};

struct Q4Batch {
  const Q4Params &p;
  int num_seqs;
  bool tell;  // report what is bad
  __device__ __forceinline__ ShareSeq seq(int s) const {
    ShareSeq q;
    q.len = __ldg(p.seq_lens + s);
    q.row0 = s;
    q.n = 1;
    q.units = p.num_kv_heads;
    bool bad = q.len < 0 || q.len > p.max_seq_len;
    if (p.q_start) {
      q.row0 = __ldg(p.q_start + s);
      const int e = __ldg(p.q_start + s + 1);
      q.n = e - q.row0;
      bad = bad || q.row0 < 0 || q.n < 0 || e > p.num_rows || q.n > q.len;
      q.units = bad ? 0 : p.num_kv_heads * ((q.n + p.chunk_tokens - 1) / p.chunk_tokens);
    }
    if (bad) {
      if (tell) report(p.status, kStatusBadInput);
      q.len = 0;
    }
    q.steps = (int)(((long long)q.len + kShareStep - 1) / kShareStep);
    if (q.steps == 0) q.units = 0;
    return q;
  }
};

}  // namespace

template <typename T, int D, int NT, bool CHUNK>
__global__ void __launch_bounds__(kQ4Threads, Q4Shape<D, NT>::CTAS)
    pa_q4_kernel(const __grid_constant__ Q4Params p, const __grid_constant__ ShareSpace space) {
  using Z = Q4Shape<D, NT>;
  constexpr int NG = Z::NG, RB = Z::RB, CPR = Z::CPR, GM = Z::GM, NST = Z::STAGES, KW = 4 * NG;
  extern __shared__ __align__(128) uint8_t smem_q4[];
  __shared__ ShareScan<kQ4Threads> s_scan;
  __shared__ float s_m[kQ4Warps][GM];               // a warp's maximum in use
  __shared__ float2 s_sum[kQ4Warps][GM][NG];        // its sums of w a, w b
  __shared__ float s_top[GM];                       // the merged maximum

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t *ring = smem_q4 + warp * (NST * Z::STAGE);
  const uint32_t ring_u32 = smem_u32(ring);
  float *obuf = reinterpret_cast<float *>(smem_q4 + kQ4Warps * NST * Z::STAGE);

  pdl_wait_primary();
  Q4Batch batch{p, p.num_seqs, blockIdx.x == 0};
  share_scan<kQ4Threads>(batch, s_scan);
  batch.tell = false;
  const long long total = s_scan.cum[kQ4Threads];
  const int shares = share_count(total, gridDim.x, 1), me = blockIdx.x;
  long long line = share_begin(total, me, shares), line_end = share_begin(total, me + 1, shares);
  if (me >= shares) line = line_end = total;

  // outputs of empty sequences
  if (!CHUNK)
    for (int s = me; s < p.num_seqs; s += gridDim.x)
      if (batch.seq(s).len == 0) {
        uint4 *o = reinterpret_cast<uint4 *>(static_cast<T *>(p.out) + (size_t)s * p.num_heads * D);
        for (int i = threadIdx.x; i < p.num_heads * D / 8; i += kQ4Threads) o[i] = make_uint4(0u, 0u, 0u, 0u);
      }

  // ---- the walk over the share, one tile ahead of the copies
  ShareWalk walk;
  walk.begin(batch, s_scan, line, line_end);
  bool joined = false;
  int in_piece = 0, f_flags = 0, f_tok = 0, f_end = 0, e0 = -1, e1 = -1;
  int u_rows = 0, u_row0 = 0, u_kvh = 0, u_lim = 0, u_dest = 0;
  const int32_t *table = p.block_tables;
  auto fetch = [&]() {
    if (in_piece == 0) {
      if (walk.left <= 0) {
        f_flags = kQ4End;
        return;
      }
      const int n = walk.piece(), step = walk.step;
      int rg = 0;
      u_kvh = walk.unit;
      u_rows = p.group;
      u_row0 = walk.s;
      u_lim = walk.q.len - 1;
      f_end = walk.q.len;
      if (CHUNK) {
        const int nrg = (walk.q.n + p.chunk_tokens - 1) / p.chunk_tokens;
        u_kvh = walk.unit / nrg;
        rg = walk.unit - u_kvh * nrg;
        const int t0 = rg * p.chunk_tokens, nt = min(p.chunk_tokens, walk.q.n - t0);
        u_rows = nt * p.group;
        u_row0 = walk.q.row0 + t0;
        u_lim = walk.q.len - walk.q.n + t0;
        f_end = u_lim + nt;
      }
      const bool ends = step + n == walk.q.steps;
      u_dest = step > 0 ? kQ4Place0 : ends ? kQ4Whole : kQ4Place1;
      if (u_dest == kQ4Place1 && threadIdx.x == 0) {
        ShareJoin j{};
        j.parts = share_of(total, line + walk.q.steps - 1, shares) - me + 1;
        j.rows = u_rows;
        j.group = p.group;
        j.stride = p.num_heads;
        j.out_row = (long long)u_row0 * p.num_heads + u_kvh * p.group;
        space.join[me] = j;
      }
      joined = joined || u_dest == kQ4Place1;
      table = p.block_tables + (size_t)walk.s * p.max_blocks_per_seq;
      line += n;
      in_piece = n;
      f_tok = step * kShareStep + warp * 16;
      f_flags = kQ4First;
      walk.next(batch);
    } else {
      f_tok += kShareStep;
      f_flags = 0;
    }
    if (--in_piece == 0) f_flags |= kQ4Last;
    e0 = f_tok < f_end ? __ldg(table + (f_tok >> p.log2_block_size)) : -1;
    e1 = f_tok + 8 < f_end ? __ldg(table + ((f_tok + 8) >> p.log2_block_size)) : -1;
  };
  fetch();

  // ---- one stage of copies: the fetched tile's codes and scales
  auto issue = [&](int slot) {
    const uint32_t st = ring_u32 + (uint32_t)slot * Z::STAGE;
    if (lane == 0) {
      Q4Head *h = reinterpret_cast<Q4Head *>(ring + slot * Z::STAGE + Z::HEAD);
      *reinterpret_cast<int4 *>(h) = make_int4(f_flags, max(min(f_end - f_tok, 16), 0), f_tok, u_lim);
      *(reinterpret_cast<int4 *>(h) + 1) = make_int4(u_rows, u_row0, u_kvh, u_dest);
    }
    if (!(f_flags & kQ4End)) {
      const int valid = f_end - f_tok;
      bool ok0 = valid > 0, ok1 = valid > 8;
      if ((ok0 && (unsigned)e0 >= (unsigned)p.num_blocks) || (ok1 && (unsigned)e1 >= (unsigned)p.num_blocks)) {
        report(p.status, kStatusBadInput);  // those rows are taken as zeros
        ok0 = ok0 && (unsigned)e0 < (unsigned)p.num_blocks;
        ok1 = ok1 && (unsigned)e1 < (unsigned)p.num_blocks;
      }
      // the first row's place in the cache of each half of the tile
      const size_t s0 = ok0 ? ((size_t)e0 * p.num_kv_heads + u_kvh) * p.block_size + (f_tok & (p.block_size - 1)) : 0;
      const size_t s1 =
          ok1 ? ((size_t)e1 * p.num_kv_heads + u_kvh) * p.block_size + ((f_tok + 8) & (p.block_size - 1)) : 0;
#pragma unroll
      for (int j = 0; j < (16 * CPR + 31) / 32; ++j) {
        const int i = lane + 32 * j, r = i / CPR, c = i % CPR;  // CPR 2: 32 pieces in all
        const int pl = Z::place(r);
        const uint32_t dst = st + (uint32_t)(pl * RB + (((c >> 1) ^ Z::swap(pl)) << 5) + ((c & 1) << 4));
        const size_t src = (r < 8 ? s0 : s1) * RB + (size_t)((r & 7) * RB + c * 16);
        const uint32_t n = (r < 8 ? ok0 : ok1) && r < valid ? 16u : 0u;
        const size_t from = n ? src : 0;
        cp_async16(dst + Z::KEYS, p.key_codes + from, n);
        cp_async16(dst + Z::VALUES, p.value_codes + from, n);
      }
      {
        const int r = lane & 15;
        const uint32_t n = (r < 8 ? ok0 : ok1) && r < valid ? 4u * NG : 0u;
        const size_t src = n ? ((r < 8 ? s0 : s1) + (size_t)(r & 7)) * (4 * NG) : 0;
        const void *from = (lane < 16 ? static_cast<const uint8_t *>(p.key_scales)
                                      : static_cast<const uint8_t *>(p.value_scales)) + src;
        const uint32_t dst = st + (lane < 16 ? Z::KSC : Z::VSC) + r * 4 * NG;
        cp_async_small<4 * NG>(dst, from, n);
      }
      fetch();
    }
    cp_async_commit();
  };

#pragma unroll
  for (int i = 0; i < NST - 1; ++i) issue(i);

  // ---- the tiles
  uint32_t qf[NT][KW][2];      // Q^T fragments, in the keys' order of elements
  float qsum[NT][NG][2];       // scale_log2 x the sum of the group's q, of this lane's columns
  float o[NT][KW][4];          // O^T: rows 64 gr + 8 g + 2 mt (+ 1), columns 2t, 2t + 1
  float sa[NT][NG][2], sb[NT][NG][2], m[NT][2];
  int lim[CHUNK ? NT : 1][2];

  for (int slot = 0;; slot = slot + 1 == NST ? 0 : slot + 1) {
    cp_async_wait<NST - 2>();
    __syncwarp();
    uint8_t *stage = ring + slot * Z::STAGE;
    const Q4Head h = *reinterpret_cast<const Q4Head *>(stage + Z::HEAD);
    if (h.flags & kQ4End) break;
    issue(slot == 0 ? NST - 1 : slot - 1);

    if (h.flags & kQ4First) {
      // queries: lane (g, t) has elements 16 t .. 16 t + 15 of each group of column g
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int c = nt * 8 + g;
        const bool live = c < h.rows;
        const size_t row = (size_t)(h.row0 + c / p.group) * p.num_heads + (size_t)(h.kvh * p.group + c % p.group);
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.query) + (live ? row : 0) * D) + 2 * t;
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
          if (live) {
            a = __ldg(src + gr * 8);
            b = __ldg(src + gr * 8 + 1);
          }
          const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 f = MmaOp<T>::unpack(w[i]);
            sum += f.x + f.y;
          }
          // k-step 4 gr + 2 wi + h2: codes 2 h2, 2 h2 + 4 | 2 h2 + 1, 2 h2 + 5 of word wi
#pragma unroll
          for (int wi = 0; wi < 2; ++wi)
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
              qf[nt][4 * gr + 2 * wi + h2][0] = prmt(w[4 * wi + h2], w[4 * wi + h2 + 2], 0x5410);
              qf[nt][4 * gr + 2 * wi + h2][1] = prmt(w[4 * wi + h2], w[4 * wi + h2 + 2], 0x7632);
            }
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          qsum[nt][gr][0] = __shfl_sync(0xffffffffu, sum, 8 * t) * p.scale_log2;
          qsum[nt][gr][1] = __shfl_sync(0xffffffffu, sum, 8 * t + 4) * p.scale_log2;
          sa[nt][gr][0] = sa[nt][gr][1] = sb[nt][gr][0] = sb[nt][gr][1] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < KW; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][i][e] = 0.f;
        m[nt][0] = m[nt][1] = -CUDART_INF_F;
        if (CHUNK)
#pragma unroll
          for (int e = 0; e < 2; ++e) lim[nt][e] = h.lim_base + (nt * 8 + 2 * t + e) / p.group + 1;
      }
    }

    if (h.valid > 0) {
      // ---- scores: x = scale_log2 q . K of tokens g, g + 8 and columns 2t, 2t + 1
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nt][e] = 0.f;
      const int pa0 = Z::place(g);  // rows g and g + 8: places pa0, pa0 + 8, swapped alike
      const uint8_t *krow = stage + Z::KEYS + pa0 * RB;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        const int off = ((gr ^ Z::swap(pa0)) << 5) + 8 * t;
        const uint2 wa = *reinterpret_cast<const uint2 *>(krow + off);
        const uint2 wb = *reinterpret_cast<const uint2 *>(krow + 8 * RB + off);
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nt][e] = 0.f;
#pragma unroll
        for (int wi = 0; wi < 2; ++wi) {
          const uint32_t a = wi ? wa.y : wa.x, b = wi ? wb.y : wb.x;
          const uint32_t a0 = code_pair<T, 0>(a), a1 = code_pair<T, 1>(a), a2 = code_pair<T, 2>(a), a3 = code_pair<T, 3>(a);
          const uint32_t b0 = code_pair<T, 0>(b), b1 = code_pair<T, 1>(b), b2 = code_pair<T, 2>(b), b3 = code_pair<T, 3>(b);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int ks = 4 * gr + 2 * wi;
            MmaOp<T>::run(acc[nt], a0, b0, a1, b1, qf[nt][ks][0], qf[nt][ks][1]);
            MmaOp<T>::run(acc[nt], a2, b2, a3, b3, qf[nt][ks + 1][0], qf[nt][ks + 1][1]);
          }
        }
        const float2 za = __half22float2(*reinterpret_cast<const __half2 *>(stage + Z::KSC + (g * NG + gr) * 4));
        const float2 zb = __half22float2(*reinterpret_cast<const __half2 *>(stage + Z::KSC + ((g + 8) * NG + gr) * 4));
        const float la = fmaf(-16.f, za.y, za.x), lb = fmaf(-16.f, zb.y, zb.x);
        const float ta = za.y * p.scale_log2, tb = zb.y * p.scale_log2;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          x[nt][0] = fmaf(ta, acc[nt][0], fmaf(la, qsum[nt][gr][0], x[nt][0]));
          x[nt][1] = fmaf(ta, acc[nt][1], fmaf(la, qsum[nt][gr][1], x[nt][1]));
          x[nt][2] = fmaf(tb, acc[nt][2], fmaf(lb, qsum[nt][gr][0], x[nt][2]));
          x[nt][3] = fmaf(tb, acc[nt][3], fmaf(lb, qsum[nt][gr][1], x[nt][3]));
        }
      }
      // ---- the running maximum, raised when a score is 2^8 above it: any
      // reference serves the sums as long as nothing overflows
      bool up = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (h.valid < 16) {
          if (g >= h.valid) x[nt][0] = x[nt][1] = -CUDART_INF_F;
          if (g + 8 >= h.valid) x[nt][2] = x[nt][3] = -CUDART_INF_F;
        }
        if (CHUNK) {
          if (h.tok0 + g >= lim[nt][0]) x[nt][0] = -CUDART_INF_F;
          if (h.tok0 + g >= lim[nt][1]) x[nt][1] = -CUDART_INF_F;
          if (h.tok0 + g + 8 >= lim[nt][0]) x[nt][2] = -CUDART_INF_F;
          if (h.tok0 + g + 8 >= lim[nt][1]) x[nt][3] = -CUDART_INF_F;
        }
        up = up || fmaxf(x[nt][0], x[nt][2]) > m[nt][0] + kQ4Margin || fmaxf(x[nt][1], x[nt][3]) > m[nt][1] + kQ4Margin;
      }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float t0 = fmaxf(x[nt][0], x[nt][2]), t1 = fmaxf(x[nt][1], x[nt][3]);
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) {
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
          }
          t0 = fmaxf(t0, m[nt][0]), t1 = fmaxf(t1, m[nt][1]);
          const float f0 = t0 == -CUDART_INF_F ? 1.f : exp2f(m[nt][0] - t0);
          const float f1 = t1 == -CUDART_INF_F ? 1.f : exp2f(m[nt][1] - t1);
          m[nt][0] = t0, m[nt][1] = t1;
#pragma unroll
          for (int i = 0; i < KW; ++i) {
            o[nt][i][0] *= f0, o[nt][i][1] *= f1;
            o[nt][i][2] *= f0, o[nt][i][3] *= f1;
          }
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            sa[nt][gr][0] *= f0, sa[nt][gr][1] *= f1;
            sb[nt][gr][0] *= f0, sb[nt][gr][1] *= f1;
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float m0 = m[nt][0] == -CUDART_INF_F ? 0.f : m[nt][0];
        const float m1 = m[nt][1] == -CUDART_INF_F ? 0.f : m[nt][1];
        x[nt][0] = ex2f(x[nt][0] - m0), x[nt][1] = ex2f(x[nt][1] - m1);
        x[nt][2] = ex2f(x[nt][2] - m0), x[nt][3] = ex2f(x[nt][3] - m1);
      }
      // ---- O^T += V^T P^T, group by group: a lane's word g of tokens 2t, 2t + 1
      // (places t, t + 4) and of the eight behind
      const uint8_t *vrow = stage + Z::VALUES + t * RB;
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        const float2 za = __half22float2(*reinterpret_cast<const __half2 *>(stage + Z::VSC + (g * NG + gr) * 4));
        const float2 zb = __half22float2(*reinterpret_cast<const __half2 *>(stage + Z::VSC + ((g + 8) * NG + gr) * 4));
        const float ta = fmaxf(za.y, kQ4LeastStep), tb = fmaxf(zb.y, kQ4LeastStep);
        const float ra = __frcp_rn(ta), rb = __frcp_rn(tb);
        const float ba = fmaf(za.x, ra, -16.f), bb = fmaf(zb.x, rb, -16.f);
        uint32_t pf[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t lo = MmaOp<__nv_bfloat16>::pack(x[nt][0] * ta, x[nt][1] * ta);
          const uint32_t hi = MmaOp<__nv_bfloat16>::pack(x[nt][2] * tb, x[nt][3] * tb);
          const float2 wl = MmaOp<__nv_bfloat16>::unpack(lo), wh = MmaOp<__nv_bfloat16>::unpack(hi);
          sa[nt][gr][0] = fmaf(wl.x, ra, fmaf(wh.x, rb, sa[nt][gr][0]));
          sa[nt][gr][1] = fmaf(wl.y, ra, fmaf(wh.y, rb, sa[nt][gr][1]));
          sb[nt][gr][0] = fmaf(wl.x, ba, fmaf(wh.x, bb, sb[nt][gr][0]));
          sb[nt][gr][1] = fmaf(wl.y, ba, fmaf(wh.y, bb, sb[nt][gr][1]));
          pf[nt][0] = movmatrix_trans(lo);
          pf[nt][1] = movmatrix_trans(hi);
        }
        const int off = ((gr ^ Z::swap(t)) << 5) + 4 * g, off4 = ((gr ^ Z::swap(t + 4)) << 5) + 4 * g;
        const uint32_t w0 = *reinterpret_cast<const uint32_t *>(vrow + off);
        const uint32_t w1 = *reinterpret_cast<const uint32_t *>(vrow + 4 * RB + off4);
        const uint32_t w2 = *reinterpret_cast<const uint32_t *>(vrow + 8 * RB + off);
        const uint32_t w3 = *reinterpret_cast<const uint32_t *>(vrow + 12 * RB + off4);
        using B = __nv_bfloat16;
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // codes 0 .. 3, then 4 .. 7 of the word
          const uint32_t sel = half ? 0x7632 : 0x5410;
          const uint32_t a = prmt(w0, w1, sel), b = prmt(w2, w3, sel);
          // halves of a: codes 4 half .. + 3 of tokens 2t and 2t + 1, so pair I is code I of both
          const uint32_t a0 = code_pair<B, 0>(a), a1 = code_pair<B, 1>(a), a2 = code_pair<B, 2>(a), a3 = code_pair<B, 3>(a);
          const uint32_t b0 = code_pair<B, 0>(b), b1 = code_pair<B, 1>(b), b2 = code_pair<B, 2>(b), b3 = code_pair<B, 3>(b);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            MmaOp<B>::run(o[nt][4 * gr + 2 * half], a0, a1, b0, b1, pf[nt][0], pf[nt][1]);
            MmaOp<B>::run(o[nt][4 * gr + 2 * half + 1], a2, a3, b2, b3, pf[nt][0], pf[nt][1]);
          }
        }
      }
    }

    if (h.flags & kQ4Last) {
      // ---- the four warps' sums of this piece become one
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int gr = 0; gr < NG; ++gr)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              sa[nt][gr][e] += __shfl_xor_sync(0xffffffffu, sa[nt][gr][e], d);
              sb[nt][gr][e] += __shfl_xor_sync(0xffffffffu, sb[nt][gr][e], d);
            }
        if (g == 0) {
          s_m[warp][nt * 8 + 2 * t] = m[nt][0];
          s_m[warp][nt * 8 + 2 * t + 1] = m[nt][1];
        }
      }
      __syncthreads();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float f[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = nt * 8 + 2 * t + e;
          const float top = fmaxf(fmaxf(s_m[0][c], s_m[1][c]), fmaxf(s_m[2][c], s_m[3][c]));
          f[e] = m[nt][e] == -CUDART_INF_F ? 0.f : exp2f(m[nt][e] - top);
          if (g == 0) {
            if (warp == 0) s_top[c] = top;
#pragma unroll
            for (int gr = 0; gr < NG; ++gr) s_sum[warp][c][gr] = make_float2(sa[nt][gr][e] * f[e], sb[nt][gr][e] * f[e]);
          }
        }
#pragma unroll
        for (int i = 0; i < KW; ++i) {
          o[nt][i][0] *= f[0], o[nt][i][1] *= f[1];
          o[nt][i][2] *= f[0], o[nt][i][3] *= f[1];
        }
      }
      // warps 2 and 3 put theirs down, 0 and 1 add their own on top
      float *ob = obuf + (warp & 1) * (GM * Z::OROW);
#pragma unroll
      for (int turn = 0; turn < 2; ++turn) {
        if ((warp >> 1) != turn) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int gr = 0; gr < NG; ++gr)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                // rows 64 gr + 8 g + 0 .. 7 of column 8 nt + 2 t + e
                float4 *dst = reinterpret_cast<float4 *>(ob + (nt * 8 + 2 * t + e) * Z::OROW + 64 * gr + 8 * g);
                float4 a = make_float4(o[nt][4 * gr][e], o[nt][4 * gr][e + 2], o[nt][4 * gr + 1][e], o[nt][4 * gr + 1][e + 2]);
                float4 b = make_float4(o[nt][4 * gr + 2][e], o[nt][4 * gr + 2][e + 2], o[nt][4 * gr + 3][e], o[nt][4 * gr + 3][e + 2]);
                if (turn == 1) {
                  const float4 c = dst[0], d = dst[1];
                  a.x += c.x, a.y += c.y, a.z += c.z, a.w += c.w;
                  b.x += d.x, b.y += d.y, b.z += d.z, b.w += d.w;
                }
                dst[0] = a;
                dst[1] = b;
              }
        }
        __syncthreads();
      }
      // rows out, a warp a row, a lane four columns of every 128
      for (int c = warp; c < h.rows; c += kQ4Warps) {
        const float top = s_top[c];
        const float s0 = (s_sum[0][c][0].x + s_sum[1][c][0].x) + (s_sum[2][c][0].x + s_sum[3][c][0].x);
        const size_t place = (2 * (size_t)me + (h.dest == kQ4Place1 ? 1 : 0)) * 16 + c;
        if (h.dest != kQ4Whole && lane == 0) space.ml[place] = make_float2(top, s0);
#pragma unroll
        for (int d = lane * 4; d < D; d += 128) {
          const int gr = d >> 6;
          const float a = (s_sum[0][c][gr].x + s_sum[1][c][gr].x) + (s_sum[2][c][gr].x + s_sum[3][c][gr].x);
          const float b = (s_sum[0][c][gr].y + s_sum[1][c][gr].y) + (s_sum[2][c][gr].y + s_sum[3][c][gr].y);
          const float4 u = *reinterpret_cast<const float4 *>(obuf + c * Z::OROW + d);
          const float4 v = *reinterpret_cast<const float4 *>(obuf + (GM + c) * Z::OROW + d);
          // (groups round their weights apart: a piece's outputs take its first
          // group's sum as theirs)
          const float inv = a > 0.f ? (h.dest == kQ4Whole ? 1.f / a : s0 / a) : (a == 0.f ? 0.f : a);
          const float r0 = (u.x + v.x + b) * inv, r1 = (u.y + v.y + b) * inv;
          const float r2 = (u.z + v.z + b) * inv, r3 = (u.w + v.w + b) * inv;
          if (h.dest == kQ4Whole) {
            const size_t row = (size_t)(h.row0 + c / p.group) * p.num_heads + (size_t)(h.kvh * p.group + c % p.group);
            store4(static_cast<T *>(p.out) + row * D + d, r0, r1, r2, r3);
          } else {
            *reinterpret_cast<float4 *>(space.o + place * D + d) = make_float4(r0, r1, r2, r3);
          }
        }
      }
    }
  }
  if (!joined && threadIdx.x == 0) space.join[me].parts = 0;
  pdl_launch_dependents();
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
  return pa::share_bytes(16, head_size, nullptr, nullptr);
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
  st = host_ensure_smem(k.fn, k.smem);
  if (st != PA_OK) return st;
  const int ctas = sms * k.ctas < kShareMaxCtas ? sms * k.ctas : kShareMaxCtas;
  ShareSpace space;
  share_bytes(16, head_size, workspace, &space);
  void *args[2] = {&p, &space};
  st = host_launch(k.fn, (unsigned)ctas, 1, kQ4Threads, k.smem, stream, args, "launch 4-bit attention kernel");
  if (st != PA_OK) return st;
  JoinParams j{};
  j.space = space;
  j.out = out;
  j.ctas = ctas;
  j.place_step = 1;
  j.max_rows = 16;
  j.width = head_size;
  void *jargs[1] = {&j};
  return host_launch(share_join_kernel(dtype == PA_DTYPE_BF16), (unsigned)(2 * sms), 1, kJoinThreads, 0, stream,
                     jargs, "launch join kernel");
}

}  // extern "C"
