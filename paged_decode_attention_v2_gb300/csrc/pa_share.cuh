// Attention split into equal shares of work: every CTA (or pair of CTAs) of a
// grid that fits the GPU takes the same number of steps of 64 keys, one after
// another through the batch's units, and a second kernel joins the units that
// ended up in several shares.
//
// A unit is what one item of rows reads: a sequence's keys, for one KV head
// and one group of query rows.  The steps of all units stand in one line, unit
// behind unit; share w of W is steps [w T / W, (w + 1) T / W) of the T.  So
// each share's work is equal to a step whatever the lengths are, a share has
// at most two units that it does not hold whole (its first and its last), and
// the space for partial results is two places a share, whatever the batch.
// Every CTA works its share out of the lengths by itself: a scan over the
// sequences, which all CTAs do at once, instead of a launch that would plan.
#pragma once

#include <math_constants.h>

#include "pa_device.cuh"

namespace pa {

constexpr int kShareStep = 64;         // keys of a step
constexpr int kShareMaxCtas = 8 * 152; // places for partial results in a workspace

// What a CTA leaves for the join of the unit that its share ends inside of:
// parts pieces (its own place 1, then place 0 of the next shares), each of
// `rows` rows.  Row r goes to out row out_row + (r / group) * stride + r % group.
struct ShareJoin {
  int parts;  // 0: nothing to join
  int rows;
  int group, stride;
  long long out_row;
  int pad[2];
};

// Layout of a workspace: the status block, the ShareJoins, the pieces' (maximum,
// sum) a row, their unnormalised outputs; 256-byte aligned each.
struct ShareSpace {
  ShareJoin *join;  // [ctas]
  float2 *ml;       // [ctas][2][rows]: maximum (log2 units), sum of exp2(x - maximum)
  float *o;         // [ctas][2][rows][width]: sum of exp2(x - maximum) v
};
__host__ inline size_t share_bytes(int rows, int width, void *base, ShareSpace *s) {
  const size_t joins = (size_t)kShareMaxCtas * sizeof(ShareJoin);
  const size_t ml = (size_t)kShareMaxCtas * 2 * rows * sizeof(float2);
  const size_t o = (size_t)kShareMaxCtas * 2 * rows * width * sizeof(float);
  size_t at = kStatusBytes;
  if (s) {
    s->join = reinterpret_cast<ShareJoin *>(static_cast<char *>(base) + at);
    s->ml = reinterpret_cast<float2 *>(static_cast<char *>(base) + at + joins);
    s->o = reinterpret_cast<float *>(static_cast<char *>(base) + at + joins + ml);
  }
  return at + joins + ml + o;  // (each a multiple of 256: kShareMaxCtas is one of 64)
}

// A sequence as the plan sees it.
struct ShareSeq {
  int len;    // its keys
  int row0;   // its first query row
  int n;      // its query rows (tokens)
  int units;  // 0: nothing to do for it
  int steps;  // of a unit
};

// The batch's side of the plan: Batch has seq(s), a ShareSeq with units and
// steps set, and num_seqs.
template <int THREADS>
struct ShareScan {
  long long cum[THREADS + 1];  // steps before each thread's sequences
  long long warp_sum[THREADS / 32];
};

__device__ __forceinline__ long long shfl_up64(long long v, int d) {
  return __shfl_up_sync(0xffffffffu, v, d);
}

// By THREADS threads (the first of the CTA), with all of the CTA's threads at
// the barriers: fills scan.cum.
template <int THREADS, class Batch>
__device__ __forceinline__ void share_scan(const Batch &b, ShareScan<THREADS> &scan) {
  const int t = threadIdx.x, per = (b.num_seqs + THREADS - 1) / THREADS;
  long long own = 0;
  if (t < THREADS) {
    for (int s = t * per; s < min(b.num_seqs, (t + 1) * per); ++s) {
      const ShareSeq q = b.seq(s);
      own += (long long)q.units * q.steps;
    }
  }
  long long incl = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = shfl_up64(incl, d);
    if ((t & 31) >= d) incl += o;
  }
  if (t < THREADS && (t & 31) == 31) scan.warp_sum[t >> 5] = incl;
  __syncthreads();
  if (t < THREADS) {
    long long before = 0;
    for (int w = 0; w < (t >> 5); ++w) before += scan.warp_sum[w];
    scan.cum[t] = before + incl - own;
    if (t == THREADS - 1) scan.cum[THREADS] = before + incl;
  }
  __syncthreads();
}

// Share w of W of T steps: its first step.
__device__ __forceinline__ long long share_begin(long long T, int w, int W) { return T * w / W; }

// The share that step x (< T) is in.
__device__ __forceinline__ int share_of(long long T, long long x, int W) {
  int w = (int)min((long long)W - 1, x * W / T);
  while (w > 0 && share_begin(T, w, W) > x) --w;
  while (w < W - 1 && share_begin(T, w + 1, W) <= x) ++w;
  return w;
}

// The shares of a plan: no more than there are, and none with less than `least`
// steps where there could be fewer.
__device__ __forceinline__ int share_count(long long T, int most, int least) {
  const long long w = (T + least - 1) / least;
  return w < 1 ? 1 : w < most ? (int)w : most;
}

// A walk over the pieces of units in steps [at, end) of the line.
struct ShareWalk {
  long long left;  // steps of the share from here on
  int s;           // sequence
  ShareSeq q;
  int unit, step;  // of the sequence, of the unit

  template <int THREADS, class Batch>
  __device__ __forceinline__ void begin(const Batch &b, const ShareScan<THREADS> &scan, long long at,
                                        long long end) {
    left = end - at;
    s = b.num_seqs;
    if (left <= 0) return;
    int lo = 0, hi = THREADS - 1;  // the last thread whose sequences start at or before it
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (scan.cum[mid] <= at)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int per = (b.num_seqs + THREADS - 1) / THREADS;
    long long x = at - scan.cum[lo];
    s = lo * per;
    while (true) {
      q = b.seq(s);
      const long long n = (long long)q.units * q.steps;
      if (x < n) break;
      x -= n;
      if (++s >= b.num_seqs) {  // (lengths that change under the call: stop)
        left = 0;
        return;
      }
    }
    unit = (int)(x / q.steps);
    step = (int)(x - (long long)unit * q.steps);
  }
  // steps of this piece
  __device__ __forceinline__ int piece() const {
    return (int)min(left, (long long)(q.steps - step));
  }
  // on to the next piece
  template <class Batch>
  __device__ __forceinline__ void next(const Batch &b) {
    const int n = piece();
    left -= n;
    step += n;
    if (left <= 0 || step < q.steps) return;
    step = 0;
    if (++unit < q.units) return;
    unit = 0;
    do {
      if (++s >= b.num_seqs) {
        left = 0;
        return;
      }
      q = b.seq(s);
    } while (q.units == 0);
  }
};

// Joins the units that lie in several shares:
//   out = sum_k 2^(m_k - M) o_k / sum_k 2^(m_k - M) l_k,  M = max_k m_k
// over the pieces k in their order.  A unit of few pieces is a warp's work a
// row and 128 columns; one of many pieces is a CTA's, whose warps take pieces
// in turn.
struct JoinParams {
  ShareSpace space;
  void *out;       // [..][width], rows as the ShareJoins say
  int ctas;        // of the attention kernel
  int place_step;  // CTAs between a unit's pieces (2: pairs take a unit each)
  int max_rows, width;
};

const void *share_join_kernel(int dtype_bf16);
constexpr int kJoinThreads = 256;

}  // namespace pa
