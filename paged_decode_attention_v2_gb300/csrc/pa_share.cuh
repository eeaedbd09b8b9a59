// Attention cut into shares of work: each worker (a warp, a CTA) of a grid that
// fills the GPU once takes shares of the batch's keys, in steps, one after
// another, and a second kernel joins the units that ended up in several shares.
//
// A unit is what one item of rows reads: a sequence's keys, for one KV head
// and one group of query rows.  The steps of all units stand in one line, unit
// behind unit, and a share is a stretch of the line, whatever units it cuts.
// Every worker has a large share first, all equal; where pieces are cheap and
// there is work enough, the rest of the line is cut into small ones that the
// workers take from a counter as they get done, since SMs do not run alike (with
// equal shares alone, CTAs of the same work ended between 50 and 76 us).  A share
// has at most two units that it does not hold whole, its first and its last, so
// the space for partial results is two places a share, whatever the batch.  Every
// CTA works the shares out of the
// lengths by itself: a scan over the sequences, which all CTAs do at once,
// instead of a launch that would plan.
//
// To begin and end a unit takes as long as a few of its steps, so a unit stands
// in the line with a head of that many steps before its own.  (Without heads, a
// warp whose share held eight short sequences ended 15 us after the rest: 64
// sequences of 16 to 32768 keys took 51 us, with heads of three steps 41.)
#pragma once

#include <math_constants.h>

#include "pa.h"
#include "pa_device.cuh"

namespace pa {

// A workspace, behind its status block: the units to join, then the places'
// (reference, sum) a row and their unnormalised outputs; 256-byte aligned each.
// Ints of the status block: shares taken, units to join of few and of many
// pieces, join CTAs done.
constexpr int kShareTaken = 16, kShareFew = 17, kShareMany = 18, kShareDone = 19;
constexpr int kJoinFew = 64; // pieces that one warp joins by itself

// A unit whose keys lie in several shares: parts pieces (place 1 of `share`,
// then place 0 of the next shares, `by` apart), each of `rows` rows.  Row r
// goes to out row out_row + (r / group) * stride + r % group.
struct alignas(16) ShareJoin {
  int share, parts, by, rows;
  int group, stride;
  long long out_row;
};

struct ShareSpace {
  ShareJoin *join;  // [shares]: units of few pieces from the front, of many from the back
  // m: what the weights are relative to, log2 units (any that keeps them in range)
  float2 *ml;       // [shares][2][rows]: m, sum of exp2(x - m)
  float *o;         // [shares][2][rows][width]: sum of exp2(x - m) v
  int *counters;    // the status block
  int shares;
};
// (shares: a multiple of 64)
inline size_t share_bytes(int shares, int rows, int width, void *base, ShareSpace *s) {
  const size_t joins = (size_t)shares * sizeof(ShareJoin);
  const size_t ml = (size_t)shares * 2 * rows * sizeof(float2);
  const size_t o = (size_t)shares * 2 * rows * width * sizeof(float);
  if (s) {
    char *at = static_cast<char *>(base) + kStatusBytes;
    s->join = reinterpret_cast<ShareJoin *>(at);
    s->ml = reinterpret_cast<float2 *>(at + joins);
    s->o = reinterpret_cast<float *>(at + joins + ml);
    s->counters = static_cast<int *>(base);
    s->shares = shares;
  }
  return kStatusBytes + joins + ml + o;
}

// a / b of numbers >= 0, in 32 bits where they fit (a tenth of the instructions)
__device__ __forceinline__ long long div_steps(long long a, long long b) {
  return ((unsigned long long)(a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// The shares of a line of `total` steps: `big` equal ones over its first
// big_total steps, `small` equal ones over the rest (alone: large ones alone).
constexpr int kShareSmall = 1;     // small shares for each large one,
constexpr int kShareSmallPct = 35; // over this much of the line,
constexpr int kShareTwo = 24;      // where there are this many steps a worker
constexpr int kShareLeast = 2;     // steps of a share where there are not enough for all
struct SharePlan {
  long long total, big_total;
  int big, small;
  __device__ __forceinline__ void make(long long steps, int workers, bool alone = false) {
    total = big_total = steps;
    const long long most = (steps + kShareLeast - 1) / kShareLeast;
    big = most < workers ? (int)most : workers;
    small = 0;
    if (!alone && steps >= (long long)workers * kShareTwo) {
      small = kShareSmall * workers;
      big_total = div_steps(steps, 100) * (100 - kShareSmallPct);
    }
  }
  // the first step of share i
  __device__ __forceinline__ long long begin(int i) const {
    if (i >= big + small) return total;
    if (i < big) return div_steps(big_total * i, big);
    return big_total + div_steps((total - big_total) * (i - big), small);
  }
  // the share that step x (< total) is in
  __device__ __forceinline__ int of(long long x) const {
    int i = x < big_total ? (int)div_steps(x * big, big_total)
                          : big + (int)div_steps((x - big_total) * small, total - big_total);
    i = min(i, big + small - 1);
    while (i > 0 && begin(i) > x) --i;
    while (begin(i + 1) <= x) ++i;
    return i;
  }
};

// A sequence as the plan sees it.
struct ShareSeq {
  int len;    // its keys
  int row0;   // its first query row
  int n;      // its query rows (tokens)
  int units;  // 0: nothing to do for it
  int steps;  // of a unit
  int head;   // what it costs to begin and end one, in steps: stands before its steps in the line
};

// The batch's side of the plan: Batch has num_seqs; read(s), a sequence's
// (len, row0, n), checked, no keys and no rows if it is bad; seq(int4), the ShareSeq
// of it.
template <int THREADS_, int CACHE_>
struct ShareScan {
  static constexpr int THREADS = THREADS_, CACHE = CACHE_;  // CACHE: sequences kept in shared memory
  long long cum[THREADS + 1];  // the line before each thread's sequences
  long long warp_sum[THREADS / 32];
  int4 cache[CACHE];
};

template <class Scan, class Batch>
__device__ __forceinline__ ShareSeq share_seq(const Batch &b, const Scan &scan, int s) {
  return b.seq(b.num_seqs <= Scan::CACHE ? scan.cache[s] : b.read(s));
}

// By THREADS threads (the first of the CTA), with all of the CTA's threads at
// the barriers: fills the scan.
template <class Scan, class Batch>
__device__ __forceinline__ void share_scan(const Batch &b, Scan &scan) {
  constexpr int THREADS = Scan::THREADS;
  const int t = threadIdx.x, per = (b.num_seqs + THREADS - 1) / THREADS;
  long long own = 0;
  if (t < THREADS) {
    for (int s = t * per; s < min(b.num_seqs, (t + 1) * per); ++s) {
      const int4 r = b.read(s);
      if (b.num_seqs <= Scan::CACHE) scan.cache[s] = r;
      const ShareSeq q = b.seq(r);
      own += (long long)q.units * (q.head + q.steps);
    }
  }
  long long incl = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, d);
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

// A walk over the pieces of units in a share.
struct ShareWalk {
  long long line;  // where the walk is
  long long left;  // steps of the share from here on
  int s;           // sequence
  ShareSeq q;
  int unit, at;    // of the sequence, of the unit (its head, then its steps)

  template <class Scan, class Batch>
  __device__ __forceinline__ void begin(const Batch &b, const Scan &scan, long long from, long long end) {
    constexpr int THREADS = Scan::THREADS;
    line = from;
    left = end - from;
    if (left <= 0) return;
    int lo = 0, hi = THREADS - 1;  // the last thread whose sequences start at or before it
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (scan.cum[mid] <= from)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int per = (b.num_seqs + THREADS - 1) / THREADS;
    long long x = from - scan.cum[lo];
    s = lo * per;
    while (true) {
      q = share_seq(b, scan, s);
      const long long n = (long long)q.units * (q.head + q.steps);
      if (x < n) break;
      x -= n;
      if (++s >= b.num_seqs) {  // (lengths that change under the call: stop)
        left = 0;
        return;
      }
    }
    unit = (int)div_steps(x, q.head + q.steps);
    at = (int)(x - (long long)unit * (q.head + q.steps));
    if (at + left <= q.head) left = 0;  // (a share that ends in a head has none of the unit)
  }
  // this piece: its first step, how many, the place of the unit's last in the line
  __device__ __forceinline__ int first() const { return max(at - q.head, 0); }
  __device__ __forceinline__ int steps() const {
    return (int)min(left + at - q.head, (long long)q.steps) - first();
  }
  __device__ __forceinline__ long long last() const { return line - at + q.head + q.steps - 1; }
  // on to the next piece
  template <class Scan, class Batch>
  __device__ __forceinline__ void next(const Batch &b, const Scan &scan) {
    const int n = (int)min(left, (long long)(q.head + q.steps - at));
    line += n;
    left -= n;
    if (left <= 0) return;  // (else the unit is done)
    at = 0;
    if (++unit == q.units) {
      unit = 0;
      do {
        if (++s >= b.num_seqs) {
          left = 0;
          return;
        }
        q = share_seq(b, scan, s);
      } while (q.units == 0);
    }
    if (left <= q.head) left = 0;
  }
};

// Notes a unit to join (by one thread).
__device__ __forceinline__ void share_join(const ShareSpace &space, const ShareJoin &j) {
  if (j.parts <= kJoinFew)
    space.join[atomicAdd(space.counters + kShareFew, 1)] = j;
  else
    space.join[space.shares - 1 - atomicAdd(space.counters + kShareMany, 1)] = j;
}

// Joins the units that lie in several shares:
//   out = sum_k 2^(m_k - M) o_k / sum_k 2^(m_k - M) l_k,  M = max_k m_k
// over the pieces k in their order.
struct JoinParams {
  ShareSpace space;
  void *out;  // [..][width], rows as the ShareJoins say
  int max_rows, item_rows, width;  // rows of a place, of the largest unit
};
// Launches the join behind an attention kernel.  If that fails, the counters, which
// the join would have reset, are cleared: the next call would take them for its own.
pa_status_t share_launch_join(const JoinParams &p, int dtype_bf16, int sms, void *stream);

}  // namespace pa
