// The join of attention that was cut into shares (pa_share.cuh).
//
// A unit of few pieces is a warp's work a row (or 128 columns of it); one of many
// is a CTA's a row and 32 columns, so that hundreds of pieces are a few loads
// deep.  Bound: the launch and a chain of three loads (how many units, the unit,
// its pieces); the bytes are a few MB that the attention kernel left in L2.  It
// adds 4 us to 8 us; four pieces at once in a warp took no less, and 16 instead
// of 64 as the most of few took 35 us instead of 32 in all for drafts.  Three CTAs
// an SM leave a thread 80 registers: 40 to 64 bytes of spills are loaded again.
#include "pa_share.cuh"

#include "pa_host.h"

namespace pa {

namespace {

constexpr int kJoinThreads = 256, kJoinCtas = 3;  // CTAs: an SM's
constexpr int kJoinWarps = kJoinThreads / 32;

// Sums over a row's pieces of four columns in each of C stretches of 128.
template <int C>
struct JoinSum {
  float m, l;
  float4 o[C];
};
template <int C>
__device__ __forceinline__ void join_scale(JoinSum<C> &a, float m) {
  const float f = exp2f(a.m - m);
  a.l *= f;
#pragma unroll
  for (int c = 0; c < C; ++c) a.o[c].x *= f, a.o[c].y *= f, a.o[c].z *= f, a.o[c].w *= f;
  a.m = m;
}
__device__ __forceinline__ void join_add(float4 &a, float f, const float4 &o) {
  a.x += o.x * f, a.y += o.y * f, a.z += o.z * f, a.w += o.w * f;
}
// A sum joins another.
__device__ __forceinline__ void join_sum(JoinSum<1> &a, const JoinSum<1> &b) {
  const float m = fmaxf(a.m, b.m), f = exp2f(b.m - m);
  join_scale(a, m);
  a.l += b.l * f;
  join_add(a.o[0], f, b.o[0]);
}
__device__ __forceinline__ ShareJoin load_join(const ShareJoin *at) {
  const int4 a = __ldcg(reinterpret_cast<const int4 *>(at)), b = __ldcg(reinterpret_cast<const int4 *>(at) + 1);
  ShareJoin j;
  j.share = a.x, j.parts = a.y, j.by = a.z, j.rows = a.w;
  j.group = b.x, j.stride = b.y;
  j.out_row = (long long)((unsigned long long)(uint32_t)b.w << 32 | (uint32_t)b.z);
  return j;
}

// The pieces k = first, first + by, ... of a row's columns col .. + 3 (of each
// stretch of 128), eight loads in flight.
template <int C>
__device__ __forceinline__ void join_pieces(const JoinParams &p, const ShareJoin &j, int row, int col,
                                            int first, int by, JoinSum<C> &a) {
  constexpr int U = 8 / C;
  a.m = -3.402823466e38f;
  a.l = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) a.o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = first; k0 < j.parts; k0 += by * U) {
    float2 ml[U];
    float4 v[U][C];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = k0 + i * by;
      ml[i] = make_float2(a.m, 0.f);
#pragma unroll
      for (int c = 0; c < C; ++c) v[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < j.parts) {
        const size_t place = k == 0 ? 2 * (size_t)j.share + 1 : 2 * ((size_t)j.share + (size_t)k * j.by);
        const size_t at = place * p.max_rows + row;
        ml[i] = __ldcg(p.space.ml + at);
#pragma unroll
        for (int c = 0; c < C; ++c)
          v[i][c] = __ldcg(reinterpret_cast<const float4 *>(p.space.o + at * p.width + col + 128 * c));
      }
    }
    float m = a.m;
#pragma unroll
    for (int i = 0; i < U; ++i) m = fmaxf(m, ml[i].x);
    join_scale(a, m);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const float f = exp2f(ml[i].x - m);
      a.l += ml[i].y * f;
#pragma unroll
      for (int c = 0; c < C; ++c) join_add(a.o[c], f, v[i][c]);
    }
  }
}

template <typename T, int C>
__device__ __forceinline__ void join_store(const JoinParams &p, const ShareJoin &j, int row, int col,
                                           const JoinSum<C> &a) {
  const float inv = a.l == 0.f ? 0.f : 1.f / a.l;  // (no key seen: zeros)
  const long long r = j.out_row + (long long)(row / j.group) * j.stride + row % j.group;
  T *out = static_cast<T *>(p.out) + r * p.width + col;
#pragma unroll
  for (int c = 0; c < C; ++c)
    store4(out + 128 * c, a.o[c].x * inv, a.o[c].y * inv, a.o[c].z * inv, a.o[c].w * inv);
}

}  // namespace

template <typename T, int C>
__global__ void __launch_bounds__(kJoinThreads, kJoinCtas) pa_share_join_kernel(const __grid_constant__ JoinParams p) {
  __shared__ JoinSum<1> s_part[kJoinWarps * 4][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool live = lane * 4 < p.width;  // (width 64: half a warp)

  pdl_wait_primary();
  pdl_launch_dependents();
  const int per = p.item_rows, shares = p.space.shares;
  const int narrow = p.width / 32, wide = per * narrow;
  const int warps = gridDim.x * kJoinWarps;
  int i = blockIdx.x * kJoinWarps + warp;
  // (an item's unit is read with the item before it, the first with the counts: what
  // the list holds behind its end is not used)
  ShareJoin j = load_join(p.space.join + min(i / (per * C), shares - 1));
  ShareJoin jm = load_join(p.space.join + max(shares - 1 - (int)blockIdx.x / wide, 0));
  const int few = __ldcg(p.space.counters + kShareFew) * per;
  const int many = __ldcg(p.space.counters + kShareMany) * wide;
  // rows of units of few pieces: a warp's each, or (while there are warps for it) a
  // warp's every 128 columns
  if (C > 1 && few * C <= warps) {
    const int row = i / C % per, col = i % C * 128 + lane * 4;
    if (i < few * C && row < j.rows) {
      JoinSum<1> s;
      join_pieces(p, j, row, col, 0, 1, s);
      join_store<T>(p, j, row, col, s);
    }
  } else {
    if (C > 1) j = load_join(p.space.join + min(i / per, shares - 1));
    while (i < few) {
      const int row = i % per;
      i += warps;
      const ShareJoin next = load_join(p.space.join + min(i / per, shares - 1));
      if (row < j.rows && live) {
        JoinSum<C> s;
        join_pieces(p, j, row, lane * 4, 0, 1, s);
        join_store<T>(p, j, row, lane * 4, s);
      }
      j = next;
    }
  }
  // of many: 32 columns a CTA; a warp takes four pieces at once, eight lanes each
  for (i = blockIdx.x; i < many;) {
    const int row = i / narrow % per, col = i % narrow * 32 + (lane & 7) * 4;
    i += gridDim.x;
    const ShareJoin next = load_join(p.space.join + max(shares - 1 - i / wide, 0));
    if (row < jm.rows) {
      JoinSum<1> s;
      join_pieces(p, jm, row, col, warp * 4 + (lane >> 3), kJoinWarps * 4, s);
      s_part[warp * 4 + (lane >> 3)][lane & 7] = s;
      __syncthreads();
      if (warp == 0) {
        // lanes 8 q .. 8 q + 7 join every fourth of them, then the four their sums
        JoinSum<1> r = s_part[lane >> 3][lane & 7];
        for (int w = 4 + (lane >> 3); w < kJoinWarps * 4; w += 4) join_sum(r, s_part[w][lane & 7]);
#pragma unroll
        for (int d = 8; d < 32; d <<= 1) {
          JoinSum<1> q;
          q.m = __shfl_xor_sync(0xffffffffu, r.m, d);
          q.l = __shfl_xor_sync(0xffffffffu, r.l, d);
          q.o[0].x = __shfl_xor_sync(0xffffffffu, r.o[0].x, d);
          q.o[0].y = __shfl_xor_sync(0xffffffffu, r.o[0].y, d);
          q.o[0].z = __shfl_xor_sync(0xffffffffu, r.o[0].z, d);
          q.o[0].w = __shfl_xor_sync(0xffffffffu, r.o[0].w, d);
          join_sum(r, q);
        }
        if (lane < 8) join_store<T>(p, jm, row, col, r);
      }
      __syncthreads();
    }
    jm = next;
  }
  // the counters as the next call needs them: no CTA has one to read any more
  __syncthreads();
  if (threadIdx.x == 0 && atomicAdd(p.space.counters + kShareDone, 1) == (int)gridDim.x - 1) {
    p.space.counters[kShareTaken] = 0;
    p.space.counters[kShareFew] = 0;
    p.space.counters[kShareMany] = 0;
    p.space.counters[kShareDone] = 0;
  }
}

pa_status_t share_launch_join(const JoinParams &p, int dtype_bf16, int sms, void *stream) {
#define PICK(C)                                                                          \
  (dtype_bf16 ? reinterpret_cast<const void *>(&pa_share_join_kernel<__nv_bfloat16, C>) \
              : reinterpret_cast<const void *>(&pa_share_join_kernel<__half, C>))
  const void *fn = p.width == 512 ? PICK(4) : p.width == 256 ? PICK(2) : PICK(1);
#undef PICK
  void *args[1] = {const_cast<JoinParams *>(&p)};
  const pa_status_t st = host_launch(fn, (unsigned)(kJoinCtas * sms), 1, kJoinThreads, 0, stream, args, "launch join kernel");
  if (st != PA_OK) host_clear(p.space.counters + kShareTaken, (kShareDone - kShareTaken + 1) * sizeof(int), stream);
  return st;
}

}  // namespace pa
