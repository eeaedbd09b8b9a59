// The join of attention that was cut into shares (pa_share.cuh).
//
// A unit of few pieces is a warp's work a row and 128 columns; one of many is a
// CTA's a row and 32 columns, so that hundreds of pieces are a few loads deep.  Bound: the launch and a chain of
// three loads (how many units, the unit, its pieces); the bytes are a few MB
// that the attention kernel left in L2.
#include "pa_share.cuh"

namespace pa {

namespace {

constexpr int kJoinWarps = kJoinThreads / 32;

__device__ __forceinline__ ShareJoin load_join(const ShareJoin *at) {
  const int4 a = __ldcg(reinterpret_cast<const int4 *>(at)), b = __ldcg(reinterpret_cast<const int4 *>(at) + 1);
  ShareJoin j;
  j.share = a.x, j.parts = a.y, j.by = a.z, j.rows = a.w;
  j.group = b.x, j.stride = b.y;
  j.out_row = (long long)((unsigned long long)(uint32_t)b.w << 32 | (uint32_t)b.z);
  return j;
}

// The pieces k = first, first + by, ... of four columns of a row: their maximum,
// sum and weighted outputs.
struct JoinSum {
  float m, l;
  float4 o;
};
__device__ __forceinline__ void join_scale(JoinSum &a, float m) {
  const float f = exp2f(a.m - m);
  a.l *= f;
  a.o.x *= f, a.o.y *= f, a.o.z *= f, a.o.w *= f;
  a.m = m;
}
__device__ __forceinline__ void join_add(JoinSum &a, float f, float l, const float4 &o) {
  a.l += l * f;
  a.o.x += o.x * f, a.o.y += o.y * f, a.o.z += o.z * f, a.o.w += o.w * f;
}
__device__ __forceinline__ void join_pieces(const JoinParams &p, const ShareJoin &j, int row, int col,
                                            int first, int by, JoinSum &a) {
  constexpr int U = 8;  // loads in flight
  a.m = -3.402823466e38f;
  a.l = 0.f;
  a.o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k0 = first; k0 < j.parts; k0 += by * U) {
    float2 ml[U];
    float4 v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = k0 + i * by;
      ml[i] = make_float2(a.m, 0.f);
      v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (k < j.parts) {
        const size_t place = k == 0 ? 2 * (size_t)j.share + 1 : 2 * ((size_t)j.share + (size_t)k * j.by);
        const size_t at = place * p.max_rows + row;
        ml[i] = __ldcg(p.space.ml + at);
        v[i] = __ldcg(reinterpret_cast<const float4 *>(p.space.o + at * p.width + col));
      }
    }
    float m = a.m;
#pragma unroll
    for (int i = 0; i < U; ++i) m = fmaxf(m, ml[i].x);
    join_scale(a, m);
#pragma unroll
    for (int i = 0; i < U; ++i) join_add(a, exp2f(ml[i].x - m), ml[i].y, v[i]);
  }
}

template <typename T>
__device__ __forceinline__ void join_store(const JoinParams &p, const ShareJoin &j, int row, int col,
                                           const JoinSum &a) {
  const float inv = a.l == 0.f ? 0.f : 1.f / a.l;  // (no key seen: zeros)
  const long long r = j.out_row + (long long)(row / j.group) * j.stride + row % j.group;
  store4(static_cast<T *>(p.out) + r * p.width + col, a.o.x * inv, a.o.y * inv, a.o.z * inv,
         a.o.w * inv);
}

}  // namespace

template <typename T>
__global__ void __launch_bounds__(kJoinThreads, kJoinCtas) pa_share_join_kernel(const __grid_constant__ JoinParams p) {
  __shared__ JoinSum s_part[kJoinWarps * 4][8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = (p.width + 127) / 128;
  const bool live = lane * 4 < p.width;  // (width 64: half a warp)

  pdl_wait_primary();
  pdl_launch_dependents();
  // (an item's unit is read with the item before it, the first with the counts: what
  // the list holds behind its end is not used)
  const int per = p.max_rows * chunks, shares = p.space.shares;
  const int narrow = p.width / 32, wide = p.max_rows * narrow;
  int i = blockIdx.x * kJoinWarps + warp;
  ShareJoin j = load_join(p.space.join + min(i / per, shares - 1));
  ShareJoin jm = load_join(p.space.join + max(shares - 1 - (int)blockIdx.x / wide, 0));
  const int few = __ldcg(p.space.counters + kShareFew) * per;
  const int many = __ldcg(p.space.counters + kShareMany) * wide;
  // rows of units of few pieces: a warp's each
  while (i < few) {
    const int row = i / chunks % p.max_rows, col = i % chunks * 128 + lane * 4;
    i += gridDim.x * kJoinWarps;
    const ShareJoin next = load_join(p.space.join + min(i / per, shares - 1));
    if (row < j.rows && live) {
      JoinSum s;
      join_pieces(p, j, row, col, 0, 1, s);
      join_store<T>(p, j, row, col, s);
    }
    j = next;
  }
  // of many: 32 columns a CTA; a warp takes four pieces at once, eight lanes each
  for (i = blockIdx.x; i < many;) {
    const int row = i / narrow % p.max_rows, col = i % narrow * 32 + (lane & 7) * 4;
    i += gridDim.x;
    const ShareJoin next = load_join(p.space.join + max(shares - 1 - i / wide, 0));
    if (row < jm.rows) {
      JoinSum s;
      join_pieces(p, jm, row, col, warp * 4 + (lane >> 3), kJoinWarps * 4, s);
      s_part[warp * 4 + (lane >> 3)][lane & 7] = s;
      __syncthreads();
      if (warp == 0) {
        // lanes 8 q .. 8 q + 7 join every fourth of them, then the four their sums
        JoinSum r = s_part[lane >> 3][lane & 7];
        for (int w = 4 + (lane >> 3); w < kJoinWarps * 4; w += 4) {
          const JoinSum &q = s_part[w][lane & 7];
          const float m = fmaxf(r.m, q.m);
          join_scale(r, m);
          join_add(r, exp2f(q.m - m), q.l, q.o);
        }
#pragma unroll
        for (int d = 8; d < 32; d <<= 1) {
          JoinSum q;
          q.m = __shfl_xor_sync(0xffffffffu, r.m, d);
          q.l = __shfl_xor_sync(0xffffffffu, r.l, d);
          q.o.x = __shfl_xor_sync(0xffffffffu, r.o.x, d);
          q.o.y = __shfl_xor_sync(0xffffffffu, r.o.y, d);
          q.o.z = __shfl_xor_sync(0xffffffffu, r.o.z, d);
          q.o.w = __shfl_xor_sync(0xffffffffu, r.o.w, d);
          const float m = fmaxf(r.m, q.m);
          join_scale(r, m);
          join_add(r, exp2f(q.m - m), q.l, q.o);
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

const void *share_join_kernel(int dtype_bf16) {
  return dtype_bf16 ? reinterpret_cast<const void *>(&pa_share_join_kernel<__nv_bfloat16>)
                    : reinterpret_cast<const void *>(&pa_share_join_kernel<__half>);
}

}  // namespace pa
