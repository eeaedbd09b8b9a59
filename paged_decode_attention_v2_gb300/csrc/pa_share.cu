// The join of attention that was split into equal shares (pa_share.cuh).
//
// Bound: the launch and a chain of three loads (the units, their maxima, their
// outputs); the bytes are a few MB that the attention kernel left in L2.
#include "pa_share.cuh"

namespace pa {

namespace {

constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinFew = 6;  // pieces that one warp takes by itself

// The pieces k = first, first + by, ... of a row's 128 columns: their maximum,
// sum and weighted outputs (lane: four columns).
struct JoinSum {
  float m, l;
  float4 o;
};
__device__ __forceinline__ void join_pieces(const JoinParams &p, int cta, const ShareJoin &j, int row,
                                            int col, int first, int by, JoinSum &a) {
  constexpr int U = 4;  // loads in flight
  a.m = -CUDART_INF_F;
  a.l = 0.f;
  a.o = make_float4(0.f, 0.f, 0.f, 0.f);
  auto place = [&](int k) -> size_t {
    // its own place 1, then place 0 of the shares behind it
    const size_t pl = k == 0 ? 2 * (size_t)cta + 1 : 2 * ((size_t)cta + (size_t)k * p.place_step);
    return pl * p.max_rows + row;
  };
  for (int k0 = first; k0 < j.parts; k0 += by * U) {
    float2 ml[U];
    float4 v[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int k = k0 + i * by;
      if (k < j.parts) {
        const size_t at = place(k);
        ml[i] = __ldcg(p.space.ml + at);
        v[i] = __ldcg(reinterpret_cast<const float4 *>(p.space.o + at * p.width + col));
      } else {
        ml[i] = make_float2(-CUDART_INF_F, 0.f);
        v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    float m = a.m;
#pragma unroll
    for (int i = 0; i < U; ++i) m = fmaxf(m, ml[i].x);
    if (m == -CUDART_INF_F) continue;  // no key seen yet
    const float f = exp2f(a.m - m);
    a.l *= f;
    a.o.x *= f, a.o.y *= f, a.o.z *= f, a.o.w *= f;
    a.m = m;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const float g = exp2f(ml[i].x - m);
      if (g == 0.f) continue;  // (a piece that saw no key may hold anything)
      a.l += ml[i].y * g;
      a.o.x += v[i].x * g, a.o.y += v[i].y * g, a.o.z += v[i].z * g, a.o.w += v[i].w * g;
    }
  }
}

template <typename T>
__device__ __forceinline__ void join_store(const JoinParams &p, const ShareJoin &j, int row, int col,
                                           const JoinSum &a) {
  const float inv = a.l > 0.f ? 1.f / a.l : 0.f;
  const long long r = j.out_row + (long long)(row / j.group) * j.stride + row % j.group;
  store4(static_cast<T *>(p.out) + r * p.width + col, a.o.x * inv, a.o.y * inv, a.o.z * inv,
         a.o.w * inv);
}

}  // namespace

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) pa_share_join_kernel(const __grid_constant__ JoinParams p) {
  __shared__ int s_rows[kShareMaxCtas];   // rows to join of each CTA's unit
  __shared__ int s_sum[2][kJoinThreads + 1];  // of units of few pieces, of many; before each thread's
  __shared__ JoinSum s_part[kJoinWarps][32];
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int chunks = p.width / 128 > 0 ? p.width / 128 : 1;
  const bool live = lane * 4 < p.width;  // (width 64: half a warp)

  pdl_wait_primary();
  pdl_launch_dependents();
  const int per = (p.ctas + kJoinThreads - 1) / kJoinThreads;
  int few = 0, many = 0;
  for (int c = t * per; c < min(p.ctas, (t + 1) * per); ++c) {
    const int parts = __ldcg(&p.space.join[c].parts);
    const int rows = parts > 0 ? __ldcg(&p.space.join[c].rows) : 0;
    s_rows[c] = parts > kJoinFew ? -rows : rows;
    if (parts > kJoinFew)
      many += rows;
    else
      few += rows;
  }
  // running sums over the threads
  int a = few, b = many;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, a, d), y = __shfl_up_sync(0xffffffffu, b, d);
    if (lane >= d) a += x, b += y;
  }
  __shared__ int s_w[2][kJoinWarps];
  if (lane == 31) s_w[0][warp] = a, s_w[1][warp] = b;
  __syncthreads();
  for (int w = 0; w < warp; ++w) a += s_w[0][w], b += s_w[1][w];
  s_sum[0][t] = a - few;
  s_sum[1][t] = b - many;
  if (t == kJoinThreads - 1) s_sum[0][kJoinThreads] = a, s_sum[1][kJoinThreads] = b;
  __syncthreads();
  // the CTA and row of the i-th row to join of one kind
  auto find = [&](int kind, int i, int &row) -> int {
    int lo = 0, hi = kJoinThreads - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (s_sum[kind][mid] <= i)
        lo = mid;
      else
        hi = mid - 1;
    }
    int x = i - s_sum[kind][lo], c = lo * per;
    while (true) {
      const int n = kind ? max(-s_rows[c], 0) : max(s_rows[c], 0);
      if (x < n) break;
      x -= n;
      ++c;
    }
    row = x;
    return c;
  };
  // of few pieces: a warp's each
  const int total_few = s_sum[0][kJoinThreads] * chunks;
  for (int i = blockIdx.x * kJoinWarps + warp; i < total_few; i += gridDim.x * kJoinWarps) {
    int row;
    const int c = find(0, i / chunks, row), col = (i % chunks) * 128 + lane * 4;
    const ShareJoin j = p.space.join[c];
    if (live) {
      JoinSum s;
      join_pieces(p, c, j, row, col, 0, 1, s);
      join_store<T>(p, j, row, col, s);
    }
  }
  // of many: the CTA's
  const int total_many = s_sum[1][kJoinThreads] * chunks;
  for (int i = blockIdx.x; i < total_many; i += gridDim.x) {
    int row;
    const int c = find(1, i / chunks, row), col = (i % chunks) * 128 + lane * 4;
    const ShareJoin j = p.space.join[c];
    JoinSum s;
    if (live) {
      join_pieces(p, c, j, row, col, warp, kJoinWarps, s);
      s_part[warp][lane] = s;
    }
    __syncthreads();
    if (warp == 0 && live) {
      float m = -CUDART_INF_F;
      for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, s_part[w][lane].m);
      JoinSum r;
      r.m = m;
      r.l = 0.f;
      r.o = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int w = 0; w < kJoinWarps; ++w) {
        const JoinSum &q = s_part[w][lane];
        if (q.m == -CUDART_INF_F) continue;
        const float g = exp2f(q.m - m);
        r.l += q.l * g;
        r.o.x += q.o.x * g, r.o.y += q.o.y * g, r.o.z += q.o.z * g, r.o.w += q.o.w * g;
      }
      join_store<T>(p, j, row, col, r);
    }
    __syncthreads();
  }
}

const void *share_join_kernel(int dtype_bf16) {
  return dtype_bf16 ? reinterpret_cast<const void *>(&pa_share_join_kernel<__nv_bfloat16>)
                    : reinterpret_cast<const void *>(&pa_share_join_kernel<__half>);
}

}  // namespace pa
