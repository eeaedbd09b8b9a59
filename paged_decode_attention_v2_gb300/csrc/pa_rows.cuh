// What the calls that append rows to a paged cache share: the two 16-byte
// chunks of a head that a thread rotates, and where a row goes.
#pragma once

#include <type_traits>

#include "pa_device.cuh"

namespace pa {
namespace {

template <typename T>
struct Chunk2 {  // two 16-byte chunks
  static constexpr int N = 16 / (int)sizeof(T);
  uint4 a, b;
};

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
template <typename T>
__device__ __forceinline__ uint4 narrow(const float (&f)[16 / sizeof(T)]) {
  if constexpr (sizeof(T) == 4) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  } else {
    return make_uint4(MmaOp<T>::pack(f[0], f[1]), MmaOp<T>::pack(f[2], f[3]),
                      MmaOp<T>::pack(f[4], f[5]), MmaOp<T>::pack(f[6], f[7]));
  }
}

// The chunk indices of unit u of a head, rot of whose units are rotated.
__device__ __forceinline__ void unit_chunks(int u, int rot, bool interleaved, int &a, int &b) {
  if (u < rot && !interleaved) {
    a = u;
    b = u + rot;
  } else {
    a = 2 * u;
    b = 2 * u + 1;
  }
}

// The cosines and sines of a unit's angles; cs: the row's [cos | sin] of
// `half` angles each.
template <int N>
struct Angles {
  float c[N], s[N];
  __device__ __forceinline__ void load(const float *cs, int u, int half) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 cv = __ldg(reinterpret_cast<const float4 *>(cs + u * N + i));
      const float4 sv = __ldg(reinterpret_cast<const float4 *>(cs + half + u * N + i));
      c[i] = cv.x, c[i + 1] = cv.y, c[i + 2] = cv.z, c[i + 3] = cv.w;
      s[i] = sv.x, s[i + 1] = sv.y, s[i + 2] = sv.z, s[i + 3] = sv.w;
    }
  }
};

// x c - y s and x c + y s: contracted to a fused multiply-add, or (EACH) with
// each of the three operations rounded by itself, as plain tensor operations do
template <bool EACH>
__device__ __forceinline__ float turn_sub(float x, float c, float y, float s) {
  return EACH ? __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s)) : x * c - y * s;
}
template <bool EACH>
__device__ __forceinline__ float turn_add(float x, float c, float y, float s) {
  return EACH ? __fadd_rn(__fmul_rn(x, c), __fmul_rn(y, s)) : x * c + y * s;
}

// Rotate a unit in place (fp32 arithmetic, one rounding to T).
template <typename T, bool EACH = false>
__device__ __forceinline__ void rotate_unit(Chunk2<T> &x, const Angles<Chunk2<T>::N> &r,
                                            bool interleaved) {
  constexpr int N = Chunk2<T>::N;
  float a[N], b[N], ya[N], yb[N];
  widen<T>(x.a, a);
  widen<T>(x.b, b);
  if (!interleaved) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      ya[i] = turn_sub<EACH>(a[i], r.c[i], b[i], r.s[i]);
      yb[i] = turn_add<EACH>(b[i], r.c[i], a[i], r.s[i]);
    }
  } else {
    // pairs (0,1), (2,3) ... of the 2N consecutive elements; pair j has angle j
#pragma unroll
    for (int j = 0; j < N / 2; ++j) {
      ya[2 * j] = turn_sub<EACH>(a[2 * j], r.c[j], a[2 * j + 1], r.s[j]);
      ya[2 * j + 1] = turn_add<EACH>(a[2 * j + 1], r.c[j], a[2 * j], r.s[j]);
      yb[2 * j] = turn_sub<EACH>(b[2 * j], r.c[N / 2 + j], b[2 * j + 1], r.s[N / 2 + j]);
      yb[2 * j + 1] = turn_add<EACH>(b[2 * j + 1], r.c[N / 2 + j], b[2 * j], r.s[N / 2 + j]);
    }
  }
  x.a = narrow<T>(ya);
  x.b = narrow<T>(yb);
}

// A row's sequence, token, chunk end and page; false: nothing to do for it (a
// padding row, an empty slot) or bad input (reported).
struct RowInfo {
  int tok, tok_end;  // tok_end: the chunk's end, L
  int blk;           // the token's page (not yet checked)
  bool starts;       // its chunk's first row
};
// (by a warp, for one row)
template <class Params>
__device__ __forceinline__ bool locate_row(const Params &p, int row, RowInfo &o) {
  const int lane = threadIdx.x & 31;
  int s = row, i = 0, n = 1;
  if (p.q_start) {
    check_starts(p.q_start, p.num_seqs, row, p.num_rows, p.status);
    const int lo = first_above(p.q_start, p.num_seqs + 1, row);
    if (lo > p.num_seqs) return false;  // behind the last sequence
    if (lo == 0) {                      // before the first chunk: q_start[0] must be 0
      if (lane == 0) report(p.status, kStatusBadInput);
      return false;
    }
    s = lo - 1;
    const int q0 = __ldg(p.q_start + s), q1 = __ldg(p.q_start + lo);
    i = row - q0;
    n = q1 - q0;
    if (q0 < 0 || i < 0 || i >= n || q1 > p.num_rows) {  // decreasing, or past the rows
      if (lane == 0) report(p.status, kStatusBadInput);
      return false;
    }
  }
  const int L = __ldg(p.seq_lens + s);
  if (!p.q_start && L == 0) return false;  // an empty slot of a decode batch
  if (L < n || L > p.max_seq_len) {
    if (lane == 0) report(p.status, kStatusBadInput);
    return false;
  }
  o.tok = L - n + i;
  o.tok_end = L;
  o.starts = i == 0;
  o.blk = __ldg(p.block_tables + (size_t)s * p.max_blocks_per_seq + (o.tok >> p.log2_block_size));
  return true;
}

// The row's position; -1 (reported) if the table does not hold it.
template <class Params>
__device__ __forceinline__ int row_position(const Params &p, int row, int tok) {
  const int pos = p.positions ? __ldg(p.positions + row) : tok;
  if (p.rotary_dim && (unsigned)pos >= (unsigned)p.max_position) {
    report(p.status, kStatusBadInput);
    return -1;
  }
  return p.rotary_dim ? pos : 0;
}

}  // namespace
}  // namespace pa
