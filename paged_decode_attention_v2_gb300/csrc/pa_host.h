// Host helpers that the entry points of several translation units share
// (defined in pa_api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>

#include "pa.h"

namespace pa {

// Record a CUDA error for pa_last_cuda_error and return PA_ERR_CUDA.
pa_status_t host_fail_cuda(const char *what, cudaError_t e);
// SMs of the current device.
pa_status_t host_sm_count(int *sms);
// Raise a kernel's dynamic shared-memory limit once per (kernel, device).
pa_status_t host_ensure_smem(const void *fn, size_t bytes);

// TMA's view of rows of `width` 16-bit elements, eight at a time: boxes of
// unit_rows rows (a multiple of 8) from row 8 y at (0, 0, 0, y), landing as
// [8 rows][panel][row][128 bytes] in the 128-byte swizzle.
pa_status_t host_cache_map(CUtensorMap *map, const void *base, int dtype, int width, long long rows,
                           int unit_rows);
// The same rows one panel at a time: boxes of box_rows rows by 64 elements from
// (x, row), landing as [row][128 bytes]; zeros behind the last row.
pa_status_t host_rows_map(CUtensorMap *map, const void *base, int dtype, int width, long long rows,
                          int box_rows);

inline bool host_aligned(const void *p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// The rules every call on the paged cache shares (no pointers): sizes the
// kernels are built for, a table that can hold max_seq_len.
pa_status_t host_check_cache(int dtype, int num_heads, int num_kv_heads, int head_size,
                             int num_blocks, int block_size, int max_blocks_per_seq,
                             int max_seq_len);

// Launch a kernel chained to the one before it in the stream by programmatic
// dependent launch (the kernel itself waits for that one before its first
// global access).
pa_status_t host_launch(const void *fn, unsigned grid_x, unsigned grid_y, int threads, size_t smem,
                        void *stream, void **args, const char *what);

// Zero `bytes` of device memory in the stream, after a launch that failed: what of
// this fails too is the caller's next call's error.
void host_clear(void *at, size_t bytes, void *stream);

}  // namespace pa
