"""Python binding of libpa, the GB300 paged decode attention library.

Argument marshalling only: every step of the computation runs in libpa's
CUDA kernels.  The functions carry the C ABI's names (``include/pa.h``) and
take torch tensors for the buffers; the torch stream is passed through as a
raw ``cudaStream_t``.  There is no fallback: if ``_lib/libpa.so`` is missing
(build it with ``python -m paged_decode_attention_v2_gb300.build_lib``) the
first call raises.

Layouts: query/out [num_seqs, num_heads, head_size]; key/value cache
[num_blocks, num_kv_heads, block_size, head_size]; block_tables int32
[num_seqs, max_blocks_per_seq]; seq_lens int32 [num_seqs].
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libpa.so")

PA_OK = 0
PA_ERR_INVALID_ARG = 1
PA_ERR_UNSUPPORTED = 2
PA_ERR_WORKSPACE_TOO_SMALL = 3
PA_ERR_CUDA = 4
PA_ERR_DEVICE_BAD_INPUT = 5
PA_ERR_DEVICE_TIMEOUT = 6

PA_DTYPE_F32, PA_DTYPE_BF16, PA_DTYPE_F16 = 0, 1, 2
PA_VARIANT_AUTO, PA_VARIANT_V1, PA_VARIANT_V2 = 0, 1, 2
PA_MATH_AUTO, PA_MATH_SIMT, PA_MATH_TENSOR = 0, 1, 2
PA_DEBUG_STALL_CONSUMERS = 1
PA_DEBUG_NO_TCGEN05 = 2
PA_DEBUG_TCGEN05_KEYS = 4

_DTYPES = {torch.float32: PA_DTYPE_F32, torch.bfloat16: PA_DTYPE_BF16,
           torch.float16: PA_DTYPE_F16}

# Every function the header declares (checked against include/pa.h by tests).
EXPORTS = ("pa_workspace_bytes", "pa_workspace_layout", "pa_workspace_init",
           "pa_v1_forward", "pa_v2_forward", "pa_forward", "pa_choose_v2", "pa_choose_v2_chunks",
           "pa_read_device_status", "pa_status_string", "pa_last_cuda_error",
           "pa_version", "pa_v2_forward_noalloc", "pa_host_staging_bytes", "pa_forward_host",
           "pa_chunks_forward", "pa_v2_partials", "pa_v2_combine", "pa_append_kv",
           "pa_select_blocks", "pa_sparse_forward", "pa_sparse_workspace_bytes",
           "pa_prefix_forward", "pa_prefix_workspace_bytes", "pa_q4_append", "pa_q4_forward",
           "pa_q4_workspace_bytes", "pa_latent_append", "pa_latent_forward",
           "pa_latent_workspace_bytes", "pa_call")


# pa_call's numbers, and the words of each call (q: pointer or integer, d: float)
_Q4_APPEND = (0, struct.Struct("34q").pack)
_Q4_FORWARD = (1, struct.Struct("18qd4q").pack)
_LATENT_APPEND = (2, struct.Struct("6qd24q").pack)
_LATENT_FORWARD = (3, struct.Struct("15qd5q").pack)


class PAError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_text(status)} (status {status})")


class pa_options_t(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int32), ("math", ctypes.c_int32),
                ("num_stages", ctypes.c_int32), ("debug_flags", ctypes.c_int32),
                ("wait_limit_ns", ctypes.c_uint64), ("phase1_event", ctypes.c_void_p),
                ("ctas_per_sm", ctypes.c_int32), ("fuse_partitions", ctypes.c_int32),
                ("share_kv", ctypes.c_int32)]


_lib = None
_lock = threading.Lock()

_FWD_ARGS = [ctypes.c_void_p] * 6 + [ctypes.c_int] * 8 + [ctypes.c_float, ctypes.c_int,
                                                           ctypes.c_int, ctypes.c_void_p,
                                                           ctypes.c_size_t, ctypes.c_void_p]


def load_library(path: str = LIB_PATH):
    """Load libpa (no fallback: raises if the shared library is absent)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"libpa.so not found at {path}; build it with "
                "`python -m paged_decode_attention_v2_gb300.build_lib`")
        lib = ctypes.CDLL(path)
        ci, cs, vp = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
        lib.pa_workspace_bytes.restype = cs
        lib.pa_workspace_bytes.argtypes = [ci] * 5
        lib.pa_workspace_layout.restype = ci
        lib.pa_workspace_layout.argtypes = [ci] * 5 + [ctypes.POINTER(cs)]
        lib.pa_workspace_init.restype = ci
        lib.pa_workspace_init.argtypes = [vp, cs, vp]
        for name in ("pa_v1_forward", "pa_v2_forward"):
            f = getattr(lib, name)
            f.restype = ci
            f.argtypes = _FWD_ARGS
        lib.pa_v2_partials.restype = ci
        lib.pa_v2_partials.argtypes = (_FWD_ARGS[1:17] + [ci, ci] + _FWD_ARGS[17:])
        lib.pa_v2_combine.restype = ci
        lib.pa_v2_combine.argtypes = [vp, vp] + [ci] * 6 + [vp, cs, vp]
        lib.pa_v2_forward_noalloc.restype = ci
        lib.pa_v2_forward_noalloc.argtypes = _FWD_ARGS[:17] + [vp]
        lib.pa_forward.restype = ci
        lib.pa_forward.argtypes = _FWD_ARGS + [ctypes.POINTER(pa_options_t)]
        lib.pa_chunks_forward.restype = ci
        lib.pa_chunks_forward.argtypes = ([vp] * 7 + [ci] * 10 +
                                          [ctypes.c_float, ci, ci, vp, cs, vp,
                                           ctypes.POINTER(pa_options_t)])
        lib.pa_host_staging_bytes.restype = cs
        lib.pa_host_staging_bytes.argtypes = [ci] * 5
        lib.pa_forward_host.restype = ci
        lib.pa_forward_host.argtypes = (_FWD_ARGS[:17] + [vp, cs] + _FWD_ARGS[17:] +
                                        [ctypes.POINTER(pa_options_t)])
        ll = ctypes.c_longlong
        lib.pa_append_kv.restype = ci
        lib.pa_append_kv.argtypes = [vp] * 7 + [ll] * 3 + [vp] * 5 + [ci] * 13 + [vp, cs, vp]
        lib.pa_prefix_workspace_bytes.restype = cs
        lib.pa_prefix_workspace_bytes.argtypes = [ci] * 8
        lib.pa_prefix_forward.restype = ci
        lib.pa_prefix_forward.argtypes = ([vp] * 9 + [ci] * 11 +
                                          [ctypes.c_float, ci, ci, vp, cs, vp,
                                           ctypes.POINTER(pa_options_t)])
        lib.pa_sparse_workspace_bytes.restype = cs
        lib.pa_sparse_workspace_bytes.argtypes = [ci] * 8
        lib.pa_select_blocks.restype = ci
        lib.pa_select_blocks.argtypes = [vp] * 6 + [ci] * 14 + [vp, cs, vp]
        lib.pa_sparse_forward.restype = ci
        lib.pa_sparse_forward.argtypes = ([vp] * 9 + [ci] * 12 + [ctypes.c_float, ci, ci, vp, cs,
                                                                  vp])
        lib.pa_call.restype = ci
        lib.pa_call.argtypes = [ci, ctypes.c_char_p]
        lib.pa_latent_workspace_bytes.restype = cs
        lib.pa_latent_workspace_bytes.argtypes = [ci]
        lib.pa_latent_append.restype = ci
        lib.pa_latent_append.argtypes = ([vp] * 6 + [ctypes.c_float] + [ll] * 4 + [vp] * 5 +
                                         [ci] * 12 + [vp, cs, vp])
        lib.pa_latent_forward.restype = ci
        lib.pa_latent_forward.argtypes = ([vp] * 6 + [ci] * 9 + [ctypes.c_float, ci, vp, cs, vp,
                                                                 ctypes.POINTER(pa_options_t)])
        lib.pa_q4_workspace_bytes.restype = cs
        lib.pa_q4_workspace_bytes.argtypes = [ci]
        lib.pa_q4_append.restype = ci
        lib.pa_q4_append.argtypes = [vp] * 10 + [ll] * 3 + [vp] * 5 + [ci] * 13 + [vp, cs, vp]
        lib.pa_q4_forward.restype = ci
        lib.pa_q4_forward.argtypes = [vp] * 9 + [ci] * 9 + [ctypes.c_float, ci, vp, cs, vp]
        lib.pa_choose_v2.restype = ci
        lib.pa_choose_v2.argtypes = [ci] * 5
        lib.pa_choose_v2_chunks.restype = ci
        lib.pa_choose_v2_chunks.argtypes = [ci] * 8
        lib.pa_read_device_status.restype = ci
        lib.pa_read_device_status.argtypes = [vp, vp]
        lib.pa_status_string.restype = ctypes.c_char_p
        lib.pa_status_string.argtypes = [ci]
        lib.pa_last_cuda_error.restype = ctypes.c_char_p
        lib.pa_last_cuda_error.argtypes = []
        lib.pa_version.restype = ci
        lib.pa_version.argtypes = []
        _lib = lib
        return lib


def status_text(status: int) -> str:
    return load_library().pa_status_string(int(status)).decode()


def _packed(call, what, *args) -> None:
    """A call through pa_call: its arguments as one string of 64-bit words (a foreign
    call of 34 arguments takes five times as long)."""
    status = (_lib or load_library()).pa_call(call[0], call[1](*args))
    if status:
        _check(status, what)


def _check(status: int, what: str) -> int:
    if status != PA_OK:
        if status == PA_ERR_CUDA:
            what = f"{what} [{load_library().pa_last_cuda_error().decode()}]"
        raise PAError(status, what)
    return status


# The current stream's handle without the Stream object (3 us a call) where torch
# offers it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream_handle(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_current_device())
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: torch.Tensor | None) -> int:
    if t is None:
        return 0
    if not t.is_contiguous():
        raise ValueError("libpa takes contiguous tensors")
    return t.data_ptr()


# ---------------------------------------------------------------------------
# Workspace

def pa_workspace_bytes(num_seqs: int, num_heads: int, head_size: int, max_seq_len: int,
                       partition_size: int) -> int:
    return int(load_library().pa_workspace_bytes(num_seqs, num_heads, head_size,
                                                 max_seq_len, partition_size))


def pa_workspace_layout(num_seqs: int, num_heads: int, head_size: int, max_seq_len: int,
                        partition_size: int) -> tuple[int, int, int, int, int]:
    off = (ctypes.c_size_t * 5)()
    _check(load_library().pa_workspace_layout(num_seqs, num_heads, head_size, max_seq_len,
                                              partition_size, off), "pa_workspace_layout")
    return tuple(int(x) for x in off)


def pa_workspace_init(workspace: torch.Tensor, stream=None) -> None:
    _check(load_library().pa_workspace_init(_ptr(workspace), workspace.numel() *
                                            workspace.element_size(),
                                            _stream_handle(stream)), "pa_workspace_init")


def alloc_workspace(num_seqs: int, num_heads: int, head_size: int, max_seq_len: int,
                    partition_size: int, device=None, stream=None) -> torch.Tensor:
    """A zero-status workspace large enough for V2 (and so for V1)."""
    n = max(pa_workspace_bytes(num_seqs, num_heads, head_size, max_seq_len, partition_size), 256)
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    pa_workspace_init(ws, stream)
    return ws


# ---------------------------------------------------------------------------
# Forward calls

def _fwd_args(out, query, key_cache, value_cache, block_tables, seq_lens, scale,
              partition_size, workspace, max_seq_len, stream):
    if query.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {query.dtype}")
    B, H, D = query.shape
    nb, hkv, bs, d2 = key_cache.shape
    if max_seq_len is None:
        max_seq_len = block_tables.shape[1] * bs
    return (_ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache), _ptr(block_tables),
            _ptr(seq_lens), B, H, hkv, D, nb, bs, block_tables.shape[1], int(max_seq_len),
            float(scale), int(partition_size), _DTYPES[query.dtype], _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream_handle(stream))


def pa_v1_forward(out, query, key_cache, value_cache, block_tables, seq_lens, scale,
                  partition_size, workspace, max_seq_len=None, stream=None) -> None:
    """V1: one pass over each whole sequence (see include/pa.h)."""
    _check(load_library().pa_v1_forward(*_fwd_args(
        out, query, key_cache, value_cache, block_tables, seq_lens, scale, partition_size,
        workspace, max_seq_len, stream)), "pa_v1_forward")


def pa_v2_forward(out, query, key_cache, value_cache, block_tables, seq_lens, scale,
                  partition_size, workspace, max_seq_len=None, stream=None) -> None:
    """V2: partition kernel + log-sum-exp reduce (see include/pa.h)."""
    _check(load_library().pa_v2_forward(*_fwd_args(
        out, query, key_cache, value_cache, block_tables, seq_lens, scale, partition_size,
        workspace, max_seq_len, stream)), "pa_v2_forward")


def pa_v2_partials(query, key_cache, value_cache, block_tables, seq_lens, scale,
                   partition_size, workspace, part_begin=0, part_end=2 ** 31 - 1,
                   max_seq_len=None, stream=None) -> None:
    """Phase 1 of V2 over partitions [part_begin, part_end) of every sequence,
    into their workspace slots (see include/pa.h)."""
    a = _fwd_args(query, query, key_cache, value_cache, block_tables, seq_lens, scale,
                  partition_size, workspace, max_seq_len, stream)
    _check(load_library().pa_v2_partials(*a[1:17], int(part_begin), int(part_end), *a[17:]),
           "pa_v2_partials")


def pa_v2_combine(out, seq_lens, partition_size, workspace, max_seq_len, num_kv_heads=None,
                  stream=None) -> None:
    """Phase 2 of V2 alone: out [B, H, D] from the partials in the workspace
    (see include/pa.h).  ``num_kv_heads`` is unused (Phase 2 works per query
    head) and accepted for symmetry with the forward calls."""
    if out.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {out.dtype}")
    B, H, D = out.shape
    _check(load_library().pa_v2_combine(
        _ptr(out), _ptr(seq_lens), B, H, D, int(max_seq_len), int(partition_size),
        _DTYPES[out.dtype], _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream_handle(stream)), "pa_v2_combine")


def pa_v2_forward_noalloc(out, query, key_cache, value_cache, block_tables, seq_lens, scale,
                          partition_size, max_seq_len=None, stream=None) -> None:
    """V2 without a caller workspace, for callers that cannot allocate device
    memory: scratch comes from the library's fixed 32 MiB device array (one
    per GPU, shared by all calls; overlapping calls race)."""
    args = _fwd_args(out, query, key_cache, value_cache, block_tables, seq_lens, scale,
                     partition_size, torch.empty(0, dtype=torch.uint8), max_seq_len, stream)
    _check(load_library().pa_v2_forward_noalloc(*args[:17], args[19]),
           "pa_v2_forward_noalloc")


def _event_handle(ev):
    """The cudaEvent_t of a torch.cuda.Event (or a raw handle), or None."""
    if ev is None:
        return None
    h = ev.cuda_event if hasattr(ev, "cuda_event") else int(ev)
    if not h:
        raise ValueError("phase1_event has no CUDA event yet (torch creates it at the "
                         "first record(); record it once before passing it)")
    return h


def pa_forward(out, query, key_cache, value_cache, block_tables, seq_lens, scale,
               partition_size, workspace, max_seq_len=None, stream=None, variant=PA_VARIANT_AUTO,
               math=PA_MATH_AUTO, num_stages=0, debug_flags=0, wait_limit_ns=0,
               phase1_event=None, ctas_per_sm=0, fuse_partitions=0) -> None:
    """V1 or V2 chosen by pa_choose_v2, or forced through the options.
    ``phase1_event`` (a torch.cuda.Event) is recorded between V2's two kernels."""
    opts = pa_options_t(variant, math, num_stages, debug_flags, wait_limit_ns,
                        _event_handle(phase1_event), ctas_per_sm, fuse_partitions)
    _check(load_library().pa_forward(*_fwd_args(
        out, query, key_cache, value_cache, block_tables, seq_lens, scale, partition_size,
        workspace, max_seq_len, stream), ctypes.byref(opts)), "pa_forward")


def pa_chunks_forward(out, query, key_cache, value_cache, block_tables, seq_lens, q_start,
                      scale, partition_size, workspace, max_seq_len=None, max_chunk=None,
                      stream=None, variant=PA_VARIANT_AUTO, num_stages=0, ctas_per_sm=0,
                      phase1_event=None, debug_flags=0, wait_limit_ns=0,
                      share_kv=0) -> None:
    """Multi-token queries over the paged cache (see include/pa.h): query and
    out [num_rows, H, D]; the chunk of sequence s is rows q_start[s] ..
    q_start[s+1]-1 (int32 on the device), its last tokens.  max_chunk bounds
    the chunk lengths (default: max_seq_len)."""
    if query.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {query.dtype}")
    R, H, D = query.shape
    nb, hkv, bs, d2 = key_cache.shape
    B = seq_lens.numel()
    if q_start.numel() != B + 1 or q_start.dtype != torch.int32:
        raise ValueError("q_start must be int32 [num_seqs + 1]")
    if max_seq_len is None:
        max_seq_len = block_tables.shape[1] * bs
    mc = int(max_chunk) if max_chunk is not None else int(max_seq_len)
    opts = pa_options_t(variant, PA_MATH_AUTO, num_stages, debug_flags, wait_limit_ns,
                        _event_handle(phase1_event), ctas_per_sm, 0, share_kv)
    _check(load_library().pa_chunks_forward(
        _ptr(out), _ptr(query), _ptr(key_cache), _ptr(value_cache), _ptr(block_tables),
        _ptr(seq_lens), _ptr(q_start), B, R, mc, H, hkv, D, nb, bs, block_tables.shape[1],
        int(max_seq_len), float(scale), int(partition_size), _DTYPES[query.dtype],
        _ptr(workspace), workspace.numel() * workspace.element_size(), _stream_handle(stream),
        ctypes.byref(opts)), "pa_chunks_forward")


def _pointers(first, workspace, same, ints, *more):
    """Data pointers of the workspace, of `same` (tensors of first's dtype), of
    `ints` (int32) and of `more` ((dtype, tensors) each), in this order, 0 for
    None; all contiguous, on the current CUDA device."""
    dtype = first.dtype
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    index = first.get_device()
    if index < 0 or index != _current_device():
        raise ValueError(f"tensors on {first.device}: libpa runs on the current CUDA device")
    out = []
    for want, tensors in ((workspace.dtype, (workspace,)), (dtype, same), (torch.int32, ints), *more):
        for t in tensors:
            if t is None:
                out.append(0)
                continue
            if t.dtype is not want or t.get_device() != index:
                raise ValueError("libpa takes tensors of one dtype, and int32 tables, lengths and "
                                 "starts, on one device")
            if not t.is_contiguous():
                raise ValueError("libpa takes contiguous tensors")
            out.append(t.data_ptr())
    return out


def _rows(t, like, heads: int, head_size: int):
    """(pointer, elements between rows, rows) of a [rows, heads, head_size] tensor
    whose rows are contiguous, of the dtype and on the device of `like`."""
    if t.dim() != 3 or t.dtype is not like.dtype or t.get_device() != like.get_device():
        raise ValueError("libpa takes [rows, heads, head_size] tensors of the caches' dtype and device")
    rows, h, d = t.shape
    if h != heads or d != head_size:
        raise ValueError(f"expected [rows, {heads}, {head_size}], got {list(t.shape)}")
    step, s1, s2 = t.stride()
    if s2 != 1 or (h > 1 and s1 != d):
        raise ValueError("libpa takes rows of contiguous heads")
    return t.data_ptr(), step if rows > 1 else h * d, rows


def _angles(cos_sin, like, rotary_dim):
    """(pointer, positions, rotary_dim) of a float32 [max_position, rotary_dim] table on
    the device of `like`; rotary_dim None is its width."""
    if cos_sin is None:
        return 0, 0, int(rotary_dim or 0)
    if cos_sin.dtype is not torch.float32 or cos_sin.dim() != 2 \
            or cos_sin.get_device() != like.get_device():
        raise ValueError("cos_sin must be float32 [max_position, rotary_dim]")
    max_position, width = cos_sin.shape
    if rotary_dim is None:
        rotary_dim = width
    elif rotary_dim != width and rotary_dim != 0:
        raise ValueError("cos_sin must be float32 [max_position, rotary_dim]")
    return _ptr(cos_sin), max_position, int(rotary_dim)


def pa_append_kv(key_cache, value_cache, key, value, block_tables, seq_lens, workspace,
                 query=None, query_out=None, key_bounds=None, cos_sin=None, positions=None,
                 q_start=None, rotary_dim=None, interleaved=False, max_seq_len=None,
                 stream=None) -> None:
    """Append key / value [rows, Hkv, D] (rows may be strided slices) to the
    paged cache, keys rotated by cos_sin [max_position, rotary_dim] on the way
    and query [rows, H, D] rotated into query_out; key_bounds [num_blocks, Hkv,
    2, D] follows the keys (see include/pa.h).  seq_lens are the lengths after
    the append.  rotary_dim defaults to cos_sin's width."""
    shape = key_cache.shape
    nb, hkv, bs, D = shape
    ws, kc, vc, kb, qo, bt, sl, qs, pos = _pointers(
        key_cache, workspace, (key_cache, value_cache, key_bounds, query_out),
        (block_tables, seq_lens, q_start, positions))
    kp, kst, R = _rows(key, key_cache, hkv, D)
    vp, vst, rows = _rows(value, key_cache, hkv, D)
    B = seq_lens.numel()
    if value_cache.shape != shape or rows != R:
        raise ValueError("key and value (and their caches) differ in shape")
    if qs and q_start.numel() != B + 1:
        raise ValueError("q_start must be int32 [num_seqs + 1]")
    if block_tables.dim() != 2 or block_tables.shape[0] != B:
        raise ValueError("block_tables must be int32 [num_seqs, max_blocks_per_seq]")
    blocks = block_tables.shape[1]
    if pos and positions.numel() != R:
        raise ValueError("positions must be int32 [rows]")
    if kb and key_bounds.shape != (nb, hkv, 2, D):
        raise ValueError("key_bounds must be [num_blocks, num_kv_heads, 2, head_size]")
    H, qp, qst = hkv, 0, 0
    if query is not None:
        if query.dim() != 3 or query_out is None or query_out.shape != query.shape:
            raise ValueError("query and query_out must both be [rows, num_heads, head_size]")
        H = query.shape[1]
        qp, qst, rows = _rows(query, key_cache, H, D)
        if rows != R:
            raise ValueError("query and query_out must both be [rows, num_heads, head_size]")
    elif query_out is not None:
        raise ValueError("query_out without a query")
    cs, max_position, rotary_dim = _angles(cos_sin, key_cache, rotary_dim)
    if max_seq_len is None:
        max_seq_len = blocks * bs
    _check((_lib or load_library()).pa_append_kv(
        kc, vc, kb, qo, qp, kp, vp, qst, kst, vst, cs, pos, bt, sl, qs, B, R, H, hkv, D, nb, bs,
        blocks, int(max_seq_len), rotary_dim, int(interleaved), max_position,
        _DTYPES[key_cache.dtype], ws, workspace.numel() * workspace.element_size(),
        _stream_handle(stream)), "pa_append_kv")


def pa_prefix_workspace_bytes(num_seqs: int, num_prefixes: int, num_heads: int, num_kv_heads: int,
                              head_size: int, max_seq_len: int, max_prefix_len: int,
                              partition_size: int) -> int:
    return int(load_library().pa_prefix_workspace_bytes(
        num_seqs, num_prefixes, num_heads, num_kv_heads, head_size, max_seq_len, max_prefix_len,
        partition_size))


def alloc_prefix_workspace(num_seqs: int, num_prefixes: int, num_heads: int, num_kv_heads: int,
                           head_size: int, max_seq_len: int, max_prefix_len: int,
                           partition_size: int, device=None, stream=None) -> torch.Tensor:
    """A zeroed workspace for pa_prefix_forward, with these sizes or smaller ones."""
    n = pa_prefix_workspace_bytes(num_seqs, num_prefixes, num_heads, num_kv_heads, head_size,
                                  max_seq_len, max_prefix_len, partition_size)
    if n == 0:
        raise ValueError("bad sizes for a prefix workspace")
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    pa_workspace_init(ws, stream)
    return ws


def pa_prefix_forward(out, query, key_cache, value_cache, block_tables, seq_lens, prefix_tables,
                      prefix_lens, prefix_start, scale, partition_size, workspace,
                      max_seq_len=None, max_prefix_len=None, stream=None, num_stages=0,
                      ctas_per_sm=0, debug_flags=0, wait_limit_ns=0) -> None:
    """Decode attention for sequences that share prefixes (see include/pa.h):
    prefix_tables int32 [num_prefixes, max_prefix_blocks], prefix_lens int32
    [num_prefixes], prefix_start int32 [num_prefixes + 1]; block_tables and
    seq_lens are the sequences' own tokens."""
    B, H, D = query.shape
    nb, hkv, bs, D2 = key_cache.shape
    ws, o, q, kc, vc, bt, sl, pt, pl, ps = _pointers(
        query, workspace, (out, query, key_cache, value_cache),
        (block_tables, seq_lens, prefix_tables, prefix_lens, prefix_start))
    G = prefix_lens.numel()
    if out.shape != query.shape or D2 != D or value_cache.shape != key_cache.shape:
        raise ValueError("query and out, or the caches, differ in shape")
    if block_tables.dim() != 2 or block_tables.shape[0] != B or seq_lens.numel() != B:
        raise ValueError("block_tables must be int32 [num_seqs, max_blocks_per_seq]")
    if prefix_tables.dim() != 2 or prefix_tables.shape[0] != G or prefix_start.numel() != G + 1:
        raise ValueError("prefix_tables must be int32 [num_prefixes, max_prefix_blocks], "
                         "prefix_start int32 [num_prefixes + 1]")
    blocks, pblocks = block_tables.shape[1], prefix_tables.shape[1]
    if max_seq_len is None:
        max_seq_len = blocks * bs
    if max_prefix_len is None:
        max_prefix_len = pblocks * bs
    opts = pa_options_t(PA_VARIANT_V2, PA_MATH_AUTO, num_stages, debug_flags, wait_limit_ns, None,
                        ctas_per_sm, 0, 0)
    _check((_lib or load_library()).pa_prefix_forward(
        o, q, kc, vc, bt, sl, pt, pl, ps, B, G, H, hkv, D, nb, bs, blocks, pblocks,
        int(max_seq_len), int(max_prefix_len), float(scale), int(partition_size),
        _DTYPES[query.dtype], ws, workspace.numel() * workspace.element_size(),
        _stream_handle(stream), ctypes.byref(opts)), "pa_prefix_forward")


def pa_sparse_workspace_bytes(num_rows: int, num_heads: int, num_kv_heads: int, head_size: int,
                              block_size: int, max_seq_len: int, num_selected: int,
                              partition_size: int) -> int:
    return int(load_library().pa_sparse_workspace_bytes(
        num_rows, num_heads, num_kv_heads, head_size, block_size, max_seq_len, num_selected,
        partition_size))


def alloc_sparse_workspace(num_rows: int, num_heads: int, num_kv_heads: int, head_size: int,
                           block_size: int, max_seq_len: int, num_selected: int,
                           partition_size: int, device=None, stream=None) -> torch.Tensor:
    """A zeroed workspace for pa_select_blocks and pa_sparse_forward."""
    n = pa_sparse_workspace_bytes(num_rows, num_heads, num_kv_heads, head_size, block_size,
                                  max_seq_len, num_selected, partition_size)
    if n == 0:
        raise ValueError("bad sizes for a sparse workspace")
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    pa_workspace_init(ws, stream)
    return ws


def _sparse_shapes(selected, query, key_bounds, block_tables, seq_lens, q_start, hkv):
    R, H, D = query.shape
    B = seq_lens.numel()
    if q_start is not None and q_start.numel() != B + 1:
        raise ValueError("q_start must be int32 [num_seqs + 1]")
    if block_tables.dim() != 2 or block_tables.shape[0] != B:
        raise ValueError("block_tables must be int32 [num_seqs, max_blocks_per_seq]")
    if selected is not None and (selected.dim() != 3 or selected.shape[:2] != (R, hkv)):
        raise ValueError("selected must be int32 [rows, num_kv_heads, num_selected]")
    if key_bounds is not None and (key_bounds.dim() != 4 or key_bounds.shape[1:] != (hkv, 2, D)):
        raise ValueError("key_bounds must be [num_blocks, num_kv_heads, 2, head_size]")
    return R, H, D, B


def pa_select_blocks(selected, query, key_bounds, block_tables, seq_lens, block_size: int,
                     partition_size, workspace, sink_blocks=0, recent_blocks=1, q_start=None,
                     max_seq_len=None, stream=None) -> None:
    """Choose the blocks that each (row, KV head) attends to from the pages' key
    bounds into selected, int32 [rows, Hkv, num_selected] (see include/pa.h)."""
    nb, hkv = key_bounds.shape[:2]
    ws, q, kb, sel, bt, sl, qs = _pointers(query, workspace, (query, key_bounds),
                                           (selected, block_tables, seq_lens, q_start))
    R, H, D, B = _sparse_shapes(selected, query, key_bounds, block_tables, seq_lens, q_start, hkv)
    if max_seq_len is None:
        max_seq_len = block_tables.shape[1] * block_size
    _check((_lib or load_library()).pa_select_blocks(
        sel, q, kb, bt, sl, qs, B, R, H, hkv, D, nb, block_size, block_tables.shape[1],
        int(max_seq_len), selected.shape[2], sink_blocks, recent_blocks, int(partition_size),
        _DTYPES[query.dtype], ws, workspace.numel() * workspace.element_size(),
        _stream_handle(stream)), "pa_select_blocks")


def pa_sparse_forward(out, selected, query, key_cache, value_cache, block_tables, seq_lens, scale,
                      partition_size, workspace, key_bounds=None, num_selected=None,
                      sink_blocks=0, recent_blocks=1, q_start=None, max_seq_len=None,
                      stream=None) -> None:
    """Attention over selected blocks (see include/pa.h): with key_bounds they
    are selected in the call and written to `selected` (None: not wanted, give
    num_selected); without, `selected` is read."""
    nb, hkv, bs, D = key_cache.shape
    ws, o, q, kc, vc, kb, sel, bt, sl, qs = _pointers(
        query, workspace, (out, query, key_cache, value_cache, key_bounds),
        (selected, block_tables, seq_lens, q_start))
    R, H, D2, B = _sparse_shapes(selected, query, key_bounds, block_tables, seq_lens, q_start, hkv)
    if out.shape != query.shape or D2 != D or value_cache.shape != key_cache.shape \
            or (kb and key_bounds.shape[0] != nb):
        raise ValueError("query and out, or the caches and their bounds, differ in shape")
    if selected is not None:
        if num_selected not in (None, selected.shape[2]):
            raise ValueError("num_selected differs from selected's last dimension")
        num_selected = selected.shape[2]
    elif num_selected is None:
        raise ValueError("num_selected or a selected tensor is needed")
    blocks = block_tables.shape[1]
    if max_seq_len is None:
        max_seq_len = blocks * bs
    _check((_lib or load_library()).pa_sparse_forward(
        o, sel, q, kc, vc, kb, bt, sl, qs, B, R, H, hkv, D, nb, bs, blocks,
        int(max_seq_len), int(num_selected), sink_blocks, recent_blocks, float(scale),
        int(partition_size), _DTYPES[query.dtype], ws,
        workspace.numel() * workspace.element_size(), _stream_handle(stream)), "pa_sparse_forward")


def pa_q4_workspace_bytes(head_size: int) -> int:
    return int(load_library().pa_q4_workspace_bytes(head_size))


def alloc_q4_workspace(head_size: int, device=None, stream=None) -> torch.Tensor:
    """A zeroed workspace for pa_q4_forward calls of any batch."""
    n = pa_q4_workspace_bytes(head_size)
    if n == 0:
        raise ValueError("bad head size for a 4-bit workspace")
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    pa_workspace_init(ws, stream)
    return ws


def alloc_q4_cache(num_blocks: int, num_kv_heads: int, block_size: int, head_size: int, device=None):
    """(codes, scales) of an empty cache in 4 bits, for keys or for values: uint8
    [num_blocks, Hkv, block_size, D / 2] and float16 [num_blocks, Hkv, block_size,
    D / 64, 2]."""
    shape = (num_blocks, num_kv_heads, block_size)
    return (torch.zeros(*shape, head_size // 2, dtype=torch.uint8, device=device or "cuda"),
            torch.zeros(*shape, head_size // 64, 2, dtype=torch.float16, device=device or "cuda"))


def _q4_shapes(key_cache, value_cache, key_scales, value_scales, block_tables, seq_lens, q_start, head_size):
    nb, hkv, bs, half = key_cache.shape
    if value_cache.shape != key_cache.shape or half * 2 != head_size:
        raise ValueError("key_cache and value_cache must be [num_blocks, num_kv_heads, block_size, "
                         "head_size / 2]")
    if key_scales.shape != (nb, hkv, bs, head_size // 64, 2) or value_scales.shape != key_scales.shape:
        raise ValueError("key_scales and value_scales must be [num_blocks, num_kv_heads, block_size, "
                         "head_size / 64, 2]")
    B = seq_lens.numel()
    if q_start is not None and q_start.numel() != B + 1:
        raise ValueError("q_start must be int32 [num_seqs + 1]")
    if block_tables.dim() != 2 or block_tables.shape[0] != B:
        raise ValueError("block_tables must be int32 [num_seqs, max_blocks_per_seq]")
    return nb, hkv, bs, B


def pa_q4_append(key_cache, value_cache, key_scales, value_scales, key, value, block_tables,
                 seq_lens, workspace, query=None, query_out=None, key_out=None, value_out=None,
                 cos_sin=None, positions=None, q_start=None, rotary_dim=None, interleaved=False,
                 max_seq_len=None, stream=None) -> None:
    """Append key / value [rows, Hkv, D] (rows may be strided slices) to a cache in
    4 bits: key_cache, value_cache uint8 [num_blocks, Hkv, block_size, D / 2],
    key_scales, value_scales float16 [num_blocks, Hkv, block_size, D / 64, 2] (see
    include/pa.h).  Keys and query are rotated as by pa_append_kv; key_out and
    value_out [rows, Hkv, D] receive the values that the cache then holds."""
    if key.dim() != 3:
        raise ValueError("key must be [rows, num_kv_heads, head_size]")
    D = key.shape[2]
    ws, qo, ko, vo, bt, sl, qs, pos, kc, vc, ks, vs = _pointers(
        key, workspace, (query_out, key_out, value_out), (block_tables, seq_lens, q_start, positions),
        (torch.uint8, (key_cache, value_cache)), (torch.float16, (key_scales, value_scales)))
    nb, hkv, bs, B = _q4_shapes(key_cache, value_cache, key_scales, value_scales, block_tables,
                                seq_lens, q_start, D)
    kp, kst, R = _rows(key, key, hkv, D)
    vp, vst, rows = _rows(value, key, hkv, D)
    if rows != R or any(t is not None and t.shape != (R, hkv, D) for t in (key_out, value_out)):
        raise ValueError("key and value (and key_out, value_out) differ in shape")
    if pos and positions.numel() != R:
        raise ValueError("positions must be int32 [rows]")
    H, qp, qst = hkv, 0, 0
    if query is not None:
        if query.dim() != 3 or query_out is None or query_out.shape != query.shape:
            raise ValueError("query and query_out must both be [rows, num_heads, head_size]")
        H = query.shape[1]
        qp, qst, rows = _rows(query, key, H, D)
        if rows != R:
            raise ValueError("query and query_out must both be [rows, num_heads, head_size]")
    elif query_out is not None:
        raise ValueError("query_out without a query")
    cs, max_position, rotary_dim = _angles(cos_sin, key, rotary_dim)
    blocks = block_tables.shape[1]
    if max_seq_len is None:
        max_seq_len = blocks * bs
    _packed(_Q4_APPEND, "pa_q4_append",
            kc, vc, ks, vs, qo, ko, vo, qp, kp, vp, qst, kst, vst, cs, pos, bt, sl, qs, B, R, H, hkv,
            D, nb, bs, blocks, max_seq_len, rotary_dim, interleaved, max_position,
            _DTYPES[key.dtype], ws, workspace.nbytes, _stream_handle(stream))


def pa_q4_forward(out, query, key_cache, value_cache, key_scales, value_scales, block_tables,
                  seq_lens, scale, workspace, q_start=None, max_seq_len=None, stream=None) -> None:
    """Decode attention over a cache in 4 bits (pa_q4_append's), one query row a
    sequence or, with q_start, chunks of them as in pa_chunks_forward (see
    include/pa.h)."""
    R, H, D = query.shape
    ws, o, q, bt, sl, qs, kc, vc, ks, vs = _pointers(
        query, workspace, (out, query), (block_tables, seq_lens, q_start),
        (torch.uint8, (key_cache, value_cache)), (torch.float16, (key_scales, value_scales)))
    nb, hkv, bs, B = _q4_shapes(key_cache, value_cache, key_scales, value_scales, block_tables,
                                seq_lens, q_start, D)
    if out.shape != query.shape:
        raise ValueError("query and out differ in shape")
    blocks = block_tables.shape[1]
    if max_seq_len is None:
        max_seq_len = blocks * bs
    _packed(_Q4_FORWARD, "pa_q4_forward",
            o, q, kc, vc, ks, vs, bt, sl, qs, B, R, H, hkv, D, nb, bs, blocks, max_seq_len, scale,
            _DTYPES[query.dtype], ws, workspace.nbytes, _stream_handle(stream))


def pa_latent_workspace_bytes(latent_dim: int) -> int:
    return int(load_library().pa_latent_workspace_bytes(latent_dim))


def alloc_latent_workspace(latent_dim: int, device=None, stream=None) -> torch.Tensor:
    """A zeroed workspace for pa_latent_forward calls of any batch."""
    n = pa_latent_workspace_bytes(latent_dim)
    if n == 0:
        raise ValueError("bad latent_dim for a latent workspace")
    ws = torch.empty(n, dtype=torch.uint8, device=device or "cuda")
    pa_workspace_init(ws, stream)
    return ws


def _latent_part(t, like, width: int):
    """(pointer, elements between rows, rows) of a [rows, width] tensor whose rows are
    contiguous, of the dtype and on the device of `like`."""
    if t.dim() != 2 or t.shape[1] != width or t.stride(1) != 1 or t.dtype is not like.dtype \
            or t.get_device() != like.get_device():
        raise ValueError(f"expected [rows, {width}] of the cache's dtype and device, rows contiguous")
    return t.data_ptr(), t.stride(0) if t.shape[0] > 1 else width, t.shape[0]


def _latent_shapes(cache, block_tables, seq_lens, q_start):
    nb, bs, width = cache.shape
    B = seq_lens.numel()
    if q_start is not None and q_start.numel() != B + 1:
        raise ValueError("q_start must be int32 [num_seqs + 1]")
    if block_tables.dim() != 2 or block_tables.shape[0] != B:
        raise ValueError("block_tables must be int32 [num_seqs, max_blocks_per_seq]")
    return nb, bs, width, B


def pa_latent_append(cache, latent, rope_key, block_tables, seq_lens, workspace, cos_sin,
                     query=None, query_rope=None, norm_weight=None, eps=0.0, positions=None,
                     q_start=None, interleaved=False, max_seq_len=None, stream=None) -> None:
    """Append rows to a cache of shared latents [num_blocks, block_size, latent_dim +
    rope_dim]: latent [rows, latent_dim], normalised with norm_weight and eps, and
    rope_key [rows, rope_dim], rotated by cos_sin [max_position, rope_dim]; query_rope
    [rows, H, rope_dim] (rows and heads may be strided; query[..., latent_dim:] itself
    too) is rotated into the last rope_dim elements of query [rows, H, latent_dim +
    rope_dim] (see include/pa.h)."""
    if latent.dim() != 2:
        raise ValueError("latent must be [rows, latent_dim]")
    nb, bs, width, B = _latent_shapes(cache, block_tables, seq_lens, q_start)
    ws, c, q, nw, bt, sl, qs, pos = _pointers(
        cache, workspace, (cache, query, norm_weight), (block_tables, seq_lens, q_start, positions))
    lat = latent.shape[1]
    rope = width - lat
    lp, lst, R = _latent_part(latent, cache, lat)
    kp, kst, rows = _latent_part(rope_key, cache, rope)
    if rows != R or (nw and norm_weight.numel() != lat):
        raise ValueError("latent and rope_key (and norm_weight) differ in shape")
    if pos and positions.numel() != R:
        raise ValueError("positions must be int32 [rows]")
    H, qp, qst, qhst = 1, 0, 0, 0
    if (query is None) != (query_rope is None):
        raise ValueError("query and query_rope go together")
    if query is not None:
        if query.dim() != 3 or query.shape[0] != R or query.shape[2] != width:
            raise ValueError("query must be [rows, num_heads, latent_dim + rope_dim]")
        H = query.shape[1]
        if query_rope.shape != (R, H, rope) or query_rope.stride(2) != 1 \
                or query_rope.dtype is not cache.dtype or query_rope.get_device() != cache.get_device():
            raise ValueError("query_rope must be [rows, num_heads, rope_dim] of the cache's dtype and "
                             "device, heads contiguous")
        qp = query_rope.data_ptr()
        qhst = query_rope.stride(1) if H > 1 else rope
        qst = query_rope.stride(0) if R > 1 else (H - 1) * qhst + rope
    cs, max_position, rotary = _angles(cos_sin, cache, None)
    if rotary != rope:
        raise ValueError("cos_sin must be float32 [max_position, rope_dim]")
    blocks = block_tables.shape[1]
    if max_seq_len is None:
        max_seq_len = blocks * bs
    _packed(_LATENT_APPEND, "pa_latent_append",
            c, q, qp, lp, kp, nw, eps, qst, qhst, lst, kst, cs, pos, bt, sl, qs, B, R, H, lat, rope,
            nb, bs, blocks, max_seq_len, interleaved, max_position, _DTYPES[cache.dtype], ws,
            workspace.nbytes, _stream_handle(stream))


def pa_latent_forward(out, query, cache, block_tables, seq_lens, scale, workspace, q_start=None,
                      max_seq_len=None, stream=None, debug_flags=0, wait_limit_ns=0) -> None:
    """Decode attention over a cache of shared latents in the absorbed form: query
    [rows, H, latent_dim + rope_dim], out [rows, H, latent_dim]; one row a sequence or,
    with q_start, chunks of them as in pa_chunks_forward (see include/pa.h)."""
    R, H, width = query.shape
    nb, bs, W, B = _latent_shapes(cache, block_tables, seq_lens, q_start)
    ws, o, q, c, bt, sl, qs = _pointers(query, workspace, (out, query, cache),
                                        (block_tables, seq_lens, q_start))
    if W != width or out.dim() != 3 or out.shape[:2] != (R, H) or out.shape[2] > width:
        raise ValueError("query must be [rows, num_heads, latent_dim + rope_dim], out [rows, "
                         "num_heads, latent_dim]")
    lat = out.shape[2]
    blocks = block_tables.shape[1]
    if max_seq_len is None:
        max_seq_len = blocks * bs
    opts = pa_options_t(0, 0, 0, debug_flags, wait_limit_ns, None, 0, 0, 0) \
        if debug_flags or wait_limit_ns else None
    _packed(_LATENT_FORWARD, "pa_latent_forward",
            o, q, c, bt, sl, qs, B, R, H, lat, width - lat, nb, bs, blocks, max_seq_len, scale,
            _DTYPES[query.dtype], ws, workspace.nbytes, _stream_handle(stream),
            ctypes.addressof(opts) if opts is not None else 0)


def pa_host_staging_bytes(num_seqs: int, num_heads: int, head_size: int,
                          max_blocks_per_seq: int, dtype) -> int:
    """Device bytes pa_forward_host stages the per-step data in."""
    code = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return int(load_library().pa_host_staging_bytes(num_seqs, num_heads, head_size,
                                                    max_blocks_per_seq, code))


def alloc_staging(query, block_tables, device=None) -> torch.Tensor:
    """A device staging buffer for pa_forward_host calls of this shape."""
    B, H, D = query.shape
    n = pa_host_staging_bytes(B, H, D, block_tables.shape[1], query.dtype)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device or "cuda")


def pa_forward_host(out_host, query_host, key_cache, value_cache, block_tables_host,
                    seq_lens_host, scale, partition_size, staging, workspace, max_seq_len=None,
                    stream=None, variant=PA_VARIANT_AUTO, math=PA_MATH_AUTO, num_stages=0,
                    ctas_per_sm=0, fuse_partitions=0) -> None:
    """pa_forward with the query, block tables, lengths and output in host
    memory (pinned for asynchronous copies): one C-ABI call enqueues the
    host-to-device copies into ``staging``, the kernels and the copy of the
    output back to ``out_host``.  Synchronise the stream before reading it."""
    for t in (out_host, query_host, block_tables_host, seq_lens_host):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError("pa_forward_host takes contiguous host tensors for "
                             "out, query, block_tables and seq_lens")
    opts = pa_options_t(variant, math, num_stages, 0, 0, None, ctas_per_sm, fuse_partitions)
    args = _fwd_args(out_host, query_host, key_cache, value_cache, block_tables_host,
                     seq_lens_host, scale, partition_size, workspace, max_seq_len, stream)
    _check(load_library().pa_forward_host(
        *args[:17], _ptr(staging), staging.numel() * staging.element_size(), *args[17:],
        ctypes.byref(opts)), "pa_forward_host")


def pa_choose_v2(num_seqs: int, num_kv_heads: int, max_seq_len: int, partition_size: int,
                 sm_count: int) -> int:
    return int(load_library().pa_choose_v2(num_seqs, num_kv_heads, max_seq_len,
                                           partition_size, sm_count))


def pa_choose_v2_chunks(num_seqs: int, num_heads: int, num_kv_heads: int, head_size: int,
                        max_chunk: int, max_seq_len: int, partition_size: int,
                        sm_count: int) -> int:
    return int(load_library().pa_choose_v2_chunks(num_seqs, num_heads, num_kv_heads, head_size,
                                                  max_chunk, max_seq_len, partition_size,
                                                  sm_count))


def pa_read_device_status(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise the stream, return and clear the kernels' status word."""
    return int(load_library().pa_read_device_status(_ptr(workspace), _stream_handle(stream)))


def pa_status_string(status: int) -> str:
    return status_text(status)


def pa_last_cuda_error() -> str:
    return load_library().pa_last_cuda_error().decode()


def pa_version() -> int:
    return int(load_library().pa_version())
