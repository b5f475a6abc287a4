"""Thin Python binding of the C ABI in include/jetlong.h (argument marshalling
only: every step of the attention runs in the CUDA library).

The names match the C entry points.  Tensors are torch CUDA tensors; the call
is enqueued on the current torch stream (or ``stream``).  A non-OK status
raises :class:`JetLongError` carrying ``jl_last_error()``.  There is no CPU
fallback: if ``libjetlong.so`` is missing, the first call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libjetlong.so")

JL_OK, JL_ERR_INVALID_ARG, JL_ERR_UNSUPPORTED, JL_ERR_CUDA, JL_ERR_WORKSPACE = range(5)
JL_BF16, JL_FP32 = 0, 1
JL_FLAG_PLAIN_CAUSAL = 0x1
JL_FLAG_SIMT = 0x2
JL_FLAG_PREROTATE_K = 0x4
JL_FLAG_ROTATE = 0x8

_lib = None


class JetLongError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{status_string(status) if _lib else status}: {msg}")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libjetlong.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with `python -m zero_shot_rope_b200.build` "
            "(there is no CPU fallback)")
    L = ctypes.CDLL(LIB_PATH)
    c_i32, c_i64, c_u32, c_sz, c_p, c_d = (ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32,
                                           ctypes.c_size_t, ctypes.c_void_p, ctypes.c_double)
    L.jl_status_string.restype = ctypes.c_char_p
    L.jl_status_string.argtypes = [ctypes.c_int]
    L.jl_last_error.restype = ctypes.c_char_p
    L.jl_last_error.argtypes = []
    L.jl_version.restype = ctypes.c_char_p
    L.jl_version.argtypes = []
    L.jl_group_size.restype = ctypes.c_int
    L.jl_group_size.argtypes = [c_i64, c_i64, ctypes.POINTER(c_i64)]
    L.jl_bifocal_prefill_workspace_size.restype = c_sz
    L.jl_bifocal_prefill_workspace_size.argtypes = [c_i32, c_i32, c_i32, c_i32, c_i32, ctypes.c_int, c_u32]
    L.jl_bifocal_prefill.restype = ctypes.c_int
    L.jl_bifocal_prefill.argtypes = [c_p, c_p, c_p, c_p, c_p, c_p, c_i32, c_i32, c_i32, c_i32, c_i32,
                                     c_i32, c_i64, c_i32, c_d, ctypes.c_int, c_u32, c_p, c_sz, c_p]
    L.jl_bifocal_prefill_kv.restype = ctypes.c_int
    L.jl_bifocal_prefill_kv.argtypes = [c_p, c_p, c_p, c_p, c_p, c_p, c_p, c_i32, c_i32, c_i32, c_i32, c_i32,
                                        c_i32, c_i32, c_i64, c_i32, c_i32, c_d, ctypes.c_int, c_u32, c_p, c_sz,
                                        c_p]
    L.jl_bifocal_decode_workspace_size.restype = c_sz
    L.jl_bifocal_decode_workspace_size.argtypes = [c_i32, c_i32, c_i32, c_i32, c_i32]
    L.jl_bifocal_decode.restype = ctypes.c_int
    L.jl_bifocal_decode.argtypes = [c_p, c_p, c_p, c_p, c_i32, c_i32, c_i32, c_i32, c_i32, c_i32, c_i64,
                                    c_i32, c_d, c_p, c_p, c_p, c_sz, ctypes.c_int, c_u32, c_p]
    L.jl_bifocal_decode_window.restype = ctypes.c_int
    L.jl_bifocal_decode_window.argtypes = [c_p, c_p, c_p, c_p, c_i32, c_i32, c_i32, c_i32, c_i32, c_i32, c_i64,
                                           c_i32, c_i32, c_d, c_p, c_p, c_p, c_sz, ctypes.c_int, c_u32, c_p]
    L.jl_bifocal_decode_noalloc.restype = ctypes.c_int
    L.jl_bifocal_decode_noalloc.argtypes = [c_p, c_p, c_p, c_p, c_i32, c_i32, c_i32, c_i32, c_i32, c_i32,
                                            c_i64, c_i32, c_d, c_p, c_p, ctypes.c_int, c_u32, c_p]
    L.jl_bifocal_decode_noalloc_error.restype = ctypes.c_int
    L.jl_bifocal_decode_noalloc_error.argtypes = [ctypes.POINTER(c_i32), c_p]
    L.jl_paged_append.restype = ctypes.c_int
    L.jl_paged_append.argtypes = ([c_p] * 6 + [c_i64, c_i32, c_p, c_p] + [c_i32] * 8 +
                                  [c_i64, c_p, c_p, c_d, ctypes.c_int, c_u32, c_p])
    L.jl_bifocal_select_pages_workspace_size.restype = c_sz
    L.jl_bifocal_select_pages_workspace_size.argtypes = [c_i32] * 4
    L.jl_bifocal_select_pages.restype = ctypes.c_int
    L.jl_bifocal_select_pages.argtypes = ([c_p] * 3 + [c_i64, c_i32, c_p] + [c_i32] * 9 +
                                          [c_i64, c_i32, c_d, c_p, c_p, c_sz, ctypes.c_int, c_u32, c_p])
    L.jl_bifocal_decode_paged_workspace_size.restype = c_sz
    L.jl_bifocal_decode_paged_workspace_size.argtypes = [c_i32] * 2
    L.jl_bifocal_decode_paged.restype = ctypes.c_int
    L.jl_bifocal_decode_paged.argtypes = ([c_p] * 4 + [c_i64, c_i32, c_p, c_p] + [c_i32] * 7 +
                                          [c_i64, c_i64, c_i32, c_i32, c_d, c_p, c_p, c_p, c_sz, ctypes.c_int,
                                           c_u32, c_p])
    L.jl_paged_call.restype = ctypes.c_int
    L.jl_paged_call.argtypes = [c_i32, ctypes.c_char_p, c_i32]
    L.jl_debug_set_wait_limit.restype = ctypes.c_int
    L.jl_debug_set_wait_limit.argtypes = [ctypes.c_ulonglong]
    _lib = L
    return L


def status_string(s: int) -> str:
    return lib().jl_status_string(int(s)).decode()


def last_error() -> str:
    return lib().jl_last_error().decode()


def _check(status: int):
    if status != JL_OK:
        raise JetLongError(status, last_error())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return JL_BF16
    if t.dtype == torch.float32:
        return JL_FP32
    raise TypeError(f"unsupported dtype {t.dtype}")


def jl_group_size(L: int, w_pretrained: int) -> int:
    g = ctypes.c_int64(0)
    _check(lib().jl_group_size(int(L), int(w_pretrained), ctypes.byref(g)))
    return int(g.value)


def jl_bifocal_prefill_workspace_size(batch, total_tokens, n_q_heads, n_kv_heads, head_dim,
                                      dtype=torch.bfloat16, flags=0) -> int:
    code = JL_BF16 if dtype == torch.bfloat16 else JL_FP32
    return int(lib().jl_bifocal_prefill_workspace_size(batch, total_tokens, n_q_heads, n_kv_heads,
                                                       head_dim, code, flags))


def jl_bifocal_decode_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, max_seqlen) -> int:
    return int(lib().jl_bifocal_decode_workspace_size(batch, n_q_heads, n_kv_heads, head_dim, max_seqlen))


def _workspace(nbytes, device, workspace):
    if nbytes == 0:
        return None
    if workspace is not None:
        return workspace
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def jl_bifocal_prefill(q, k, v, cu_seqlens, max_seqlen, w_pretrained, w0, rope_theta, out=None,
                       lse=None, flags=0, workspace=None, stream=None):
    """Causal GQA prefill with Dynamic Bifocal RoPE over packed sequences.

    q [T, Hq, D], k/v [T, Hkv, D] (standard-RoPE q and k), cu_seqlens int32
    [B+1] on the device.  Returns (out [T, Hq, D], lse [Hq, T] or None).
    """
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    B = cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty_like(q)
    ws_bytes = jl_bifocal_prefill_workspace_size(B, T, Hq, Hkv, D, q.dtype, flags)
    ws = _workspace(ws_bytes, q.device, workspace)
    _check(lib().jl_bifocal_prefill(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(cu_seqlens),
                                    B, T, int(max_seqlen), Hq, Hkv, D, int(w_pretrained), int(w0),
                                    float(rope_theta), _dtype_code(q), int(flags), _ptr(ws),
                                    0 if ws is None else ws.numel() * ws.element_size(),
                                    _stream(stream)))
    return out, lse


def jl_bifocal_prefill_kv(q, k, v, cu_seqlens_q, cu_seqlens_k, max_seqlen_q, w_pretrained, w0, rope_theta,
                          out=None, lse=None, flags=0, workspace=None, stream=None, window=0):
    """Prefill of new tokens against keys that include an existing cache:
    sequence s has its Lq queries at the last positions of its Lk keys.
    ``window`` > 0: sliding-window layer (keys at distance >= window hidden).

    q [Tq, Hq, D]; k, v [Tk, Hkv, D]; cu_seqlens_q / cu_seqlens_k int32 [B+1]
    on the device.  Returns (out [Tq, Hq, D], lse [Hq, Tq] or None).
    """
    Tq, Hq, D = q.shape
    Tk, Hkv = k.shape[0], k.shape[1]
    B = cu_seqlens_q.numel() - 1
    if out is None:
        out = torch.empty_like(q)
    ws_bytes = jl_bifocal_prefill_workspace_size(B, Tk, Hq, Hkv, D, q.dtype, flags)
    ws = _workspace(ws_bytes, q.device, workspace)
    _check(lib().jl_bifocal_prefill_kv(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(cu_seqlens_q),
                                       _ptr(cu_seqlens_k), B, Tq, Tk, int(max_seqlen_q), Hq, Hkv, D,
                                       int(w_pretrained), int(w0), int(window), float(rope_theta), _dtype_code(q),
                                       int(flags),
                                       _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                       _stream(stream)))
    return out, lse


def jl_bifocal_decode(q, k_cache, v_cache, seqlens, max_seqlen, w_pretrained, w0, rope_theta,
                      out=None, lse=None, flags=0, workspace=None, stream=None):
    """One decode step: q [B, Hq, D] at position L_b - 1 against the cache
    [B, Lcap, Hkv, D] (rows 0 .. L_b - 1).  Returns (out [B, Hq, D], lse)."""
    B, Hq, D = q.shape
    Lcap, Hkv = k_cache.shape[1], k_cache.shape[2]
    if out is None:
        out = torch.empty_like(q)
    ws_bytes = jl_bifocal_decode_workspace_size(B, Hq, Hkv, D, int(max_seqlen))
    ws = _workspace(ws_bytes, q.device, workspace)
    _check(lib().jl_bifocal_decode(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens), B, Lcap,
                                   int(max_seqlen), Hq, Hkv, D, int(w_pretrained), int(w0),
                                   float(rope_theta), _ptr(out), _ptr(lse), _ptr(ws),
                                   0 if ws is None else ws.numel() * ws.element_size(),
                                   _dtype_code(q), int(flags), _stream(stream)))
    return out, lse


def jl_bifocal_decode_window(q, k_cache, v_cache, seqlens, max_seqlen, w_pretrained, w0, window, rope_theta,
                             out=None, lse=None, flags=0, workspace=None, stream=None):
    """jl_bifocal_decode for a sliding-window layer: the new query attends to
    the last ``window`` keys of its sequence (0: all keys)."""
    B, Hq, D = q.shape
    Lcap, Hkv = k_cache.shape[1], k_cache.shape[2]
    if out is None:
        out = torch.empty_like(q)
    ws_bytes = jl_bifocal_decode_workspace_size(B, Hq, Hkv, D, int(max_seqlen))
    ws = _workspace(ws_bytes, q.device, workspace)
    _check(lib().jl_bifocal_decode_window(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens), B, Lcap,
                                          int(max_seqlen), Hq, Hkv, D, int(w_pretrained), int(w0), int(window),
                                          float(rope_theta), _ptr(out), _ptr(lse), _ptr(ws),
                                          0 if ws is None else ws.numel() * ws.element_size(),
                                          _dtype_code(q), int(flags), _stream(stream)))
    return out, lse


JL_DECODE_NOALLOC_SCRATCH_BYTES = 4 << 20


def jl_bifocal_decode_noalloc(q, k_cache, v_cache, seqlens, max_seqlen, w_pretrained, w0, rope_theta,
                              out, lse=None, flags=0, stream=None):
    """jl_bifocal_decode for callers that cannot allocate device memory: the
    library supplies the scratch from a fixed array in its device image
    (JL_DECODE_NOALLOC_SCRATCH_BYTES), so ``out`` must be given and nothing
    is allocated.  Calls that overlap on the GPU share that array and race."""
    B, Hq, D = q.shape
    Lcap, Hkv = k_cache.shape[1], k_cache.shape[2]
    _check(lib().jl_bifocal_decode_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(seqlens), B, Lcap,
                                           int(max_seqlen), Hq, Hkv, D, int(w_pretrained), int(w0),
                                           float(rope_theta), _ptr(out), _ptr(lse), _dtype_code(q), int(flags),
                                           _stream(stream)))
    return out, lse


def jl_bifocal_decode_noalloc_error(stream=None) -> int:
    """The kernel error word of the last jl_bifocal_decode_noalloc call (0: no
    error).  Enqueues the copy on ``stream`` and synchronises it."""
    word = ctypes.c_int32(-1)
    st = _stream(stream)
    _check(lib().jl_bifocal_decode_noalloc_error(ctypes.byref(word), st))
    (stream or torch.cuda.current_stream()).synchronize()
    return int(word.value)


# ------------------------------------------------------------- paged cache
# The paged calls also check shapes, types, strides and devices here (the C
# ABI sees pointers only), run on the device of their tensors whichever is
# current, and allocate what the caller did not pass on the stream they run on.
# A generation step makes three of them per layer, so what they do on the host
# is kept short: one expression checks the usual case, everything contiguous, and
# only where it does not hold is each tensor looked at by itself.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_I32 = torch.int32

# the argument words of jl_paged_call; the packed form costs a fifth of a
# foreign call with as many arguments
_APPEND = struct.Struct("=21qd3q")
_SELECT = struct.Struct("=17qd6q")
_DECODE = struct.Struct("=19qd7q")


def _paged_call(call, words):
    status = (_lib or lib()).jl_paged_call(call, words, len(words) // 8)
    if status:
        _check(status)


def _plain(t, dtype, index):
    return t.dtype is dtype and t.get_device() == index and t.is_contiguous()


def _fits(t, shape, dtype, index):
    return t.shape == shape and t.dtype is dtype and t.get_device() == index and t.is_contiguous()


def _misfit(name, t, shape, dtype, device):
    """Raise for a tensor that is not a contiguous one of this shape, type and
    device."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)} (got {list(t.shape)})")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    raise ValueError(f"{name} must be contiguous")


def _tensor(name, t, shape, dtype, like):
    if not _fits(t, shape, dtype, like.get_device()):
        _misfit(name, t, shape, dtype, like.device)


def _pools(k_pages, v_pages, n_kv_heads, head_dim, like):
    """(page size, pages, stride between pages) of the two pools."""
    shape, dtype, index = k_pages.shape, like.dtype, like.get_device()
    if len(shape) != 4 or shape != v_pages.shape or shape[2] != n_kv_heads or shape[3] != head_dim:
        raise ValueError(f"k_pages and v_pages must both be [n_pages, page_size, {n_kv_heads}, {head_dim}] "
                         f"(got {list(k_pages.shape)}, {list(v_pages.shape)})")
    n, page = shape[0], shape[1]
    whole = page * n_kv_heads * head_dim
    if n > 0 and _fits(k_pages, shape, dtype, index) and _fits(v_pages, shape, dtype, index):
        return page, n, whole
    if k_pages.dtype != dtype or v_pages.dtype != dtype:
        raise TypeError(f"k_pages and v_pages must be {dtype} (got {k_pages.dtype}, {v_pages.dtype})")
    if k_pages.device != like.device or v_pages.device != like.device:
        raise ValueError(f"k_pages and v_pages must be on {like.device}")
    if n == 0:
        raise ValueError("the pools have no page")
    if not (k_pages[0].is_contiguous() and v_pages[0].is_contiguous()):
        raise ValueError("each page of k_pages and v_pages must be contiguous")
    if n == 1:
        return page, n, whole
    if k_pages.stride(0) != v_pages.stride(0):
        raise ValueError("k_pages and v_pages must have the same stride between pages")
    return page, n, k_pages.stride(0)


def _table(block_table, batch, like):
    """(pages per sequence, row stride) of the block table."""
    shape = block_table.shape
    if len(shape) != 2 or shape[0] != batch:
        raise ValueError(f"block_table must have shape [{batch}, max_pages] (got {list(shape)})")
    cols = shape[1]
    if _fits(block_table, shape, torch.int32, like.get_device()):
        return cols, cols
    if block_table.dtype != torch.int32:
        raise TypeError(f"block_table must be torch.int32 (got {block_table.dtype})")
    if block_table.device != like.device:
        raise ValueError(f"block_table is on {block_table.device}, expected {like.device}")
    if cols > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table's rows must be contiguous")
    return cols, (block_table.stride(0) if batch > 1 else cols)


def _heads3(name, t):
    if t.dim() != 3:
        raise ValueError(f"{name} must have three dimensions (got {list(t.shape)})")
    return t.shape


def _scratch(workspace, nbytes, like):
    """(tensor, pointer, bytes) of the workspace; the tensor keeps it alive."""
    if nbytes == 0:
        return None, 0, 0
    if workspace is None:
        workspace = like.new_empty(nbytes, dtype=torch.uint8)
        return workspace, workspace.data_ptr(), nbytes
    if workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {like.device}")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _elsewhere(t, stream):
    """The context that makes t's device, and ``stream`` if there is one,
    current."""
    if not t.is_cuda:
        return contextlib.nullcontext()
    if stream is None:
        return torch.cuda.device(t.device)
    if stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, tensors on {t.device}")
    return torch.cuda.stream(stream)


def _no_host_tensor(t, index):
    if index < 0:
        raise ValueError(f"tensors must be on a CUDA device (got {t.device})")


def _stream_of(index):
    if _raw_stream is not None:
        return _raw_stream(index)
    return torch.cuda.current_stream(index).cuda_stream


def jl_paged_append(k, v, k_pages, v_pages, block_table, cu_seqlens, seqlens, max_new, page_summary=None, q=None,
                    q_out=None, rope_theta=None, stream=None):
    """Write new tokens into a paged cache: k, v [T, Hkv, D], sequence b's rows
    cu_seqlens[b] .. cu_seqlens[b+1] - 1, the last at position seqlens[b] - 1.

    With ``rope_theta`` k (and q [T, Hq, D], if given) arrive before RoPE and
    are rotated by their positions; without it k is stored as given.
    ``max_new``, from 1 to T, is at least every sequence's number of new tokens.
    ``page_summary`` [n_pages, Hkv, 2, D], if given, is kept up to date.
    Returns the rotated q (``q_out``; it may be q itself) or None."""
    index = k.get_device()
    if stream is not None or (index >= 0 and index != _raw_device()):
        with _elsewhere(k, stream):
            return jl_paged_append(k, v, k_pages, v_pages, block_table, cu_seqlens, seqlens, max_new, page_summary, q,
                                   q_out, rope_theta)
    shape = k.shape
    T, Hkv, D = shape if len(shape) == 3 else _heads3("k", k)
    dtype = k.dtype
    code = _dtype_code(k)
    B = seqlens.numel()
    pool, table = k_pages.shape, block_table.shape
    summary = q_in = q_to = 0
    Hq = Hkv
    if q is not None:
        if rope_theta is None:
            raise ValueError("q is only rotated: it needs rope_theta")
        Hq = _heads3("q", q)[1]
    elif q_out is not None:
        raise ValueError("q_out without q")
    if (len(pool) == 4 and pool[0] > 0 and pool[2] == Hkv and pool[3] == D and len(table) == 2 and table[0] == B
            and k.is_contiguous() and _fits(v, shape, dtype, index) and _plain(k_pages, dtype, index)
            and _fits(v_pages, pool, dtype, index) and _plain(block_table, _I32, index)
            and _fits(cu_seqlens, (B + 1,), _I32, index) and _fits(seqlens, (B,), _I32, index)):
        n_pages, page, cols = pool[0], pool[1], table[1]
        page_stride, table_stride = page * Hkv * D, cols
    else:
        _tensor("k", k, shape, dtype, k)
        _tensor("v", v, shape, dtype, k)
        page, n_pages, page_stride = _pools(k_pages, v_pages, Hkv, D, k)
        cols, table_stride = _table(block_table, B, k)
        _tensor("cu_seqlens", cu_seqlens, (B + 1,), _I32, k)
        _tensor("seqlens", seqlens, (B,), _I32, k)
    if page_summary is not None:
        _tensor("page_summary", page_summary, (n_pages, Hkv, 2, D), dtype, k)
        summary = page_summary.data_ptr()
    if q is not None:
        _tensor("q", q, (T, Hq, D), dtype, k)
        if q_out is not None:
            _tensor("q_out", q_out, (T, Hq, D), dtype, k)
    _no_host_tensor(k, index)
    if q is not None:
        if q_out is None:
            q_out = torch.empty_like(q)
        q_in, q_to = q.data_ptr(), q_out.data_ptr()
    theta, flags = (0.0, 0) if rope_theta is None else (rope_theta, JL_FLAG_ROTATE)
    _paged_call(0, _APPEND.pack(
        k.data_ptr(), v.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), summary, block_table.data_ptr(),
        table_stride, cols, cu_seqlens.data_ptr(), seqlens.data_ptr(), B, T, max_new, Hq, Hkv, D, page, n_pages,
        page_stride, q_in, q_to, theta, code, flags, _stream_of(index)))
    return q_out


@functools.lru_cache(maxsize=256)
def jl_bifocal_select_pages_workspace_size(batch, n_kv_heads, max_pages, n_select) -> int:
    return int(lib().jl_bifocal_select_pages_workspace_size(batch, n_kv_heads, max_pages, n_select))


def jl_bifocal_select_pages(q, page_summary, block_table, seqlens, page_size, n_select, w_pretrained, w0, rope_theta,
                            n_first=1, n_last=1, out=None, flags=0, workspace=None, stream=None):
    """The logical pages that each new token should read: the ``n_first``
    first, the ``n_last`` newest and the highest scored others of every kv
    head, ascending, -1 behind the last: int32 [B, Hkv, n_select], for
    jl_bifocal_decode_paged.  q [B, Hq, D] at position seqlens[b] - 1."""
    index = q.get_device()
    if stream is not None or (index >= 0 and index != _raw_device()):
        with _elsewhere(q, stream):
            return jl_bifocal_select_pages(q, page_summary, block_table, seqlens, page_size, n_select, w_pretrained,
                                           w0, rope_theta, n_first, n_last, out, flags, workspace)
    shape = q.shape
    B, Hq, D = shape if len(shape) == 3 else _heads3("q", q)
    dtype = q.dtype
    code = _dtype_code(q)
    if page_summary.dim() != 4:
        raise ValueError(f"page_summary must be [n_pages, Hkv, 2, D] (got {list(page_summary.shape)})")
    n_pages, Hkv = page_summary.shape[:2]
    n_select = int(n_select)
    table = block_table.shape
    if (len(table) == 2 and table[0] == B and q.is_contiguous()
            and _fits(page_summary, (n_pages, Hkv, 2, D), dtype, index) and _plain(block_table, _I32, index)
            and _fits(seqlens, (B,), _I32, index)):
        cols = table_stride = table[1]
    else:
        _tensor("q", q, shape, dtype, q)
        _tensor("page_summary", page_summary, (n_pages, Hkv, 2, D), dtype, q)
        cols, table_stride = _table(block_table, B, q)
        _tensor("seqlens", seqlens, (B,), _I32, q)
    if out is not None:
        _tensor("out", out, (B, Hkv, n_select), torch.int32, q)
    _no_host_tensor(q, index)
    if out is None:
        out = q.new_empty((B, Hkv, max(n_select, 0)), dtype=torch.int32)
    keep, ws, ws_bytes = _scratch(workspace, jl_bifocal_select_pages_workspace_size(B, Hkv, cols, n_select), q)
    _paged_call(1, _SELECT.pack(
        q.data_ptr(), page_summary.data_ptr(), block_table.data_ptr(), table_stride, cols, seqlens.data_ptr(),
        B, Hq, Hkv, D, page_size, n_pages, n_select, n_first, n_last, w_pretrained, w0, rope_theta, out.data_ptr(), ws,
        ws_bytes, code, flags, _stream_of(index)))
    return out


@functools.lru_cache(maxsize=256)
def jl_bifocal_decode_paged_workspace_size(batch, head_dim) -> int:
    return int(lib().jl_bifocal_decode_paged_workspace_size(batch, head_dim))


def jl_bifocal_decode_paged(q, k_pages, v_pages, block_table, seqlens, w_pretrained, w0, rope_theta, page_list=None,
                            window=0, out=None, lse=None, flags=0, workspace=None, stream=None):
    """One decode step over a paged cache: q [B, Hq, D] at position
    seqlens[b] - 1 against the pages of block_table [B, max_pages]; only those
    of ``page_list`` [B, Hkv, n] if given, only the last ``window`` keys if
    not 0.  Returns (out [B, Hq, D], lse [B, Hq] or None)."""
    index = q.get_device()
    if stream is not None or (index >= 0 and index != _raw_device()):
        with _elsewhere(q, stream):
            return jl_bifocal_decode_paged(q, k_pages, v_pages, block_table, seqlens, w_pretrained, w0, rope_theta,
                                           page_list, window, out, lse, flags, workspace)
    shape = q.shape
    B, Hq, D = shape if len(shape) == 3 else _heads3("q", q)
    dtype = q.dtype
    code = _dtype_code(q)
    pool, table = k_pages.shape, block_table.shape
    if len(pool) != 4:
        raise ValueError(f"k_pages must be [n_pages, page_size, Hkv, D] (got {list(pool)})")
    Hkv = pool[2]
    if (pool[0] > 0 and pool[3] == D and len(table) == 2 and table[0] == B and q.is_contiguous()
            and _plain(k_pages, dtype, index) and _fits(v_pages, pool, dtype, index)
            and _plain(block_table, _I32, index) and _fits(seqlens, (B,), _I32, index)):
        n_pages, page, cols = pool[0], pool[1], table[1]
        page_stride, table_stride = page * Hkv * D, cols
    else:
        _tensor("q", q, shape, dtype, q)
        page, n_pages, page_stride = _pools(k_pages, v_pages, Hkv, D, q)
        cols, table_stride = _table(block_table, B, q)
        _tensor("seqlens", seqlens, (B,), _I32, q)
    listed, n_list = 0, 0
    if page_list is not None:
        n_list = page_list.shape[-1] if page_list.dim() == 3 else 0
        _tensor("page_list", page_list, (B, Hkv, n_list), torch.int32, q)
        # an empty list's own pointer may be null: nothing of it is read
        listed = page_list.data_ptr() or block_table.data_ptr()
    lse_to = 0
    if lse is not None:
        _tensor("lse", lse, (B, Hq), torch.float32, q)
        lse_to = lse.data_ptr()
    if out is not None:
        _tensor("out", out, shape, dtype, q)
    _no_host_tensor(q, index)
    if out is None:
        out = torch.empty_like(q)
    keep, ws, ws_bytes = _scratch(workspace, jl_bifocal_decode_paged_workspace_size(B, D), q)
    _paged_call(2, _DECODE.pack(
        q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(), table_stride, cols,
        seqlens.data_ptr(), listed, n_list, B, Hq, Hkv, D, page, n_pages, page_stride, w_pretrained, w0, window,
        rope_theta, out.data_ptr(), lse_to, ws, ws_bytes, code, flags, _stream_of(index)))
    return out, lse
