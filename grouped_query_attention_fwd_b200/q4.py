"""The 4-bit KV cache: append, read back and attention over it.

Argument marshalling over the C ABI of ``include/gqa.h`` ("4-bit cache"), which
defines the record that a token's K or V row of one head becomes:

    cache = torch.zeros(B, Hkv, capacity, q4_record_bytes(D), dtype=torch.uint8, device="cuda")

Calls with arguments of sizes and strides already seen reuse the checked
problem descriptor of the first such call; pointers are taken anew each time.
Each call in a captured graph has a workspace of its own, which every replay
clears: a caller who wants ``device_status`` after replays passes a workspace.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import threading

from . import (GQA_DTYPE_BF16, GQA_DTYPE_F16, GQA_OK, WORKSPACE_HEAD_BYTES, GQAError, Plan,
               Problem, _lens_ptr, _lib, _offset, _stream_object, _table, _torch, _workspaces,
               make_problem, workspace_for)

_vp = ctypes.c_void_p


class Q4RowsDesc(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32), ("advance", ctypes.c_int32),
        ("batch", ctypes.c_int64), ("heads_kv", ctypes.c_int64), ("capacity", ctypes.c_int64),
        ("head_dim", ctypes.c_int64), ("n", ctypes.c_int64),
        ("cache_k_stride", ctypes.c_int64 * 4), ("cache_v_stride", ctypes.c_int64 * 4),
        ("k_stride", ctypes.c_int64 * 4), ("v_stride", ctypes.c_int64 * 4),
        ("counts", _vp), ("starts", _vp), ("start", ctypes.c_int64),
        ("block_table", _vp), ("block_table_stride", ctypes.c_int64),
        ("page_size", ctypes.c_int64), ("num_pages", ctypes.c_int64),
    ]


_lib.gqa_q4_record_bytes.argtypes = [ctypes.c_int64]
_lib.gqa_q4_record_bytes.restype = ctypes.c_int64
_lib.gqa_kv_append_q4.argtypes = [ctypes.POINTER(Q4RowsDesc), _vp, _vp, _vp, _vp, _vp, _vp,
                                  ctypes.c_size_t, _vp]
_lib.gqa_kv_append_q4.restype = ctypes.c_int
_lib.gqa_kv_read_q4.argtypes = [ctypes.POINTER(Q4RowsDesc), _vp, _vp, _vp, _vp, _vp, _vp,
                                ctypes.c_size_t, _vp]
_lib.gqa_kv_read_q4.restype = ctypes.c_int
_lib.gqa_query_q4.argtypes = [ctypes.POINTER(Problem), ctypes.c_int, ctypes.POINTER(Plan)]
_lib.gqa_query_q4.restype = ctypes.c_int
_lib.gqa_forward_q4.argtypes = [ctypes.POINTER(Problem), _vp, _vp, _vp, _vp, _vp, _vp,
                                ctypes.c_size_t, _vp]
_lib.gqa_forward_q4.restype = ctypes.c_int

# Checked descriptors, per thread (a call writes its pointers into the one it
# uses).  The key is everything that the checks look at: types, devices, sizes,
# strides of every tensor, never an address, and the scalars as plain numbers
# (a 0-d tensor is one by its value, not by its identity).
_seen = threading.local()
_MAX_SEEN = 1024


def _known(kind):
    seen = getattr(_seen, kind, None)
    if seen is None:
        seen = {}
        setattr(_seen, kind, seen)
    return seen


def _remember(seen, key, value):
    if len(seen) >= _MAX_SEEN:
        seen.clear()
    seen[key] = value
    return value


def _like(t):
    """What the checks see of a tensor."""
    return t.dtype, t.shape, t.stride(), t.get_device()


def _ptr(t):
    return None if t is None else t.data_ptr()


# torch's functions that every call needs (filled in by the first call: torch is
# imported no earlier than a tensor exists).
_device_now = _stream_now = _capturing = None


def _bind_torch():
    global _device_now, _stream_now, _capturing
    c = _torch()._C
    _device_now, _stream_now = c._cuda_getDevice, c._cuda_getCurrentRawStream
    _capturing = c._cuda_isCurrentStreamCapturing


def q4_record_bytes(head_dim: int) -> int:
    """Bytes of one token's K (or V) row of one head in a 4-bit cache."""
    n = _lib.gqa_q4_record_bytes(int(head_dim))
    if n == 0:
        raise ValueError("a 4-bit cache needs a head dim that is a multiple of 8, at most 128")
    return n


def _half(dtype) -> int:
    torch = _torch()
    if dtype is torch.bfloat16:
        return GQA_DTYPE_BF16
    if dtype is torch.float16:
        return GQA_DTYPE_F16
    raise TypeError("a 4-bit cache serves bfloat16 and float16, got %s" % dtype)


def _check_caches(cache_k, cache_v):
    torch = _torch()
    if cache_k.dtype is not torch.uint8 or cache_v.dtype is not torch.uint8 or cache_k.dim() != 4:
        raise TypeError("a 4-bit cache is a uint8 tensor [B, Hkv, capacity, record], or a pool "
                        "[num_pages, Hkv, page_size, record]")
    if cache_k.shape != cache_v.shape:
        raise ValueError("the K and V caches must have one shape")


def _check_devices(idx, *tensors):
    if idx < 0:
        raise ValueError("the 4-bit cache takes CUDA tensors only (there is no CPU path)")
    for t in tensors:
        if t is not None and t.get_device() != idx:
            raise ValueError("all tensors must be on the same CUDA device")


def _elsewhere(idx, stream):
    """Contexts that make device ``idx`` and ``stream`` current, or None where
    they are (the usual case)."""
    if _device_now is None:
        _bind_torch()
    if idx < 0 or (_device_now() == idx and
                   (stream is None or int(stream) == _stream_now(idx))):
        return None
    torch = _torch()
    stack = contextlib.ExitStack()
    stack.enter_context(torch.cuda.device(idx))
    if stream is not None:
        stack.enter_context(torch.cuda.stream(_stream_object(idx, stream)))
    return stack


def _workspace(idx, stream, nbytes, workspace):
    """The caller's workspace, the cached one of the current stream, or, in a
    capture, one that belongs to the graph alone (zeroed by each replay):
    graphs replayed side by side never share one."""
    if workspace is not None:
        return workspace
    if _capturing():
        torch = _torch()
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=torch.device("cuda", idx))
        ws[:WORKSPACE_HEAD_BYTES].zero_()
        return ws
    ws = _workspaces.get((idx, stream))
    if ws is None or ws.numel() < nbytes:
        ws = workspace_for(_torch().device("cuda", idx), nbytes, stream)
    return ws


# ------------------------------------------------------------ append and read back

def _rows_desc(dtype, cache_k, cache_v, k, v, D, table, advance):
    B, Hkv, n, Dk = k.shape
    if tuple(v.shape) != tuple(k.shape) or Dk != D or cache_k.shape[1] != Hkv:
        raise ValueError("k and v rows must be [B, Hkv, n, D] with the cache's heads")
    if cache_k.shape[3] != q4_record_bytes(D):
        raise ValueError("head dim %d has records of %d bytes, the cache's are %d"
                         % (D, q4_record_bytes(D), cache_k.shape[3]))
    d = Q4RowsDesc()
    d.dtype, d.advance = _half(dtype), int(advance)
    d.batch, d.heads_kv, d.head_dim, d.n = B, Hkv, D, n
    if table is None:
        if cache_k.shape[0] != B:
            raise ValueError("the cache and the rows must have one batch size")
        d.capacity = cache_k.shape[2]
    else:
        d.num_pages, d.page_size = cache_k.shape[0], cache_k.shape[2]
        d.capacity = table.shape[1] * d.page_size
        d.block_table_stride = table.stride(0)
    for i in range(4):
        d.cache_k_stride[i], d.cache_v_stride[i] = cache_k.stride(i), cache_v.stride(i)
        d.k_stride[i], d.v_stride[i] = k.stride(i), v.stride(i)
    return d


def _check_int32(t, B, name):
    if t is not None and (t.dtype is not _torch().int32 or tuple(t.shape) != (B,) or
                          not t.is_contiguous()):
        raise ValueError("%s must be a contiguous int32 CUDA tensor of shape [B]" % name)


def kv_append_q4(cache_k, cache_v, k_new, v_new, kv_lens, new_lens=None, advance=True,
                 workspace=None, stream=None, block_table=None):
    """Quantise k_new / v_new [B, Hkv, n, D] (bf16 or fp16) into rows kv_lens[b] + t
    of the 4-bit caches [B, Hkv, capacity, q4_record_bytes(D)] (uint8), or of
    page pools [num_pages, Hkv, page_size, record] with ``block_table``.

    new_lens (int32 CUDA [B]): entry b has new_lens[b] <= n new rows (a padded
    batch).  advance: add the new rows to kv_lens (int32 CUDA [B]) in place;
    False leaves it, for layers that share one tensor of lengths.  An entry
    that does not fit is left as it was and device_status() reports
    GQA_ERR_KV_LENGTH."""
    idx = k_new.get_device()
    away = _elsewhere(idx, stream)
    if away is not None:
        with away:
            return kv_append_q4(cache_k, cache_v, k_new, v_new, kv_lens, new_lens, advance,
                                workspace, None, block_table)
    advance = bool(advance)
    key = (_like(k_new), _like(v_new), _like(cache_k), _like(cache_v), _like(kv_lens),
           None if new_lens is None else _like(new_lens),
           None if block_table is None else _like(block_table), advance)
    seen = _known("append")
    d = seen.get(key)
    if d is None:
        _check_devices(idx, v_new, kv_lens, cache_k, cache_v, new_lens, block_table)
        _check_caches(cache_k, cache_v)
        if k_new.dim() != 4 or v_new.dtype is not k_new.dtype:
            raise TypeError("k_new and v_new must be [B, Hkv, n, D] of one type")
        B = k_new.shape[0]
        if block_table is not None:
            _table(block_table, B)
        _check_int32(new_lens, B, "new_lens")
        _check_int32(kv_lens, B, "kv_lens")
        d = _remember(seen, key, _rows_desc(k_new.dtype, cache_k, cache_v, k_new, v_new,
                                            k_new.shape[3], block_table, advance))
    d.block_table = _ptr(block_table)
    d.counts = _ptr(new_lens)
    handle = _stream_now(idx)
    ws = _workspace(idx, handle, 256, workspace)
    rc = _lib.gqa_kv_append_q4(d, cache_k.data_ptr(), cache_v.data_ptr(), k_new.data_ptr(),
                               v_new.data_ptr(), kv_lens.data_ptr(), ws.data_ptr(), ws.numel(),
                               handle)
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_kv_append_q4")


def kv_read_q4(cache_k, cache_v, head_dim, dtype, kv_lens=None, start=0, n=None, out_k=None,
               out_v=None, workspace=None, stream=None, block_table=None):
    """Rows start .. start + n of the 4-bit caches as 16-bit (k, v) [B, Hkv, n, D].

    dtype: the type the cache was written with (and of the result).  start: an
    int, or an int32 CUDA tensor [B].  n defaults to the rest of the capacity.
    Rows at or past kv_lens[b] (the capacity without it) are zeros."""
    torch = _torch()
    idx = cache_k.get_device()
    away = _elsewhere(idx, stream)
    if away is not None:
        with away:
            return kv_read_q4(cache_k, cache_v, head_dim, dtype, kv_lens, start, n, out_k, out_v,
                              workspace, None, block_table)
    starts = start if isinstance(start, torch.Tensor) else None
    start = 0 if starts is not None else int(start)
    head_dim, n = int(head_dim), None if n is None else int(n)
    key = (dtype, head_dim, n, start if n is None else None, _like(cache_k), _like(cache_v),
           None if kv_lens is None else _like(kv_lens), None if starts is None else _like(starts),
           None if out_k is None else _like(out_k), None if out_v is None else _like(out_v),
           None if block_table is None else _like(block_table))
    seen = _known("read")
    known = seen.get(key)
    if known is None:
        _check_devices(idx, cache_v, kv_lens, starts, out_k, out_v, block_table)
        _check_caches(cache_k, cache_v)
        B, Hkv, capacity, _ = cache_k.shape
        if block_table is not None:
            B = block_table.shape[0]
            _table(block_table, B)
            capacity *= block_table.shape[1]
        _check_int32(starts, B, "start")
        _check_int32(kv_lens, B, "kv_lens")
        count = n if n is not None else capacity - start
        if count < 0:
            raise ValueError("n must not be negative")
        shape = (B, Hkv, count, head_dim)
        for t in (out_k, out_v):
            if t is not None and (t.shape != shape or t.dtype is not dtype):
                raise ValueError("out_k and out_v must be [B, Hkv, n, D] of the given type")
        fresh = torch.empty(shape, dtype=dtype, device="meta")
        known = _remember(seen, key, (shape, _rows_desc(
            dtype, cache_k, cache_v, fresh if out_k is None else out_k,
            fresh if out_v is None else out_v, shape[3], block_table, False)))
    shape, d = known
    k, v = out_k, out_v
    if k is None:
        k = torch.empty(shape, dtype=dtype, device=cache_k.device)
    if v is None:
        v = torch.empty_like(k) if out_k is None else torch.empty(shape, dtype=dtype,
                                                                  device=cache_k.device)
    d.block_table = _ptr(block_table)
    d.starts = _ptr(starts)
    d.start = start
    handle = _stream_now(idx)
    ws = _workspace(idx, handle, 256, workspace)
    rc = _lib.gqa_kv_read_q4(d, cache_k.data_ptr(), cache_v.data_ptr(), k.data_ptr(),
                             v.data_ptr(), _ptr(kv_lens), ws.data_ptr(), ws.numel(), handle)
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_kv_read_q4")
    return k, v


# ------------------------------------------------------------ attention

def q4_problem_for(q, cache_k, cache_v, mask=None, causal=False, scale=None, out=None,
                   causal_offset=None, window=0, kv_lens=None, block_table=None) -> Problem:
    """The C descriptor of a forward_q4 call (k and v strides in bytes)."""
    if q.dim() != 4:
        raise ValueError("q must be 4-D [B, Hq, Sq, D]")
    B, Hq, Sq, D = q.shape
    dtype = _half(q.dtype)
    if cache_k.shape[3] != q4_record_bytes(D):
        raise ValueError("head dim %d has records of %d bytes, the cache's are %d"
                         % (D, q4_record_bytes(D), cache_k.shape[3]))
    Hkv, Sk = cache_k.shape[1], cache_k.shape[2]
    if block_table is not None:
        num_pages, page_size = cache_k.shape[0], Sk
        bt_ptr, bt_stride, per_seq = _table(block_table, B)
        Sk = per_seq * page_size
    elif cache_k.shape[0] != B:
        raise ValueError("the cache must have q's batch size")
    if out is not None and (tuple(out.shape) != tuple(q.shape) or out.dtype is not q.dtype):
        raise ValueError("out must have q's shape and type")
    ost = out.stride() if out is not None else (Hq * Sq * D, Sq * D, D, 1)
    mst = None
    if mask is not None:
        if tuple(mask.shape) != (B, Sq, Sk):
            raise ValueError("mask must be [B, Sq, Sk]")
        mst = mask.stride()
    if scale is None:
        scale = 1.0 / math.sqrt(D) if D > 0 else 1.0
    p = make_problem(dtype, B, Hq, Hkv, Sq, Sk, D, q.stride(), cache_k.stride(),
                     cache_v.stride(), ost, mst, causal=causal, scale=scale,
                     causal_offset=_offset(causal, causal_offset, Sq, Sk), window=window,
                     kv_lens_ptr=None if kv_lens is None else _lens_ptr(kv_lens, B))
    if block_table is not None:
        p.block_table, p.block_table_stride = bt_ptr, bt_stride
        p.page_size, p.num_pages = page_size, num_pages
    return p


def _query(p, sm_count=0) -> Plan:
    plan = Plan()
    rc = _lib.gqa_query_q4(ctypes.byref(p), int(sm_count), ctypes.byref(plan))
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_query_q4")
    return plan


def query_q4(q, cache_k, cache_v, mask=None, causal=False, scale=None, sm_count: int = 0,
             causal_offset=None, window=0, kv_lens=None, block_table=None) -> dict:
    """What forward_q4 will do with these arguments (see ``query``)."""
    return _query(q4_problem_for(q, cache_k, cache_v, mask, causal, scale,
                                 causal_offset=causal_offset, window=window, kv_lens=kv_lens,
                                 block_table=block_table), sm_count).as_dict()


def forward_q4(q, cache_k, cache_v, mask=None, causal=False, scale=None, out=None,
               workspace=None, stream=None, causal_offset=None, window=0, kv_lens=None,
               block_table=None):
    """``forward`` with k and v in 4-bit caches [B, Hkv, Sk, q4_record_bytes(D)]
    (uint8; page pools [num_pages, Hkv, page_size, record] with block_table).
    q and the result are bf16 or fp16, the type the cache was written with;
    every other argument is ``forward``'s."""
    torch = _torch()
    idx = q.get_device()
    away = _elsewhere(idx, stream)
    if away is not None:
        with away:
            return forward_q4(q, cache_k, cache_v, mask, causal, scale, out, workspace, None,
                              causal_offset, window, kv_lens, block_table)
    causal, window = bool(causal), int(window)
    scale = None if scale is None else float(scale)
    if causal_offset is not None and not isinstance(causal_offset, str):
        causal_offset = int(causal_offset)
    key = (_like(q), _like(cache_k), _like(cache_v), None if mask is None else _like(mask),
           None if kv_lens is None else _like(kv_lens),
           None if block_table is None else _like(block_table),
           None if out is None else _like(out), causal, scale, causal_offset, window)
    seen = _known("forward")
    known = seen.get(key)
    if known is None:
        _check_devices(idx, cache_k, cache_v, mask, kv_lens, block_table, out)
        _check_caches(cache_k, cache_v)
        if mask is not None and mask.dtype not in (torch.bool, torch.uint8):
            raise TypeError("mask must be bool or uint8")
        _check_int32(kv_lens, q.shape[0], "kv_lens")
        p = q4_problem_for(q, cache_k, cache_v, mask, causal, scale, out, causal_offset, window,
                           kv_lens, block_table)
        known = _remember(seen, key, (p, _query(p).workspace_bytes, q.is_contiguous()))
    p, nbytes, contiguous = known
    if out is None:  # [B, Hq, Sq, D] laid out afresh, whatever q's strides
        out = torch.empty_like(q) if contiguous else torch.empty(q.shape, dtype=q.dtype,
                                                                 device=q.device)
    p.kv_lens = _ptr(kv_lens)
    p.block_table = _ptr(block_table)
    handle = _stream_now(idx)
    ws = _workspace(idx, handle, nbytes, workspace)
    rc = _lib.gqa_forward_q4(p, q.data_ptr(), cache_k.data_ptr(), cache_v.data_ptr(), _ptr(mask),
                             out.data_ptr(), ws.data_ptr(), ws.numel(), handle)
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_forward_q4")
    return out
