"""The 4-bit KV cache: append, read back and attention over it.

Argument marshalling over the C ABI of ``include/gqa.h`` ("4-bit cache"), which
defines the record that a token's K or V row of one head becomes:

    cache = torch.zeros(B, Hkv, capacity, q4_record_bytes(D), dtype=torch.uint8, device="cuda")

Calls with arguments of sizes and strides already seen reuse the checked
problem descriptor of the first such call; pointers are taken anew each time.
"""
from __future__ import annotations

import ctypes
import math
import threading

from . import (GQA_DTYPE_BF16, GQA_DTYPE_F16, GQA_OK, GQAError, Plan, Problem, _lens_ptr, _lib,
               _offset, _stream_object, _table, _torch, make_problem, workspace_for)

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

# Checked descriptors by sizes, strides and scalars (never by address), per
# thread: a call writes its pointers into the descriptor it uses.
_seen = threading.local()
_MAX_SEEN = 1024


def _remember(kind, key, make):
    seen = _seen.__dict__.setdefault(kind, {})
    got = seen.get(key)
    if got is None:
        if len(seen) >= _MAX_SEEN:
            seen.clear()
        got = seen[key] = make()
    return got


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


def _check_caches(cache_k, cache_v, device):
    torch = _torch()
    for c in (cache_k, cache_v):
        if c.dtype is not torch.uint8 or c.dim() != 4:
            raise TypeError("a 4-bit cache is a uint8 tensor [B, Hkv, capacity, record], or a "
                            "pool [num_pages, Hkv, page_size, record]")
        if c.device != device:
            raise ValueError("all tensors must be on the same CUDA device")
    if cache_k.shape != cache_v.shape:
        raise ValueError("the K and V caches must have one shape")


def _same_device(device, *tensors):
    if device.type != "cuda":
        raise ValueError("the 4-bit cache takes CUDA tensors only (there is no CPU path)")
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError("all tensors must be on the same CUDA device")


class _On:
    """Makes a device and the stream of a call current (nothing to do where they are)."""

    def __init__(self, device, stream):
        torch = _torch()
        self.idx = device.index
        self.contexts = []
        if torch.cuda.current_device() != self.idx:
            self.contexts.append(torch.cuda.device(self.idx))
        cur = torch.cuda.current_stream(self.idx)
        self.stream = cur.cuda_stream
        if stream is not None and int(stream) != self.stream:
            self.contexts.append(torch.cuda.stream(_stream_object(self.idx, stream)))
            self.stream = int(stream)

    def __enter__(self):
        for c in self.contexts:
            c.__enter__()
        return self

    def __exit__(self, *exc):
        for c in reversed(self.contexts):
            c.__exit__(*exc)
        return False


_HEAD = 256 + 65536  # error word, append ticket and decode tickets: what has to start at zero


def _workspace(on, nbytes, workspace):
    """The caller's workspace, the cached one of the stream, or, in a capture,
    one that belongs to the graph alone (zeroed by each replay): graphs
    replayed side by side never share one."""
    if workspace is not None:
        return workspace
    torch = _torch()
    if torch.cuda.is_current_stream_capturing():
        ws = torch.empty(max(nbytes, 256), dtype=torch.uint8,
                         device=torch.device("cuda", on.idx))
        ws[:_HEAD].zero_()
        return ws
    return workspace_for(torch.device("cuda", on.idx), nbytes, on.stream)


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


def _int32(t, B, name):
    torch = _torch()
    if t.dtype is not torch.int32 or tuple(t.shape) != (B,) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 CUDA tensor of shape [B]" % name)
    return t.data_ptr()


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
    device = k_new.device
    _same_device(device, v_new, kv_lens, new_lens, block_table)
    _check_caches(cache_k, cache_v, device)
    if k_new.dim() != 4 or v_new.dtype is not k_new.dtype:
        raise TypeError("k_new and v_new must be [B, Hkv, n, D] of one type")
    B = k_new.shape[0]
    bt = _table(block_table, B)[0] if block_table is not None else None
    key = (k_new.dtype, k_new.shape, k_new.stride(), v_new.shape, v_new.stride(), cache_k.shape,
           cache_k.stride(), cache_v.stride(), bool(advance),
           None if bt is None else (block_table.shape, block_table.stride(0)))
    d = _remember("append", key, lambda: _rows_desc(
        k_new.dtype, cache_k, cache_v, k_new, v_new, k_new.shape[3], block_table, advance))
    d.block_table = bt
    d.counts = None if new_lens is None else _int32(new_lens, B, "new_lens")
    lens = _int32(kv_lens, B, "kv_lens")
    with _On(device, stream) as on:
        ws = _workspace(on, 256, workspace)
        rc = _lib.gqa_kv_append_q4(d, cache_k.data_ptr(), cache_v.data_ptr(), k_new.data_ptr(),
                                   v_new.data_ptr(), lens, ws.data_ptr(), ws.numel(), on.stream)
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_kv_append_q4")


def kv_read_q4(cache_k, cache_v, head_dim, dtype, kv_lens=None, start=0, n=None, out_k=None,
               out_v=None, workspace=None, stream=None, block_table=None):
    """Rows start .. start + n of the 4-bit caches as 16-bit (k, v) [B, Hkv, n, D].

    dtype: the type the cache was written with (and of the result).  start: an
    int, or an int32 CUDA tensor [B].  n defaults to the rest of the capacity.
    Rows at or past kv_lens[b] (the capacity without it) are zeros."""
    torch = _torch()
    device = cache_k.device
    starts = start if isinstance(start, torch.Tensor) else None
    _same_device(device, kv_lens, starts, out_k, out_v, block_table)
    _check_caches(cache_k, cache_v, device)
    B = cache_k.shape[0]
    bt = None
    capacity = cache_k.shape[2]
    if block_table is not None:
        B = block_table.shape[0]
        bt = _table(block_table, B)[0]
        capacity *= block_table.shape[1]
    if n is None:
        n = capacity - (0 if starts is not None else int(start))
    if n < 0:
        raise ValueError("n must not be negative")
    shape = (B, cache_k.shape[1], int(n), int(head_dim))
    with _On(device, stream) as on:
        outs = []
        for t in (out_k, out_v):
            if t is None:
                t = torch.empty(shape, dtype=dtype, device=device)
            elif tuple(t.shape) != shape or t.dtype is not dtype:
                raise ValueError("out_k and out_v must be [B, Hkv, n, D] of the given type")
            outs.append(t)
        k, v = outs
        key = (dtype, shape, k.stride(), v.stride(), cache_k.shape, cache_k.stride(),
               cache_v.stride(), None if bt is None else (block_table.shape, block_table.stride(0)))
        d = _remember("read", key, lambda: _rows_desc(
            dtype, cache_k, cache_v, k, v, shape[3], block_table, False))
        d.block_table = bt
        d.starts = None if starts is None else _int32(starts, B, "start")
        d.start = 0 if starts is not None else int(start)
        lens = None if kv_lens is None else _int32(kv_lens, B, "kv_lens")
        ws = _workspace(on, 256, workspace)
        rc = _lib.gqa_kv_read_q4(d, cache_k.data_ptr(), cache_v.data_ptr(), k.data_ptr(),
                                 v.data_ptr(), lens, ws.data_ptr(), ws.numel(), on.stream)
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
    device = q.device
    _same_device(device, mask, kv_lens, block_table, out)
    _check_caches(cache_k, cache_v, device)
    if mask is not None:
        if mask.dtype is torch.bool:
            mask = mask.view(torch.uint8)
        elif mask.dtype is not torch.uint8:
            raise TypeError("mask must be bool or uint8")
    with _On(device, stream) as on:
        if out is None:
            # q's shape, laid out afresh: [B, Hq, Sq, D] contiguous
            out = torch.empty(q.shape, dtype=q.dtype, device=device)
        key = (q.dtype, q.shape, q.stride(), out.shape, out.dtype, out.stride(), cache_k.shape,
               cache_k.stride(), cache_v.stride(),
               None if mask is None else (mask.shape, mask.stride()), bool(causal), scale,
               causal_offset, window, kv_lens is None, on.idx,
               None if block_table is None else (block_table.shape, block_table.stride(0)))

        def make():
            p = q4_problem_for(q, cache_k, cache_v, mask, causal, scale, out, causal_offset,
                               window, kv_lens, block_table)
            return p, _query(p).workspace_bytes

        p, nbytes = _remember("forward", key, make)
        p.kv_lens = None if kv_lens is None else _int32(kv_lens, q.shape[0], "kv_lens")
        p.block_table = None if block_table is None else _table(block_table, q.shape[0])[0]
        ws = _workspace(on, nbytes, workspace)
        rc = _lib.gqa_forward_q4(p, q.data_ptr(), cache_k.data_ptr(), cache_v.data_ptr(),
                                 mask.data_ptr() if mask is not None else None, out.data_ptr(),
                                 ws.data_ptr(), ws.numel(), on.stream)
    if rc != GQA_OK:
        raise GQAError(rc, "gqa_forward_q4")
    return out
