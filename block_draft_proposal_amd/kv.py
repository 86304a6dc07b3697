"""Binding of the paged KV cache and the draft-tree attention
(``include/dflash_kv.h``): argument marshalling only, as in ``binding``.

Functions have the names of the C entry points, take torch tensors on one GPU
and enqueue on the current stream of that GPU (or on ``stream``)."""
from __future__ import annotations

import contextlib
import ctypes
from typing import Optional

import torch

from . import binding as _b
from .binding import _c_f32, _c_i32, _c_i64, _c_size, _c_vp

DFLASH_E4M3 = 2
DFLASH_I8 = 3
CACHE_DTYPES = {torch.bfloat16: _b.DFLASH_BF16, torch.float8_e4m3fn: DFLASH_E4M3, torch.int8: DFLASH_I8}


class KVCacheStruct(ctypes.Structure):
    """Mirror of dflash_kv_cache."""
    _fields_ = [
        ("k", _c_vp), ("v", _c_vp), ("k_scale", _c_vp), ("v_scale", _c_vp),
        ("page_stride", _c_i64), ("scale_page_stride", _c_i64), ("n_pages", _c_i64),
        ("page_size", _c_i32), ("n_kv_heads", _c_i32), ("head_dim", _c_i32), ("dtype", _c_i32),
    ]


class KVBatchStruct(ctypes.Structure):
    """Mirror of dflash_kv_batch."""
    _fields_ = [
        ("page_table", _c_vp), ("table_stride", _c_i64), ("table_width", _c_i32), ("n_req", _c_i32),
        ("start", _c_vp), ("offsets", _c_vp), ("n_rows", _c_i64),
    ]


_P_CACHE, _P_BATCH = ctypes.POINTER(KVCacheStruct), ctypes.POINTER(KVBatchStruct)
_SIGNATURES = {
    "dflash_kv_write": (_c_i32, [_P_CACHE, _P_BATCH, _c_vp, _c_i64, _c_i64, _c_vp, _c_i64, _c_i64, _c_i32, _c_vp]),
    "dflash_kv_read": (_c_i32, [_P_CACHE, _P_BATCH, _c_vp, _c_vp, _c_i32, _c_vp]),
    "dflash_kv_commit": (_c_i32, [_P_CACHE, _P_BATCH, _c_vp, _c_i64, _c_i32, _c_vp, _c_vp]),
    "dflash_tree_attention_workspace_size": (_c_size, [_P_CACHE, _c_i32, _c_i32, _c_i32]),
    "dflash_tree_attention": (_c_i32, [_P_CACHE, _P_BATCH, _c_vp, _c_i64, _c_i64, _c_i32, _c_vp, _c_i32, _c_i32,
                                       _c_f32, _c_i32, _c_vp, _c_vp, _c_size, _c_vp]),
}
EXPORTED = tuple(_SIGNATURES)

_lib = None


def _fns():
    global _lib
    if _lib is None:
        handle = _b.lib()
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
    return _lib


def _int32(x: int, name: str) -> int:
    """ctypes cuts a number to its field's 32 bits without a word."""
    if not -0x80000000 <= x <= 0x7FFFFFFF:
        raise ValueError(f"{name} = {x} does not fit 32 bits")
    return x


class KVCache:
    """A cache over tensors the caller owns.  k, v [n_pages, n_kv_heads,
    page_size, head_dim] in bf16, float8_e4m3fn or int8, each page contiguous
    and both with the same page stride (so K and V may be two slices of one
    pool); k_scale, v_scale uint8 [n_pages, n_kv_heads, page_size] for the
    8-bit types, likewise.  The object only describes the tensors; make it
    once and pass it to every call."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.dtype not in CACHE_DTYPES:
            raise ValueError("k and v must be [n_pages, n_kv_heads, page_size, head_dim] of one cache type")
        n_pages, n_kv_heads, page_size, head_dim = k.shape
        if n_pages < 1:
            raise ValueError("a cache has at least one page")
        for name, n in (("n_kv_heads", n_kv_heads), ("page_size", page_size), ("head_dim", head_dim)):
            _int32(n, name)
        scaled = k.dtype != torch.bfloat16
        if scaled != (k_scale is not None) or scaled != (v_scale is not None):
            raise ValueError("k_scale and v_scale belong to the 8-bit caches, and both to those")
        tensors = [k, v] + ([k_scale, v_scale] if scaled else [])
        for t in tensors:
            if t.device != k.device or not t.is_cuda:
                raise ValueError("the cache's tensors must be on one GPU")
            if not t[0].is_contiguous():
                raise ValueError("every page must be contiguous")
        if scaled:
            for t in (k_scale, v_scale):
                if t.dtype != torch.uint8 or tuple(t.shape) != (n_pages, n_kv_heads, page_size):
                    raise ValueError("scales must be uint8 [n_pages, n_kv_heads, page_size]")

        def page_stride(a, b):
            if n_pages == 1:
                return a[0].numel()
            if a.stride(0) != b.stride(0):
                raise ValueError("K and V must have the same page stride")
            return a.stride(0)

        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = n_pages, n_kv_heads, page_size, head_dim
        self.device = k.device
        self.struct = KVCacheStruct(k.data_ptr(), v.data_ptr(), _b._p(k_scale), _b._p(v_scale), page_stride(k, v),
                                    page_stride(k_scale, v_scale) if scaled else 0, n_pages, page_size, n_kv_heads,
                                    head_dim, CACHE_DTYPES[k.dtype])
        self.ref = ctypes.byref(self.struct)

    @classmethod
    def empty(cls, n_pages: int, n_kv_heads: int, page_size: int, head_dim: int, dtype=torch.bfloat16,
              device="cuda") -> "KVCache":
        """A cache on new, uninitialised tensors."""
        k, v = (torch.empty((n_pages, n_kv_heads, page_size, head_dim), dtype=dtype, device=device) for _ in "kv")
        if dtype == torch.bfloat16:
            return cls(k, v)
        return cls(k, v, *(torch.empty((n_pages, n_kv_heads, page_size), dtype=torch.uint8, device=device) for _ in "kv"))


def _i32(t: torch.Tensor, name: str, dim: int, device) -> None:
    if t.dtype != torch.int32 or t.dim() != dim or t.device != device or (t.numel() and t.stride(-1) != 1):
        raise ValueError(f"{name} must be int32 with {dim} dimension(s), rows contiguous, on the cache's GPU")


def _batch(cache: KVCache, page_table, start, offsets, n_rows: int) -> KVBatchStruct:
    _i32(page_table, "page_table", 2, cache.device)
    _i32(start, "start", 1, cache.device)
    n_req, width = _int32(page_table.shape[0], "page_table's rows"), _int32(page_table.shape[1], "page_table's width")
    if start.shape[0] != n_req:
        raise ValueError("page_table and start must have one row per request")
    if offsets is not None:
        _i32(offsets, "offsets", 1, cache.device)
        if offsets.shape[0] != n_req + 1:
            raise ValueError("offsets must have n_req + 1 entries")
    stride = page_table.stride(0) if n_req > 1 else width
    return KVBatchStruct(page_table.data_ptr(), stride, width, n_req, start.data_ptr(), _b._p(offsets), n_rows)


def _rows(t: torch.Tensor, name: str, cache: KVCache, heads: Optional[int]) -> None:
    if t.dim() != 3 or t.shape[2] != cache.head_dim or (heads is not None and t.shape[1] != heads) or t.stride(2) != 1:
        raise ValueError(f"{name} must be [n_rows, heads, head_dim] with contiguous head_dim, heads and head_dim the cache's")
    if t.device != cache.device:
        raise ValueError(f"{name} must be on the cache's GPU")


def _strides(t: torch.Tensor):
    """Row and head strides of [n_rows, heads, head_dim] in elements (those of
    an axis of one entry are never used and may be anything)."""
    n_rows, heads, dim = t.shape
    return (t.stride(0) if n_rows > 1 else heads * dim, t.stride(1) if heads > 1 else dim)


def _call(fn, cache: KVCache, stream, *args) -> None:
    """fn(*args, stream handle) with the cache's GPU current."""
    index = cache.device.index
    if stream is None:
        # the handle alone: 0.1 us, torch.cuda.current_stream() takes 2.6, a whole call 7
        handle = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device != cache.device:
        raise ValueError("stream belongs to another GPU than the cache")
    else:
        handle = stream.cuda_stream
    if index == torch.cuda.current_device():
        status = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            status = fn(*args, handle)
    if status:
        _b._check(status)


def _on(stream):
    """New tensors belong to the stream that uses them: the allocator then
    gives their memory to no other stream's work while it is in use."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def dflash_kv_write(cache: KVCache, k: torch.Tensor, v: torch.Tensor, *, page_table: torch.Tensor,
                    start: torch.Tensor, offsets: torch.Tensor, stream=None) -> None:
    """Stores k, v [n_rows, n_kv_heads, head_dim] (bf16 or fp32, strided views
    allowed) at their positions: row offsets[r] + i of request r goes to
    position start[r] + i.  page_table int32 [n_req, width]; start int32
    [n_req]; offsets int32 [n_req + 1]."""
    _rows(k, "k", cache, cache.n_kv_heads)
    _rows(v, "v", cache, cache.n_kv_heads)
    if k.dtype != v.dtype or k.shape[0] != v.shape[0]:
        raise ValueError("k and v must have one dtype and as many rows")
    batch = _batch(cache, page_table, start, offsets, k.shape[0])
    _call(_fns().dflash_kv_write, cache, stream, cache.ref, ctypes.byref(batch), k.data_ptr(), *_strides(k),
          v.data_ptr(), *_strides(v), _b._dtype_code(k))


def dflash_kv_read(cache: KVCache, *, page_table: torch.Tensor, start: torch.Tensor, offsets: torch.Tensor,
                   n_rows: Optional[int] = None, dtype: torch.dtype = torch.bfloat16, k_out=None, v_out=None,
                   stream=None):
    """Returns (k, v) [n_rows, n_kv_heads, head_dim]: row offsets[r] + i holds
    position start[r] + i of request r.  Give k_out and v_out, or n_rows (and
    dtype) for new tensors, whose rows behind offsets[-1] stay unset."""
    if k_out is None or v_out is None:
        if n_rows is None:
            raise ValueError("n_rows is needed without k_out and v_out")
        shape = (n_rows, cache.n_kv_heads, cache.head_dim)
        with _on(stream):
            k_out = torch.empty(shape, dtype=dtype, device=cache.device) if k_out is None else k_out
            v_out = torch.empty(shape, dtype=k_out.dtype, device=cache.device) if v_out is None else v_out
    for t, name in ((k_out, "k_out"), (v_out, "v_out")):
        _rows(t, name, cache, cache.n_kv_heads)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if k_out.dtype != v_out.dtype or k_out.shape != v_out.shape or n_rows not in (None, k_out.shape[0]):
        raise ValueError("k_out and v_out must have one dtype and n_rows rows")
    batch = _batch(cache, page_table, start, offsets, k_out.shape[0])
    _call(_fns().dflash_kv_read, cache, stream, cache.ref, ctypes.byref(batch), k_out.data_ptr(), v_out.data_ptr(),
          _b._dtype_code(k_out))
    return k_out, v_out


def dflash_kv_commit(cache: KVCache, *, page_table: torch.Tensor, start: torch.Tensor, paths: torch.Tensor,
                     path_lens: torch.Tensor, stream=None) -> None:
    """Moves the accepted nodes behind the prefix: position start[r] +
    paths[r, i] -> start[r] + i for i < path_lens[r].  paths int32 [n_req,
    width], ascending along a row; path_lens int32 [n_req]."""
    batch = _batch(cache, page_table, start, None, 0)
    _i32(paths, "paths", 2, cache.device)
    _i32(path_lens, "path_lens", 1, cache.device)
    if paths.shape[0] != batch.n_req or path_lens.shape[0] != batch.n_req:
        raise ValueError("paths and path_lens must have one row per request")
    stride = paths.stride(0) if paths.shape[0] > 1 else paths.shape[1]
    _call(_fns().dflash_kv_commit, cache, stream, cache.ref, ctypes.byref(batch), paths.data_ptr(), stride,
          _int32(paths.shape[1], "paths' width"), path_lens.data_ptr())


def tree_attention_workspace_size(cache: KVCache, *, n_req: int, max_nodes: int, n_q_heads: int) -> int:
    return _fns().dflash_tree_attention_workspace_size(cache.ref, _int32(n_req, "n_req"), _int32(max_nodes, "max_nodes"),
                                                       _int32(n_q_heads, "n_q_heads"))


def dflash_tree_attention(q: torch.Tensor, cache: KVCache, *, page_table: torch.Tensor, start: torch.Tensor,
                          offsets: torch.Tensor, max_nodes: int, mask: Optional[torch.Tensor] = None,
                          scale: Optional[float] = None, out: Optional[torch.Tensor] = None, workspace=None,
                          stream=None) -> torch.Tensor:
    """q [n_rows, n_q_heads, head_dim] bf16 (strided views allowed); the
    nodes' K and V are in the cache at positions start[r] + i.  mask int64
    [n_rows, words] (bits as unsigned: bit j % 64 of word j / 64 lets the row
    see node j) or None for a chain.  scale defaults to head_dim ** -0.5.
    Returns out bf16 [n_rows, n_q_heads, head_dim]; rows behind offsets[-1]
    are left as they were."""
    _rows(q, "q", cache, None)
    n_rows, n_q_heads, head_dim = q.shape
    _int32(max_nodes, "max_nodes")
    _int32(n_q_heads, "n_q_heads")
    batch = _batch(cache, page_table, start, offsets, n_rows)
    words = 0
    if mask is not None:
        if mask.dtype != torch.int64 or mask.dim() != 2 or mask.shape[0] != n_rows or mask.device != cache.device or \
                not mask.is_contiguous():
            raise ValueError("mask must be contiguous int64 [n_rows, words] on the cache's GPU")
        words = _int32(mask.shape[1], "mask's words")
        if words < (max_nodes + 63) // 64:              # a mask without elements has no address to tell it by
            raise ValueError("mask must have at least ceil(max_nodes / 64) words")
    if out is None:
        with _on(stream):
            out = torch.empty((n_rows, n_q_heads, head_dim), dtype=torch.bfloat16, device=cache.device)
    elif out.shape != q.shape or out.dtype != torch.bfloat16 or not out.is_contiguous() or out.device != cache.device:
        raise ValueError("out must be contiguous bf16 of q's shape on the cache's GPU")
    fns = _fns()
    if workspace is None:
        nbytes = fns.dflash_tree_attention_workspace_size(cache.ref, batch.n_req, max_nodes, n_q_heads)
        with _on(stream):
            workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=cache.device)
    elif workspace.device != cache.device or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous on the cache's GPU")
    _call(fns.dflash_tree_attention, cache, stream, cache.ref, ctypes.byref(batch), q.data_ptr(), *_strides(q),
          n_q_heads, _b._p(mask), words, max_nodes, head_dim ** -0.5 if scale is None else scale,
          _b._dtype_code(q), out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out
