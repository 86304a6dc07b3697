"""Binding of the page tables and the counts of a pool's pages
(``include/dflash_kv_pages.h``): argument marshalling only, as in ``kv``.

Functions have the names of the C entry points, take torch tensors on one GPU
and enqueue on the current stream of that GPU (or on ``stream``)."""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import binding as _b
from . import kv as _kv
from .binding import _c_i32, _c_i64, _c_size, _c_vp


class PoolStruct(ctypes.Structure):
    """Mirror of dflash_kv_pool."""
    _fields_ = [("refs", _c_vp), ("n_pages", _c_i64), ("page_size", _c_i32)]


class RowsStruct(ctypes.Structure):
    """Mirror of dflash_kv_rows."""
    _fields_ = [("page_table", _c_vp), ("table_stride", _c_i64), ("table_width", _c_i32), ("n_req", _c_i32), ("lens", _c_vp)]


class BoundsStruct(ctypes.Structure):
    """Mirror of dflash_page_bounds."""
    _fields_ = [("codes", _c_vp), ("scale", _c_vp), ("n_pages", _c_i64), ("page_size", _c_i32), ("n_kv_heads", _c_i32),
                ("head_dim", _c_i32)]


_P_POOL, _P_ROWS, _P_BOUNDS = (ctypes.POINTER(s) for s in (PoolStruct, RowsStruct, BoundsStruct))
_SIGNATURES = {
    "dflash_kv_pages_workspace_size": (_c_size, [_P_POOL, _c_i32, _c_i32]),
    "dflash_kv_resize": (_c_i32, [_P_POOL, _P_ROWS, _c_vp, _c_vp, _c_vp, _c_vp, _c_size, _c_vp]),
    "dflash_kv_fork": (_c_i32, [_P_POOL, _P_ROWS, _c_vp, _c_vp, _c_size, _c_vp]),
    "dflash_kv_compact": (_c_i32, [_P_POOL, _P_ROWS, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp, _c_size, _c_vp]),
    "dflash_kv_copy_pages": (_c_i32, [_kv._P_CACHE, _P_BOUNDS, _c_vp, _c_i64, _c_vp, _c_vp]),
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


class KVPool:
    """The counts of a pool's pages: refs int32 [n_pages], 0 for a free page.
    The object only describes the tensor; make it once and pass it to every
    call."""

    def __init__(self, refs: torch.Tensor, page_size: int):
        if refs.dtype != torch.int32 or refs.dim() != 1 or not refs.is_contiguous() or not refs.is_cuda:
            raise ValueError("refs must be contiguous int32 [n_pages] on a GPU")
        if refs.shape[0] < 1:
            raise ValueError("a pool has at least one page")
        self.refs, self.page_size, self.n_pages, self.device = refs, _kv._int32(page_size, "page_size"), refs.shape[0], refs.device
        self.struct = PoolStruct(refs.data_ptr(), refs.shape[0], page_size)
        self.ref = ctypes.byref(self.struct)


class KVBounds:
    """What is kept of each full page of a cache, to choose pages by: codes
    int8 [n_pages, n_kv_heads, 2, head_dim] (the least and the greatest key of
    each channel) and scale uint8 [n_pages, n_kv_heads].  The object only
    describes the tensors."""

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor, *, page_size: int):
        if codes.dtype != torch.int8 or codes.dim() != 4 or codes.shape[2] != 2 or not codes.is_contiguous():
            raise ValueError("codes must be contiguous int8 [n_pages, n_kv_heads, 2, head_dim]")
        if scale.dtype != torch.uint8 or scale.shape != codes.shape[:2] or not scale.is_contiguous():
            raise ValueError("scale must be contiguous uint8 [n_pages, n_kv_heads]")
        if not codes.is_cuda or scale.device != codes.device:
            raise ValueError("the bounds' tensors must be on one GPU")
        if codes.shape[0] < 1:
            raise ValueError("a pool has at least one page")
        self.codes, self.scale, self.page_size, self.device = codes, scale, _kv._int32(page_size, "page_size"), codes.device
        self.n_pages, self.n_kv_heads, self.head_dim = codes.shape[0], _kv._int32(codes.shape[1], "n_kv_heads"), codes.shape[3]
        self.struct = BoundsStruct(codes.data_ptr(), scale.data_ptr(), self.n_pages, page_size, self.n_kv_heads,
                                   _kv._int32(self.head_dim, "head_dim"))
        self.ref = ctypes.byref(self.struct)

    @classmethod
    def empty(cls, cache: "_kv.KVCache") -> "KVBounds":
        """Bounds for a cache on new, uninitialised tensors."""
        shape = (cache.n_pages, cache.n_kv_heads)
        return cls(torch.empty(shape + (2, cache.head_dim), dtype=torch.int8, device=cache.device),
                   torch.empty(shape, dtype=torch.uint8, device=cache.device), page_size=cache.page_size)


def _rows(pool: KVPool, page_table: torch.Tensor, lens: torch.Tensor) -> RowsStruct:
    device = pool.device
    _kv._i32(page_table, "page_table", 2, device)
    n_req, width = page_table.shape
    _vector(lens, "lens", n_req, device)
    if n_req > 0x7FFFFFFF or width > 0x7FFFFFFF:
        raise ValueError("page_table's shape does not fit 32 bits")
    return RowsStruct(page_table.data_ptr(), page_table.stride(0) if n_req > 1 else width, width, n_req, lens.data_ptr())


def _vector(t: torch.Tensor, name: str, n: int, device) -> None:
    if t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be contiguous int32 [{n}] on the pool's GPU")


def _pairs(t: torch.Tensor, device) -> None:
    if t.dtype != torch.int32 or t.dim() != 2 or t.shape[1] != 2 or not t.is_contiguous() or t.device != device:
        raise ValueError("copies must be contiguous int32 [n, 2] on the pool's GPU")


def _workspace(pool: KVPool, rows: RowsStruct, workspace, stream):
    if workspace is None:
        nbytes = _fns().dflash_kv_pages_workspace_size(pool.ref, rows.n_req, rows.table_width)
        with _kv._on(stream):
            workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=pool.device)
    elif workspace.device != pool.device or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous on the pool's GPU")
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _lists(pool: KVPool, copies, counts, n: int, stream):
    if copies is None or counts is None:
        with _kv._on(stream):
            copies = torch.empty((n, 2), dtype=torch.int32, device=pool.device) if copies is None else copies
            counts = torch.empty(2, dtype=torch.int32, device=pool.device) if counts is None else counts
    _pairs(copies, pool.device)
    _vector(counts, "counts", 2, pool.device)
    return copies, counts


def kv_pages_workspace_size(pool: KVPool, *, n_req: int, table_width: int) -> int:
    """Bytes that dflash_kv_resize, dflash_kv_fork and dflash_kv_compact need."""
    return _fns().dflash_kv_pages_workspace_size(pool.ref, _kv._int32(n_req, "n_req"), _kv._int32(table_width, "table_width"))


def dflash_kv_resize(pool: KVPool, *, page_table: torch.Tensor, lens: torch.Tensor, want: torch.Tensor,
                     copies: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None, workspace=None,
                     stream=None):
    """lens becomes want (int32 [n_req]); page_table int32 [n_req, width] and
    lens int32 [n_req] are updated in place.  Returns (copies, counts): the
    first counts[0] rows of copies int32 [n_req, 2] name the pages whose
    contents dflash_kv_copy_pages has to move; counts[1] is the number of free
    pages that were missing (then no request has grown)."""
    rows = _rows(pool, page_table, lens)
    _vector(want, "want", rows.n_req, pool.device)
    copies, counts = _lists(pool, copies, counts, rows.n_req, stream)
    if copies.shape[0] < rows.n_req:
        raise ValueError("copies must have a row for each request")
    keep, at, nbytes = _workspace(pool, rows, workspace, stream)
    _kv._call(_fns().dflash_kv_resize, pool, stream, pool.ref, ctypes.byref(rows), want.data_ptr(), copies.data_ptr(),
              counts.data_ptr(), at, nbytes)
    return copies, counts


def dflash_kv_fork(pool: KVPool, *, page_table: torch.Tensor, lens: torch.Tensor, parents: torch.Tensor, workspace=None,
                   stream=None) -> None:
    """Row r of page_table and lens becomes row parents[r] (int32 [n_req]; below
    0: empty), all at once; pages are shared, none is copied."""
    rows = _rows(pool, page_table, lens)
    _vector(parents, "parents", rows.n_req, pool.device)
    keep, at, nbytes = _workspace(pool, rows, workspace, stream)
    _kv._call(_fns().dflash_kv_fork, pool, stream, pool.ref, ctypes.byref(rows), parents.data_ptr(), at, nbytes)


def dflash_kv_compact(pool: KVPool, *, page_table: torch.Tensor, lens: torch.Tensor,
                      copies: Optional[torch.Tensor] = None, counts: Optional[torch.Tensor] = None,
                      page_map: Optional[torch.Tensor] = None, workspace=None, stream=None):
    """Moves the highest held pages to the lowest free ones, at most as many as
    copies int32 [max_copies, 2] has rows (n_pages // 2 without), and rewrites
    page_table.  Returns (copies, counts, page_map): counts[0] pairs whose
    contents dflash_kv_copy_pages has to move, counts[1] held pages; page_map
    int32 [n_pages] where each page is now, -1 where it was free."""
    rows = _rows(pool, page_table, lens)
    copies, counts = _lists(pool, copies, counts, pool.n_pages // 2, stream)
    if page_map is None:
        with _kv._on(stream):
            page_map = torch.empty(pool.n_pages, dtype=torch.int32, device=pool.device)
    _vector(page_map, "page_map", pool.n_pages, pool.device)
    keep, at, nbytes = _workspace(pool, rows, workspace, stream)
    _kv._call(_fns().dflash_kv_compact, pool, stream, pool.ref, ctypes.byref(rows), page_map.data_ptr(), copies.data_ptr(),
              copies.shape[0], counts.data_ptr(), at, nbytes)
    return copies, counts, page_map


def dflash_kv_copy_pages(cache: "_kv.KVCache", copies: torch.Tensor, counts: Optional[torch.Tensor] = None, *,
                         bounds: Optional[KVBounds] = None, stream=None) -> None:
    """Page copies[i, 1] of the cache (and of its bounds) becomes a copy of page
    copies[i, 0], for the first counts[0] rows, or all without counts."""
    _pairs(copies, cache.device)
    if counts is not None:
        _vector(counts, "counts", 2, cache.device)
    if bounds is not None and bounds.device != cache.device:
        raise ValueError("the bounds must be on the cache's GPU")
    _kv._call(_fns().dflash_kv_copy_pages, cache, stream, cache.ref, None if bounds is None else bounds.ref, copies.data_ptr(),
              copies.shape[0], _b._p(counts))
