"""Binding of the choice of pages and of the attention over them
(``include/dflash_kv_sparse.h``): argument marshalling only, as in ``kv``.

Functions have the names of the C entry points, take torch tensors on one GPU
and enqueue on the current stream of that GPU (or on ``stream``)."""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import binding as _b
from . import kv as _kv
from . import kv_pages as _pages
from .binding import _c_f32, _c_i32, _c_i64, _c_size, _c_vp

_C, _B, _P = _kv._P_CACHE, _kv._P_BATCH, _pages._P_BOUNDS
_SIGNATURES = {
    "dflash_kv_bounds": (_c_i32, [_C, _P, _B, _c_vp, _c_vp]),
    "dflash_kv_select_workspace_size": (_c_size, [_P, _c_i64, _c_i32]),
    "dflash_kv_select": (_c_i32, [_P, _B, _c_vp, _c_i64, _c_i64, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _c_i32, _c_vp, _c_vp,
                                  _c_size, _c_vp]),
    "dflash_sparse_attention_workspace_size": (_c_size, [_C, _c_i64, _c_i32, _c_i32, _c_i32]),
    "dflash_sparse_attention": (_c_i32, [_C, _B, _c_vp, _c_i64, _c_i64, _c_i32, _c_vp, _c_i32, _c_vp, _c_i32, _c_i32, _c_f32,
                                         _c_i32, _c_vp, _c_vp, _c_size, _c_vp]),
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


def dflash_kv_bounds(cache: "_kv.KVCache", bounds: "_pages.KVBounds", *, page_table: torch.Tensor, start: torch.Tensor,
                     end: torch.Tensor, stream=None) -> None:
    """Bounds of the pages that positions start[r] .. end[r] - 1 (int32
    [n_req], final by now) of request r have filled up."""
    if bounds.device != cache.device:
        raise ValueError("the bounds must be on the cache's GPU")
    batch = _kv._batch(cache, page_table, start, None, 0)
    _kv._i32(end, "end", 1, cache.device)
    if end.shape[0] != batch.n_req:
        raise ValueError("start and end must have one entry per request")
    _kv._call(_fns().dflash_kv_bounds, cache, stream, cache.ref, bounds.ref, ctypes.byref(batch), end.data_ptr())


def kv_select_workspace_size(bounds: "_pages.KVBounds", *, n_rows: int, table_width: int) -> int:
    return _fns().dflash_kv_select_workspace_size(bounds.ref, n_rows, _kv._int32(table_width, "table_width"))


def _space(nbytes: int, workspace, device, stream):
    if workspace is None:
        with _kv._on(stream):
            workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous on the cache's GPU")
    return workspace


def dflash_kv_select(q: torch.Tensor, bounds: "_pages.KVBounds", *, page_table: torch.Tensor, start: torch.Tensor,
                     offsets: torch.Tensor, max_nodes: int, n_take: Optional[int] = None, n_first: int = 1, n_last: int = 1,
                     out: Optional[torch.Tensor] = None, workspace=None, stream=None) -> torch.Tensor:
    """The blocks (full pages of its request's prefix) that each row of q
    [n_rows, n_q_heads, head_dim] bf16 (strided views allowed) and kv head needs
    most: int32 [n_rows, n_kv_heads, n_take], ascending, -1 behind the last; the
    first n_first and the last n_last are always among them.  Give n_take, or
    out, whose rows behind offsets[-1] are left as they were."""
    _kv._rows(q, "q", bounds, None)
    n_rows, n_q_heads, _ = q.shape
    batch = _kv._batch(bounds, page_table, start, offsets, n_rows)
    if out is None:
        if n_take is None:
            raise ValueError("n_take is needed without out")
        if n_take < 0:
            raise ValueError("n_take must be at least 1")
        with _kv._on(stream):
            out = torch.empty((n_rows, bounds.n_kv_heads, n_take), dtype=torch.int32, device=bounds.device)
    if out.dtype != torch.int32 or out.dim() != 3 or out.shape[:2] != (n_rows, bounds.n_kv_heads) or not out.is_contiguous() or \
            out.device != bounds.device or n_take not in (None, out.shape[2]):
        raise ValueError("out must be contiguous int32 [n_rows, n_kv_heads, n_take] on the bounds' GPU")
    workspace = _space(0 if workspace is not None else
                       _fns().dflash_kv_select_workspace_size(bounds.ref, n_rows, batch.table_width), workspace, bounds.device, stream)
    _kv._call(_fns().dflash_kv_select, bounds, stream, bounds.ref, ctypes.byref(batch), q.data_ptr(), *_kv._strides(q),
              _kv._int32(n_q_heads, "n_q_heads"), _kv._int32(max_nodes, "max_nodes"), _kv._int32(out.shape[2], "n_take"),
              _kv._int32(n_first, "n_first"), _kv._int32(n_last, "n_last"), _b._dtype_code(q), out.data_ptr(),
              workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out


def sparse_attention_workspace_size(cache: "_kv.KVCache", *, n_rows: int, n_take: int, max_nodes: int, n_q_heads: int) -> int:
    return _fns().dflash_sparse_attention_workspace_size(cache.ref, n_rows, _kv._int32(n_take, "n_take"),
                                                         _kv._int32(max_nodes, "max_nodes"), _kv._int32(n_q_heads, "n_q_heads"))


def dflash_sparse_attention(q: torch.Tensor, cache: "_kv.KVCache", blocks: torch.Tensor, *, page_table: torch.Tensor,
                            start: torch.Tensor, offsets: torch.Tensor, max_nodes: int, mask: Optional[torch.Tensor] = None,
                            scale: Optional[float] = None, out: Optional[torch.Tensor] = None, workspace=None,
                            stream=None) -> torch.Tensor:
    """dflash_tree_attention over the positions of blocks int32 [n_rows,
    n_kv_heads, n_take] (as dflash_kv_select gives them), the prefix behind its
    last full page, and the nodes; the other arguments are those of
    dflash_tree_attention."""
    _kv._rows(q, "q", cache, None)
    n_rows, n_q_heads, head_dim = q.shape
    _kv._int32(max_nodes, "max_nodes")
    _kv._int32(n_q_heads, "n_q_heads")
    batch = _kv._batch(cache, page_table, start, offsets, n_rows)
    if blocks.dtype != torch.int32 or blocks.dim() != 3 or blocks.shape[:2] != (n_rows, cache.n_kv_heads) or \
            not blocks.is_contiguous() or blocks.device != cache.device:
        raise ValueError("blocks must be contiguous int32 [n_rows, n_kv_heads, n_take] on the cache's GPU")
    words = 0
    if mask is not None:
        if mask.dtype != torch.int64 or mask.dim() != 2 or mask.shape[0] != n_rows or mask.device != cache.device or \
                not mask.is_contiguous():
            raise ValueError("mask must be contiguous int64 [n_rows, words] on the cache's GPU")
        words = _kv._int32(mask.shape[1], "mask's words")
        if words < (max_nodes + 63) // 64:              # a mask without elements has no address to tell it by
            raise ValueError("mask must have at least ceil(max_nodes / 64) words")
    if out is None:
        with _kv._on(stream):
            out = torch.empty((n_rows, n_q_heads, head_dim), dtype=torch.bfloat16, device=cache.device)
    elif out.shape != q.shape or out.dtype != torch.bfloat16 or not out.is_contiguous() or out.device != cache.device:
        raise ValueError("out must be contiguous bf16 of q's shape on the cache's GPU")
    n_take = _kv._int32(blocks.shape[2], "n_take")
    fns = _fns()
    workspace = _space(0 if workspace is not None else
                       fns.dflash_sparse_attention_workspace_size(cache.ref, n_rows, n_take, max_nodes, n_q_heads), workspace,
                       cache.device, stream)
    _kv._call(fns.dflash_sparse_attention, cache, stream, cache.ref, ctypes.byref(batch), q.data_ptr(), *_kv._strides(q),
              n_q_heads, blocks.data_ptr(), n_take, _b._p(mask), words, max_nodes, head_dim ** -0.5 if scale is None else scale,
              _b._dtype_code(q), out.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return out
