"""CPU checks of the C ABI of the choice of pages and the attention over them:
exports and the refusals that happen on the host.  No call here reaches a kernel
launch."""
import ctypes
import os
import re

import pytest

import block_draft_proposal_amd as D
from block_draft_proposal_amd import binding as B
from block_draft_proposal_amd import kv as K
from block_draft_proposal_amd import kv_pages as G
from block_draft_proposal_amd import kv_sparse as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dflash_kv_sparse.h")

# addresses that are never dereferenced: every call below is refused before a launch
CACHE = dict(k=1 << 40, v=2 << 40, k_scale=None, v_scale=None, page_stride=8 * 16 * 128, scale_page_stride=0,
             n_pages=10, page_size=16, n_kv_heads=8, head_dim=128, dtype=B.DFLASH_BF16)
SCALED = dict(k_scale=6 << 40, v_scale=7 << 40, scale_page_stride=8 * 16, dtype=K.DFLASH_E4M3)
BATCH = dict(page_table=3 << 40, table_stride=4, table_width=4, n_req=2, start=4 << 40, offsets=5 << 40, n_rows=8)
BOUNDS = dict(codes=12 << 40, scale=13 << 40, n_pages=10, page_size=16, n_kv_heads=8, head_dim=128)


def _structs(cache=None, batch=None, bounds=None):
    return (ctypes.byref(K.KVCacheStruct(**{**CACHE, **(cache or {})})), ctypes.byref(K.KVBatchStruct(**{**BATCH, **(batch or {})})),
            ctypes.byref(G.BoundsStruct(**{**BOUNDS, **(bounds or {})})))


def _bounds(cache=None, batch=None, bounds=None, end=8 << 40):
    c, b, x = _structs(cache, batch, bounds)
    return S._fns().dflash_kv_bounds(c, x, b, end, None)


def _select(batch=None, bounds=None, q=8 << 40, qr=32 * 128, qh=128, hq=32, nodes=4, take=3, first=1, last=1, dtype=1, out=9 << 40,
            ws=10 << 40, n=1 << 50):
    _, b, x = _structs(None, batch, bounds)
    return S._fns().dflash_kv_select(x, b, q, qr, qh, hq, nodes, take, first, last, dtype, out, ws, n, None)


def _sparse(cache=None, batch=None, q=8 << 40, qr=32 * 128, qh=128, hq=32, blocks=14 << 40, take=3, mask=None, words=0, nodes=4,
            scale=0.1, dtype=1, out=9 << 40, ws=10 << 40, n=1 << 38):
    c, b, _ = _structs(cache, batch)
    return S._fns().dflash_sparse_attention(c, b, q, qr, qh, hq, blocks, take, mask, words, nodes, scale, dtype, out, ws, n, None)


def test_library_exports_every_declared_entry_point():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(dflash_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(S.EXPORTED)
    for n in names:
        assert hasattr(D.lib(), n), n


BAD_BATCH = [(dict(n_req=-1), -1), (dict(table_width=0), -1), (dict(table_stride=3), -1), (dict(page_table=None), -1), (dict(start=None), -1)]
BAD_ROWS = [(dict(n_rows=-1), -1), (dict(n_rows=1 << 31), -1), (dict(offsets=None), -1), (dict(n_rows=(1 << 18) + 1), -2)]
BAD_BOUNDS = [(dict(codes=None), -1), (dict(scale=None), -1), (dict(codes=(12 << 40) + 8), -1), (dict(n_pages=0), -1), (dict(n_pages=1 << 31), -1),
              (dict(page_size=0), -1), (dict(page_size=65537), -1), (dict(n_kv_heads=0), -1), (dict(head_dim=96), -2),
              (dict(scale=(12 << 40) + 100), -1)]


@pytest.mark.parametrize("call", [_bounds, _select, _sparse], ids=["bounds", "select", "sparse"])
def test_bad_batches_and_bounds(call):
    for kw, code in BAD_BATCH + ([] if call is _bounds else BAD_ROWS):
        assert call(batch=kw) == code, kw
        assert B.last_error().startswith("dflash_"), kw
    if call is not _sparse:
        for kw, code in BAD_BOUNDS:
            assert call(bounds=kw) == code, kw
    if call is not _select:
        for kw, code in ((dict(head_dim=96), -2), (dict(n_pages=0), -1), (dict(k=None), -1), (dict(dtype=0), -1)):
            assert call(cache=kw) == code, kw
    assert call(batch=dict(n_req=0, page_table=None, start=None, offsets=None)) == 0
    assert B.last_error() == ""


def test_bounds_refusals():
    for kw in (dict(n_pages=11), dict(page_size=8), dict(n_kv_heads=4), dict(head_dim=64), dict(codes=1 << 40), dict(codes=2 << 40),
               dict(codes=3 << 40), dict(scale=4 << 40), dict(scale=1 << 40), dict(scale=8 << 40)):
        assert _bounds(bounds=kw) == -1, kw
    assert _bounds(end=None) == -1
    assert _bounds(batch=dict(n_req=(1 << 20) + 1)) == -2
    assert _bounds(cache=SCALED, bounds=dict(codes=6 << 40)) == -1


def test_select_refusals():
    for kw, code in ((dict(hq=0), -1), (dict(hq=12), -1), (dict(hq=8 * 65), -2), (dict(nodes=0), -1), (dict(nodes=4097), -2), (dict(take=0), -1),
                     (dict(take=65537), -1), (dict(first=-1), -1), (dict(last=-1), -1), (dict(first=2, last=2), -1),
                     (dict(first=0x7fffffff, last=0x7fffffff), -1), (dict(dtype=0), -2), (dict(dtype=7), -1), (dict(q=None), -1),
                     (dict(q=(8 << 40) + 8), -1), (dict(qr=4100), -1), (dict(qr=-8), -1), (dict(out=None), -1), (dict(out=(9 << 40) + 2), -1),
                     (dict(out=8 << 40), -1), (dict(out=12 << 40), -1), (dict(out=13 << 40), -1), (dict(out=3 << 40), -1), (dict(out=4 << 40), -1),
                     (dict(out=5 << 40), -1), (dict(out=10 << 40), -1), (dict(ws=None), -3), (dict(ws=(10 << 40) + 64), -1), (dict(ws=8 << 40), -1),
                     (dict(ws=12 << 40), -1), (dict(ws=3 << 40), -1)):
        assert _select(**kw) == code, kw
    assert _select(batch=dict(table_width=(1 << 24) + 1, table_stride=1 << 25)) == -2
    size = lambda rows, width: S._fns().dflash_kv_select_workspace_size(_structs()[2], rows, width)  # noqa: E731
    assert size(8, 4) > 0 and _select(n=size(8, 4) - 1) == -3
    assert size(8, 5) >= size(8, 4) and size(9, 4) >= size(8, 4)
    assert size(0, 4) == 0 and size(8, 0) == 0 and size((1 << 18) + 1, 4) == 0 and size(8, (1 << 24) + 1) == 0


def test_sparse_refusals():
    for kw, code in ((dict(hq=0), -1), (dict(hq=12), -1), (dict(hq=8 * 65), -2), (dict(nodes=0), -1), (dict(nodes=4097), -2), (dict(take=-1), -1),
                     (dict(take=65537), -1), (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(scale=2.0 ** 101), -1),
                     (dict(mask=11 << 40, words=0), -1), (dict(mask=11 << 40, words=1, nodes=65), -1), (dict(words=1), -1),
                     (dict(mask=(11 << 40) + 4, words=1), -1), (dict(dtype=0), -2), (dict(dtype=5), -1), (dict(q=None), -1), (dict(q=(8 << 40) + 8), -1),
                     (dict(qr=4100), -1), (dict(blocks=None), -1), (dict(blocks=(14 << 40) + 1), -1), (dict(out=None), -1), (dict(out=(9 << 40) + 2), -1),
                     (dict(out=8 << 40), -1), (dict(out=1 << 40), -1), (dict(out=2 << 40), -1), (dict(out=3 << 40), -1), (dict(out=14 << 40), -1),
                     (dict(out=11 << 40, mask=11 << 40, words=1), -1), (dict(out=10 << 40), -1), (dict(ws=None), -3), (dict(ws=(10 << 40) + 64), -1),
                     (dict(n=100), -3), (dict(ws=8 << 40), -1), (dict(ws=1 << 40), -1), (dict(ws=5 << 40), -1), (dict(ws=14 << 40), -1)):
        assert _sparse(**kw) == code, kw
    assert _sparse(cache=dict(page_size=65536, page_stride=8 * 65536 * 128), take=20000) == -2
    assert _sparse(cache=SCALED, out=6 << 40) == -1
    size = lambda **kw: S._fns().dflash_sparse_attention_workspace_size(  # noqa: E731
        _structs()[0], *({**dict(rows=8, take=3, nodes=4, hq=32), **kw}).values())
    assert size() > 0 and _sparse(n=size() - 1) == -3
    last = 0
    for kw in (dict(nodes=1), dict(), dict(nodes=4096), dict(rows=9, nodes=4096), dict(rows=9, take=4), dict(rows=1000, take=4),
               dict(rows=1 << 18, take=4), dict(rows=1 << 18, take=65536), dict(rows=1 << 18, take=65536, hq=512)):
        assert size(**kw) >= last, kw
        last = size(**kw)
    assert size(take=0) > 0
    assert size(rows=0) == size(hq=12) == size(hq=8 * 65) == size(take=-1) == size(nodes=0) == size(nodes=4097) == size(rows=(1 << 18) + 1) == 0
