"""CPU checks of the page tables' C ABI: exports, struct layout, and the
refusals that happen on the host.  No call here reaches a kernel launch."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import block_draft_proposal_amd as D
from block_draft_proposal_amd import binding as B
from block_draft_proposal_amd import kv as K
from block_draft_proposal_amd import kv_pages as G

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dflash_kv_pages.h")


def test_library_exports_every_declared_entry_point():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(dflash_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(G.EXPORTED)
    for n in names:
        assert hasattr(D.lib(), n), n


def test_struct_layout_matches_c(tmp_path):
    structs = {"dflash_kv_pool": G.PoolStruct, "dflash_kv_rows": G.RowsStruct, "dflash_page_bounds": G.BoundsStruct}
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "dflash_kv_pages.h"', "int main(void){"]
    for name, cls in structs.items():
        src.append(f'printf("{name} %zu\\n", sizeof({name}));')
        src += [f'printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    (tmp_path / "layout.c").write_text("\n".join(src + ["return 0;}"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(tmp_path / "layout.c"), "-o", str(exe)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True).stdout.splitlines())
    for name, cls in structs.items():
        assert int(got[name]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, f


# addresses that are never dereferenced: every call below is refused before a launch
POOL = dict(refs=1 << 40, n_pages=1000, page_size=16)
ROWS = dict(page_table=2 << 40, table_stride=40, table_width=40, n_req=8, lens=3 << 40)
CACHE = dict(k=8 << 40, v=9 << 40, k_scale=None, v_scale=None, page_stride=2 * 16 * 64, scale_page_stride=0, n_pages=10,
             page_size=16, n_kv_heads=2, head_dim=64, dtype=B.DFLASH_BF16)
BOUNDS = dict(codes=10 << 40, scale=11 << 40, n_pages=10, page_size=16, n_kv_heads=2, head_dim=64)


def _pool(p, r):
    return ctypes.byref(G.PoolStruct(**{**POOL, **(p or {})})), ctypes.byref(G.RowsStruct(**{**ROWS, **(r or {})}))


def _resize(pool=None, rows=None, want=4 << 40, copies=5 << 40, counts=6 << 40, ws=7 << 40, n=1 << 50):
    return G._fns().dflash_kv_resize(*_pool(pool, rows), want, copies, counts, ws, n, None)


def _fork(pool=None, rows=None, parents=4 << 40, ws=7 << 40, n=1 << 50):
    return G._fns().dflash_kv_fork(*_pool(pool, rows), parents, ws, n, None)


def _compact(pool=None, rows=None, page_map=4 << 40, copies=5 << 40, most=500, counts=6 << 40, ws=7 << 40, n=1 << 50):
    return G._fns().dflash_kv_compact(*_pool(pool, rows), page_map, copies, most, counts, ws, n, None)


def _copy(cache=None, bounds=None, copies=5 << 40, most=3, counts=6 << 40):
    at = None if bounds is None else ctypes.byref(G.BoundsStruct(**{**BOUNDS, **bounds}))
    return G._fns().dflash_kv_copy_pages(ctypes.byref(K.KVCacheStruct(**{**CACHE, **(cache or {})})), at, copies, most, counts, None)


@pytest.mark.parametrize("call", [_resize, _fork, _compact], ids=["resize", "fork", "compact"])
def test_bad_pools_and_tables(call):
    for kw in (dict(refs=None), dict(refs=(1 << 40) + 2), dict(n_pages=0), dict(n_pages=(1 << 30) + 1), dict(page_size=0), dict(page_size=65537)):
        assert call(pool=kw) == -1, kw
        assert B.last_error().startswith("dflash_kv_"), kw
    for kw, code in ((dict(n_req=-1), -1), (dict(n_req=(1 << 20) + 1), -1), (dict(table_width=0), -1), (dict(table_stride=39), -1),
                     (dict(page_table=None), -1), (dict(lens=None), -1), (dict(table_stride=1 << 60), -1),
                     (dict(n_req=1 << 20, table_width=1 << 21, table_stride=1 << 21), -2), (dict(page_table=(2 << 40) + 1), -1)):
        assert call(rows=kw) == code, kw
    assert call(ws=None) == -3 and call(n=100) == -3 and call(ws=(7 << 40) + 16) == -1


@pytest.mark.parametrize("call,names", [(_resize, ("want", "copies", "counts", "ws")), (_fork, ("parents", "ws")),
                                        (_compact, ("page_map", "copies", "counts", "ws"))], ids=["resize", "fork", "compact"])
def test_arrays_that_overlap_or_are_missing(call, names):
    for name in names:
        if name != "ws":
            assert call(**{name: None}) == -1, name
            assert call(**{name: (20 << 40) + 2}) == -1, name
        for over in (POOL["refs"], ROWS["page_table"]):
            assert call(**{name: over}) == -1, (name, over)
            assert "overlaps" in B.last_error()
    assert call(rows=dict(lens=POOL["refs"] + 256)) == -1
    assert call(rows=dict(page_table=POOL["refs"] - 256)) == -1
    need = G._fns().dflash_kv_pages_workspace_size(_pool(None, None)[0], 8, 40)
    assert need % 256 == 0 and call(ws=ROWS["lens"] - need + 256) == -1    # its last bytes reach into lens


def test_workspace_size():
    size = lambda n, w, p=None: G._fns().dflash_kv_pages_workspace_size(_pool(p, None)[0], n, w)  # noqa: E731
    last = 0
    for n in (0, 1, 2, 3, 17, 300, 5000, 1 << 20):
        assert size(n, 40) >= last
        last = size(n, 40)
        assert size(n, 40) >= size(n, 39) >= size(n, 1) > 0
    assert size(-1, 4) == 0 and size(4, 0) == 0 and size((1 << 20) + 1, 4) == 0 and size(1 << 20, 1 << 21) == 0
    assert size(4, 4, dict(n_pages=0)) == 0 and size(4, 4, dict(page_size=0)) == 0
    assert _resize(n=size(8, 40) - 1) == -3


def test_compact_and_copy_refusals():
    assert _compact(most=-1) == -1 and _compact(most=(1 << 30) + 1) == -1
    assert _copy(most=-1) == -1 and _copy(most=(1 << 30) + 1) == -1
    assert _copy(copies=None) == -1 and _copy(copies=(5 << 40) + 2) == -1 and _copy(counts=(6 << 40) + 1) == -1
    assert _copy(most=0, copies=None) == 0
    for over in (8 << 40, 9 << 40):
        assert _copy(copies=over) == -1 and _copy(counts=over) == -1
    assert _copy(cache=dict(v=CACHE["k"])) == -1 and _copy(cache=dict(head_dim=96)) == -2
    for kw, code in ((dict(codes=None), -1), (dict(scale=None), -1), (dict(codes=(10 << 40) + 8), -1), (dict(n_pages=11), -1),
                     (dict(page_size=8), -1), (dict(n_kv_heads=1), -1), (dict(head_dim=128), -1), (dict(head_dim=32), -2),
                     (dict(codes=8 << 40), -1), (dict(scale=9 << 40), -1), (dict(scale=(10 << 40) + 64), -1),
                     (dict(codes=5 << 40), -1), (dict(scale=6 << 40), -1), (dict(n_pages=0), -1), (dict(n_kv_heads=0), -1)):
        assert _copy(bounds=kw) == code, kw


def test_nothing_to_do_is_no_error():
    assert _fork(rows=dict(n_req=0, page_table=None, lens=None)) == 0
    assert B.last_error() == ""


def test_objects_refuse_what_they_do_not_describe():
    with pytest.raises(ValueError, match="refs"):
        D.KVPool(torch.zeros(4, dtype=torch.int32), 16)
    codes, scale = torch.zeros((4, 2, 2, 64), dtype=torch.int8), torch.zeros((4, 2), dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        D.KVBounds(codes, scale, page_size=16)
    with pytest.raises(ValueError, match="codes"):
        D.KVBounds(codes[:, :, :1], scale, page_size=16)
    with pytest.raises(ValueError, match="scale"):
        D.KVBounds(codes, scale[:3], page_size=16)
