"""CPU checks of the KV cache's C ABI: exports, struct layout, and the refusals
that happen on the host.  No call here reaches a kernel launch."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import block_draft_proposal_amd as D
from block_draft_proposal_amd import binding as B
from block_draft_proposal_amd import kv as K

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "dflash_kv.h")


def test_library_exports_every_declared_entry_point():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(dflash_[a-z0-9_]+)\s*\(", text)))
    assert names == sorted(K.EXPORTED) and len(names) == 5
    for n in names:
        assert hasattr(D.lib(), n), n


def test_struct_layout_matches_c(tmp_path):
    structs = {"dflash_kv_cache": K.KVCacheStruct, "dflash_kv_batch": K.KVBatchStruct}
    src = ["#include <stdio.h>", "#include <stddef.h>", '#include "dflash_kv.h"', "int main(void){"]
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
CACHE = dict(k=1 << 40, v=2 << 40, k_scale=None, v_scale=None, page_stride=8 * 16 * 128, scale_page_stride=0,
             n_pages=10, page_size=16, n_kv_heads=8, head_dim=128, dtype=B.DFLASH_BF16)
BATCH = dict(page_table=3 << 40, table_stride=4, table_width=4, n_req=2, start=4 << 40, offsets=5 << 40, n_rows=8)
SCALED = dict(k_scale=6 << 40, v_scale=7 << 40, scale_page_stride=8 * 16, dtype=K.DFLASH_E4M3)


def _structs(cache=None, batch=None):
    return (ctypes.byref(K.KVCacheStruct(**{**CACHE, **(cache or {})})), ctypes.byref(K.KVBatchStruct(**{**BATCH, **(batch or {})})))


def _write(cache=None, batch=None, k=8 << 40, v=9 << 40, kr=1024, kh=128, vr=1024, vh=128, dtype=1):
    return K._fns().dflash_kv_write(*_structs(cache, batch), k, kr, kh, v, vr, vh, dtype, None)


def _read(cache=None, batch=None, k=8 << 40, v=9 << 40, dtype=1):
    return K._fns().dflash_kv_read(*_structs(cache, batch), k, v, dtype, None)


def _commit(cache=None, batch=None, paths=8 << 40, stride=4, width=4, lens=9 << 40):
    return K._fns().dflash_kv_commit(*_structs(cache, batch), paths, stride, width, lens, None)


def _tree(cache=None, batch=None, q=8 << 40, qr=32 * 128, qh=128, hq=32, mask=None, words=0, nodes=4, scale=0.1, dtype=1,
          out=9 << 40, ws=10 << 40, ws_bytes=1 << 60):
    return K._fns().dflash_tree_attention(*_structs(cache, batch), q, qr, qh, hq, mask, words, nodes, scale, dtype, out, ws,
                                          ws_bytes, None)


BAD_CACHE = [
    (dict(dtype=0), -1), (dict(dtype=9), -1), (dict(head_dim=96), -2), (dict(head_dim=0), -2), (dict(page_size=0), -1),
    (dict(page_size=65537), -1), (dict(n_kv_heads=0), -1), (dict(n_pages=0), -1), (dict(n_pages=1 << 31), -1),
    (dict(page_stride=8 * 16 * 128 - 8), -1), (dict(page_stride=8 * 16 * 128 + 4), -1), (dict(page_stride=1 << 62), -1),
    (dict(k=None), -1), (dict(v=None), -1), (dict(k=(1 << 40) + 8), -1), (dict(k_scale=1 << 41), -1),
    (dict(dtype=K.DFLASH_I8), -1), ({**SCALED, "v_scale": None}, -1), ({**SCALED, "scale_page_stride": 100}, -1),
]
BAD_BATCH = [
    (dict(n_req=-1), -1), (dict(table_width=0), -1), (dict(table_stride=3), -1), (dict(page_table=None), -1), (dict(start=None), -1),
]
BAD_ROWS = [(dict(n_rows=-1), -1), (dict(n_rows=1 << 31), -1), (dict(offsets=None), -1)]


@pytest.mark.parametrize("call", [_write, _read, _commit, _tree], ids=["write", "read", "commit", "tree"])
def test_bad_caches_and_batches(call):
    for kw, code in BAD_CACHE:
        assert call(cache=kw) == code, kw
        assert B.last_error().startswith("dflash_"), kw
    for kw, code in BAD_BATCH + ([] if call is _commit else BAD_ROWS):
        assert call(batch=kw) == code, kw
    assert call(batch=dict(n_req=0)) == 0
    assert B.last_error() == ""
    assert K._fns().dflash_kv_read(None, None, None, None, 1, None) == -1


def test_nothing_to_do_is_no_error():
    for call in (_write, _read, _tree):
        assert call(batch=dict(n_rows=0)) == 0
        assert call(batch=dict(n_req=0, page_table=None, start=None, offsets=None)) == 0
    assert _commit(width=0, paths=None) == 0


def test_write_refusals():
    for kw in (dict(k=None), dict(v=None), dict(k=(8 << 40) + 2), dict(kr=1020), dict(vh=4), dict(kr=-8), dict(dtype=2),
               dict(dtype=0, kr=1022), dict(k=(1 << 40) + 256), dict(v=(2 << 40) + 256), dict(kr=1 << 50)):
        assert _write(**kw) == -1, kw
    assert _write(cache=SCALED, k=(6 << 40)) == -1      # over the scales
    assert _write(cache=dict(v=CACHE["k"])) == -1
    assert _write(cache={**SCALED, "v_scale": SCALED["k_scale"]}) == -1


def test_read_refusals():
    for kw in (dict(k=None), dict(v=None), dict(k=(8 << 40) + 8), dict(dtype=3), dict(v=(8 << 40) + 64), dict(k=(1 << 40) + 64),
               dict(v=2 << 40)):
        assert _read(**kw) == -1, kw


def test_commit_refusals():
    for kw in (dict(width=-1), dict(stride=3), dict(paths=None), dict(lens=None)):
        assert _commit(**kw) == -1, kw
    assert _commit(cache=dict(v=CACHE["k"])) == -1
    assert _commit(cache={**SCALED, "v_scale": SCALED["k_scale"]}) == -1


def test_tree_refusals():
    for kw, code in ((dict(hq=0), -1), (dict(hq=12), -1), (dict(hq=8 * 65), -2), (dict(nodes=0), -1), (dict(nodes=4097), -2),
                     (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
                     (dict(mask=11 << 40, words=0), -1), (dict(mask=11 << 40, words=1, nodes=65), -1), (dict(words=1), -1),
                     (dict(mask=(11 << 40) + 4, words=1), -1), (dict(dtype=0), -2), (dict(dtype=5), -1), (dict(q=None), -1),
                     (dict(q=(8 << 40) + 8), -1), (dict(qr=4100), -1), (dict(out=None), -1), (dict(out=(9 << 40) + 2), -1),
                     (dict(out=8 << 40), -1), (dict(out=(1 << 40) + 4096), -1), (dict(out=2 << 40), -1)):
        assert _tree(**kw) == code, kw
    need = K._fns().dflash_tree_attention_workspace_size(_structs()[0], 2, 4, 32)
    if need:
        assert _tree(ws_bytes=need - 1) == -3 and _tree(ws=None) == -3 and _tree(ws=(10 << 40) + 16) == -1
    assert K._fns().dflash_tree_attention_workspace_size(_structs(dict(head_dim=1))[0], 2, 4, 32) == 0
    assert K._fns().dflash_tree_attention_workspace_size(_structs()[0], 0, 4, 32) == 0
    assert K._fns().dflash_tree_attention_workspace_size(_structs()[0], 2, 4, 33) == 0


def test_extents_beyond_what_offsets_hold():
    for call in (_write, _read, _commit, _tree):
        assert call(cache=dict(page_stride=1 << 40, n_pages=1 << 30)) == -1
        assert call(cache={**SCALED, "scale_page_stride": 1 << 40, "n_pages": (1 << 31) - 1}) == -1
    assert _write(batch=dict(n_rows=(1 << 31) - 1), kr=1 << 30) == -2
    assert _write(batch=dict(n_rows=1 << 27), kr=1 << 40) == -1
    assert _tree(batch=dict(n_rows=(1 << 31) - 1), qr=1 << 40) == -1
    # grids past 2^32 threads
    assert _write(batch=dict(n_rows=1 << 28)) == -2
    assert _read(batch=dict(n_rows=1 << 28)) == -2
    assert _commit(batch=dict(n_req=1 << 22)) == -2
    assert _tree(scale=2.0 ** 101) == -1


def test_workspace_apart_from_the_rest():
    need = K._fns().dflash_tree_attention_workspace_size(_structs()[0], 2, 4, 32)
    assert need > 0
    for at in (1 << 40, 2 << 40, 8 << 40, 9 << 40):     # the cache's K and V, q, out
        assert _tree(ws=at, ws_bytes=need) == -1, at
    assert _tree(cache=SCALED, ws=6 << 40, ws_bytes=1 << 60) == -1


def test_cache_object_refuses_what_is_no_cache():
    k = torch.empty((4, 2, 16, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        D.KVCache(k, k)
    with pytest.raises(ValueError, match="one cache type"):
        D.KVCache(k, k.float())
    with pytest.raises(ValueError, match="one cache type"):
        D.KVCache(k[0], k[0])
    with pytest.raises(ValueError, match="8-bit"):
        D.KVCache(k.to(torch.int8), k.to(torch.int8))
    with pytest.raises(ValueError, match="8-bit"):
        D.KVCache(k, k, torch.empty(0), torch.empty(0))
