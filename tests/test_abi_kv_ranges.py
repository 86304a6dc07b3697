"""CPU checks of numbers beyond 32 bits: the C call takes 32-bit integers, and
a number that does not fit must not reach it cut down to one that does."""
import ctypes
import types

import pytest
import torch

import block_draft_proposal_amd as D
from block_draft_proposal_amd import kv as K
from test_abi_kv import CACHE

WRAPS = [(1 << 32) + 4, 1 << 31, -(1 << 32) + 4, -(1 << 31) - 1]


def _cache():
    struct = K.KVCacheStruct(**CACHE)
    return types.SimpleNamespace(device=torch.device("cpu"), head_dim=128, n_kv_heads=8, struct=struct, ref=ctypes.byref(struct))


@pytest.mark.parametrize("wrap", WRAPS)
def test_workspace_size(wrap):
    ok = dict(n_req=4, max_nodes=4, n_q_heads=32)
    assert D.tree_attention_workspace_size(_cache(), **ok) > 0
    for name in ok:
        with pytest.raises(ValueError, match=name):
            D.tree_attention_workspace_size(_cache(), **{**ok, name: wrap})


@pytest.mark.parametrize("wrap", WRAPS)
@pytest.mark.parametrize("mask", [False, True])
def test_attention_max_nodes(wrap, mask):
    q = torch.zeros((6, 32, 128), dtype=torch.bfloat16)
    kw = dict(page_table=torch.zeros((1, 4), dtype=torch.int32), start=torch.zeros(1, dtype=torch.int32),
              offsets=torch.zeros(2, dtype=torch.int32), mask=torch.zeros((6, 1), dtype=torch.int64) if mask else None)
    with pytest.raises(ValueError, match="max_nodes"):
        D.dflash_tree_attention(q, _cache(), max_nodes=wrap, **kw)


def test_shapes_of_tensors():
    """Tensors without memory, wider than 32 bits count."""
    meta = torch.device("meta")
    cache = _cache()
    cache.device = meta
    i32 = lambda *shape: torch.empty(shape, dtype=torch.int32, device=meta)  # noqa: E731
    wide = (1 << 32) + 4
    q = torch.empty((1, 32, 128), dtype=torch.bfloat16, device=meta)
    fine = dict(page_table=i32(1, 4), start=i32(1), offsets=i32(2))
    with pytest.raises(ValueError, match="page_table"):
        D.dflash_tree_attention(q, cache, max_nodes=4, **{**fine, "page_table": i32(1, wide)})
    with pytest.raises(ValueError, match="page_table"):
        D.dflash_tree_attention(q, cache, max_nodes=4, page_table=i32(wide, 4), start=i32(wide), offsets=i32(wide + 1))
    with pytest.raises(ValueError, match="mask"):
        D.dflash_tree_attention(q, cache, max_nodes=4, mask=torch.empty((1, wide), dtype=torch.int64, device=meta), **fine)
    with pytest.raises(ValueError, match="n_q_heads"):
        D.dflash_tree_attention(torch.empty((1, wide - 4 + 32, 128), dtype=torch.bfloat16, device=meta), cache, max_nodes=4, **fine)
    with pytest.raises(ValueError, match="paths"):
        D.dflash_kv_commit(cache, page_table=i32(1, 4), start=i32(1), paths=i32(1, wide), path_lens=i32(1))
    for shape in ((1, 1, 1, (1 << 32) + 64), (1, 1, (1 << 32) + 1, 64), (1, (1 << 32) + 1, 1, 64)):
        k = torch.empty(shape, dtype=torch.bfloat16, device=meta)
        with pytest.raises(ValueError, match="32 bits"):
            D.KVCache(k, k)
