"""GPU tests of calls of the KV cache's operators at the ends of what they
allow: idle steps, kept workspaces, layouts and sizes beside the usual ones."""
import pytest
import torch

import block_draft_proposal_amd as D
from gpu_helpers import DEV, require_gpu, say
from kv_helpers import TYPES, make_plan, rand_rows
from test_gpu_tree_attention import build

pytestmark = pytest.mark.gpu


def test_an_idle_step_with_a_tree_mask():
    require_gpu()
    say("no rows, a mask of none")
    s = build("bf16", [50, 20], [4, 6], 16, 2, 4, 64, "tree", seed=13)
    kw = dict(s["kw"], mask=s["kw"]["mask"][:0])
    assert kw["mask"].shape[1] == 1
    assert D.dflash_tree_attention(s["q"][:0], s["cache"], **kw).shape == (0, 8, 64)
    with pytest.raises(ValueError, match="words"):
        D.dflash_tree_attention(s["q"], s["cache"], **dict(s["kw"], mask=s["kw"]["mask"][:, :0].contiguous()))
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("i8", 64), ("bf16", 256)])
def test_one_workspace_for_the_largest_tree_serves_every_smaller_one(kind, dim):
    require_gpu()
    say(f"kept workspace {kind} {dim}")
    s = build(kind, [300, 20], [64, 30], 16, 2, 4, dim, "tree", seed=14)
    size = D.tree_attention_workspace_size(s["cache"], n_req=2, max_nodes=64, n_q_heads=8)
    work = torch.empty(size, dtype=torch.uint8, device=DEV)
    off = s["kw"]["offsets"]
    for nodes in (64, 33, 20, 16, 9, 8, 1):
        kw = dict(s["kw"], max_nodes=nodes, offsets=torch.stack([off[0], off[0] + nodes, off[0] + nodes + min(nodes, 30)]))
        out = D.dflash_tree_attention(s["q"], s["cache"], workspace=work, **kw)
        want = D.dflash_tree_attention(s["q"], s["cache"], **kw)
        n = nodes + min(nodes, 30)
        assert torch.equal(out[:n], want[:n]), nodes


def _one_pool(kind, n_pages, heads, page, dim, gap):
    """K, V and their scales side by side in each page of one buffer, `gap`
    bytes between pages; the buffer, and the cache on it."""
    codes, scales = heads * page * dim, heads * page
    whole = -(-(2 * codes + 2 * scales + gap) // 16) * 16
    pool = torch.full((n_pages * whole,), 77, dtype=torch.uint8, device=DEV)
    k, v = (pool.view(TYPES[kind]).as_strided((n_pages, heads, page, dim), (whole, page * dim, dim, 1), i * codes) for i in range(2))
    ks, vs = (pool.as_strided((n_pages, heads, page), (whole, page, 1), 2 * codes + i * scales) for i in range(2))
    return pool, whole, D.KVCache(k, v, ks, vs)


@pytest.mark.parametrize("gap", [0, 32])
@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_one_pool_for_codes_and_scales(kind, gap):
    require_gpu()
    say(f"one pool {kind} {gap}")
    heads, page, dim = 3, 20, 64
    (table, st, off), host, n_pages, n_rows = make_plan([3, 0, 41], [30, 7, 12], page)
    pool, whole, one = _one_pool(kind, n_pages, heads, page, dim, gap)
    apart = D.KVCache(*(None if t is None else t.contiguous() for t in (one.k, one.v, one.k_scale, one.v_scale)))
    k, v = rand_rows(n_rows, heads, dim, "bf16", 41), rand_rows(n_rows, heads, dim, "bf16", 42)
    paths = torch.tensor([[0, 4, 9, 20], [1, 2, 5, 6], [0, 3, 4, 11]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([4, 3, 4], dtype=torch.int32, device=DEV)
    for c in (one, apart):
        D.dflash_kv_write(c, k, v, page_table=table, start=st, offsets=off)
        D.dflash_kv_commit(c, page_table=table, start=st, paths=paths, path_lens=lens)
    torch.cuda.synchronize()
    for name in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(*(getattr(c, name).contiguous().view(torch.uint8) for c in (one, apart))), name
    used = 2 * heads * page * (dim + 1)
    assert (pool.view(n_pages, whole)[:, used:] == 77).all()
    reads = [D.dflash_kv_read(c, page_table=table, start=st, offsets=off, n_rows=n_rows) for c in (one, apart)]
    n = int(host[2][-1])
    for a, b in zip(*reads):
        assert torch.equal(a[:n], b[:n])


def test_overlapping_caches_are_refused_before_anything_is_written():
    require_gpu()
    say("overlapping cache")
    heads, page, dim = 2, 16, 64
    pool = torch.zeros(8 * heads * page * dim, dtype=torch.bfloat16, device=DEV)
    need = heads * page * dim
    make = lambda at: pool.as_strided((3, heads, page, dim), (2 * need, page * dim, dim, 1), at)  # noqa: E731
    (table, st, off), _, _, n_rows = make_plan([0], [20], page, spare=1)
    rows = [rand_rows(n_rows, heads, dim, "bf16", i) for i in (1, 2)]
    paths, lens = torch.tensor([[0, 3]], dtype=torch.int32, device=DEV), torch.tensor([2], dtype=torch.int32, device=DEV)
    for at in (0, 8, page * dim, need - 8, need + 8):
        cache = D.KVCache(make(0), make(at))
        with pytest.raises(D.DFlashError, match="overlap"):
            D.dflash_kv_write(cache, *rows, page_table=table, start=st, offsets=off)
        with pytest.raises(D.DFlashError, match="overlap"):
            D.dflash_kv_commit(cache, page_table=table, start=st, paths=paths, path_lens=lens)
    torch.cuda.synchronize()
    assert not pool.any()


def test_a_captured_step_that_makes_its_own_tensors():
    """Write, attention, commit and read in one graph, outputs and workspace
    made by the calls; every replay on new rows equals eager calls."""
    require_gpu()
    say("captured step, own tensors")
    s, e = (build("e4m3", [300, 20], [9, 5], 16, 2, 4, 128, "tree", seed=22) for _ in range(2))
    k, v = rand_rows(14, 2, 128, "bf16", 61, packed=False), rand_rows(14, 2, 128, "bf16", 62, packed=False)
    paths = torch.tensor([[0, 3, 8], [1, 2, 4]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([3, 2], dtype=torch.int32, device=DEV)

    def step(x):
        batch = {name: x["kw"][name] for name in ("page_table", "start", "offsets")}
        D.dflash_kv_write(x["cache"], k, v, **batch)
        out = D.dflash_tree_attention(x["q"], x["cache"], **x["kw"])
        D.dflash_kv_commit(x["cache"], page_table=batch["page_table"], start=batch["start"], paths=paths, path_lens=lens)
        return out[:14], *D.dflash_kv_read(x["cache"], n_rows=14, **batch)

    for x in (s, e):
        step(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(s)
    for i in range(4):
        k.copy_(rand_rows(14, 2, 128, "bf16", 70 + i, packed=False))
        v.copy_(rand_rows(14, 2, 128, "bf16", 80 + i, packed=False))
        graph.replay()
        want = step(e)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), i
