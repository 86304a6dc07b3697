"""GPU tests of the KV cache and the tree attention at the ends of the ranges
that the header names: thousands of nodes, large pages, many heads, other
layouts of the rows, requests past their table, long runs of empty requests."""
import numpy as np
import pytest
import torch

import block_draft_proposal_amd as D
from gpu_helpers import DEV, require_gpu, say
from kv_helpers import (attention_bound, codes_f64, dead_cache, make_plan, mask_tensor, oracle_cache, rand_rows,
                        tree_mask)
from oracle import kv_oracle as O
from test_gpu_tree_attention import build, check

pytestmark = pytest.mark.gpu


def _dense_reference(s, see):
    """One request's attention in fp64 by dense products: out, spread and reach
    as the oracle gives them.  see bool [n, start + n]."""
    cache, (table, start, offsets) = s["cache"], s["host"]
    n, a = int(offsets[1]), int(start[0])
    model = oracle_cache(*s["tensors"])
    k, v = (torch.from_numpy(np.stack([O.row_at(model, x, table[0], t) for t in range(a + n)])).to(DEV) for x in "kv")
    q = s["q"][:n].double()
    group, scale = q.shape[1] // cache.n_kv_heads, cache.head_dim ** -0.5
    see = torch.from_numpy(see).to(DEV)
    outs, spreads, reaches = [], [], []
    for h in range(q.shape[1]):
        kk, vv, qq = k[:, h // group].contiguous(), v[:, h // group].contiguous(), q[:, h].contiguous()
        none = ~see.any(-1, keepdim=True)
        w = torch.softmax((scale * (qq @ kk.T.contiguous())).masked_fill(~see, -np.inf).masked_fill(none, 0), -1).masked_fill(none, 0)
        outs.append(w @ vv)
        spreads.append(w @ vv.abs())
        reaches.append((scale * (qq.abs() @ kk.abs().T.contiguous())).masked_fill(~see, 0).amax(-1))
    return [torch.stack(x, 1).cpu().numpy() for x in (outs, spreads, reaches)]


@pytest.mark.parametrize("kind,dim,group", [("bf16", 128, 1), ("e4m3", 64, 2), ("i8", 256, 1), ("bf16", 64, 3)])
@pytest.mark.parametrize("mask", ["chain", "random"])
@pytest.mark.parametrize("nodes,start", [(4096, 37), (4095, 0), (700, 2000)])
def test_thousands_of_nodes(nodes, start, mask, kind, dim, group):
    """A prompt as one chain, and masks of up to 64 words, rows that see
    nothing among them."""
    require_gpu()
    say(f"{nodes} nodes {start} {mask} {kind} {dim} {group}")
    s = build(kind, [start], [nodes], 16, 1, group, dim, mask, seed=nodes % 91)
    out = torch.full(s["q"].shape, 3.0, dtype=torch.bfloat16, device=DEV)
    D.dflash_tree_attention(s["q"], s["cache"], out=out, **s["kw"])
    torch.cuda.synchronize()
    if mask == "chain":
        tree = np.tril(np.ones((nodes, nodes), dtype=bool))
    else:
        tree = np.unpackbits(s["bits"][:nodes].view(np.uint8), axis=-1, bitorder="little")[:, :nodes].astype(bool)
        assert start or not tree.any(-1).all()
    want, spread, reach = _dense_reference(s, np.concatenate([np.ones((nodes, start), dtype=bool), tree], axis=1))
    got = codes_f64(out)
    off = np.abs(got[:nodes] - want) / attention_bound(want, spread, reach, dim)
    assert np.isfinite(got).all() and off.max() <= 1.0, (off.max(), np.unravel_index(off.argmax(), off.shape))
    assert (got[nodes:] == 3.0).all()


@pytest.mark.parametrize("kind", ["bf16", "i8"])
@pytest.mark.parametrize("page", [257, 40000, 65535, 65536])
def test_large_pages(page, kind):
    """Positions on both sides of a page's end."""
    require_gpu()
    say(f"pages of {page} {kind}")
    s = build(kind, [page - 3, 2 * page - 1, 5], [7, 3, 2], page, 1, 2, 64, "tree", seed=page % 83, spare=0)
    check(s)
    outs = D.dflash_kv_read(s["cache"], page_table=s["kw"]["page_table"], start=s["kw"]["start"], offsets=s["kw"]["offsets"], n_rows=12)
    torch.cuda.synchronize()
    model, ref = oracle_cache(*s["tensors"]), [np.zeros((12, 1, 64)) for _ in "kv"]
    O.read(model, *s["host"], ref)
    for o, r in zip(outs, ref):
        np.testing.assert_array_equal(codes_f64(o), r)
    paths = np.array([[0, 2, 5, 6], [1, 2, 0, 0], [1, 0, 0, 0]], dtype=np.int32)
    lens = np.array([4, 2, 1], dtype=np.int32)
    D.dflash_kv_commit(s["cache"], page_table=s["kw"]["page_table"], start=s["kw"]["start"], paths=torch.from_numpy(paths).to(DEV),
                       path_lens=torch.from_numpy(lens).to(DEV))
    torch.cuda.synchronize()
    O.commit(model, s["host"][0], s["host"][1], paths, lens)
    moved = oracle_cache(*s["tensors"])
    for name in ("k", "v"):
        np.testing.assert_array_equal(moved[name], model[name])


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("heads,group", [(64, 2), (1024, 1)])
def test_many_heads(heads, group, kind):
    require_gpu()
    say(f"{heads} heads {group} {kind}")
    s = build(kind, [21, 0], [3, 2], 16, heads, group, 64, "tree", seed=31)
    check(s)
    n = int(s["host"][2][-1])
    outs = D.dflash_kv_read(s["cache"], page_table=s["kw"]["page_table"], start=s["kw"]["start"], offsets=s["kw"]["offsets"], n_rows=n)
    model, ref = oracle_cache(*s["tensors"]), [np.zeros((n, heads, 64)) for _ in "kv"]
    O.read(model, *s["host"], ref)
    paths, lens = np.array([[0, 2], [1, 0]], dtype=np.int32), np.array([2, 1], dtype=np.int32)
    D.dflash_kv_commit(s["cache"], page_table=s["kw"]["page_table"], start=s["kw"]["start"], paths=torch.from_numpy(paths).to(DEV),
                       path_lens=torch.from_numpy(lens).to(DEV))
    torch.cuda.synchronize()
    O.commit(model, s["host"][0], s["host"][1], paths, lens)
    moved = oracle_cache(*s["tensors"])
    for o, r, name in zip(outs, ref, "kv"):
        np.testing.assert_array_equal(codes_f64(o), r)
        np.testing.assert_array_equal(moved[name], model[name])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_rows_laid_out_head_first(kind, io):
    """[heads, rows, head_dim] seen as [rows, heads, head_dim]: the head's
    stride is the larger."""
    require_gpu()
    say(f"head first {kind} {io}")
    heads, dim = 3, 128
    (table, st, off), host, n_pages, n_rows = make_plan([40, 3], [11, 30], 16, seed=2)
    k, v = (rand_rows(n_rows, heads, dim, io, i, packed=False) for i in (51, 52))
    first = lambda x: x.transpose(0, 1).contiguous().transpose(0, 1)  # noqa: E731
    assert first(k).stride() == (dim, n_rows * dim, 1)
    caches = [dead_cache(kind, n_pages, heads, 16, dim) for _ in range(2)]
    D.dflash_kv_write(D.KVCache(*caches[0]), k, v, page_table=table, start=st, offsets=off)
    D.dflash_kv_write(D.KVCache(*caches[1]), first(k), first(v), page_table=table, start=st, offsets=off)
    torch.cuda.synchronize()
    for a, b in zip(*caches):
        assert a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    s = build(kind, [40, 3], [11, 30], 16, heads, 4, dim, "tree", seed=15)
    want = D.dflash_tree_attention(s["q"], s["cache"], **s["kw"])
    got = D.dflash_tree_attention(first(s["q"].contiguous()), s["cache"], **s["kw"])
    assert torch.equal(got[:41], want[:41])


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_a_mask_wider_than_its_nodes_need(kind):
    require_gpu()
    say(f"wide mask {kind}")
    check(build(kind, [33, 0], [10, 40], 16, 2, 3, 128, "random", seed=16, words=3))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_a_request_past_its_table_with_rows_that_see_nothing(kind):
    """Those are zeros, the request's others NaN, the other request as before."""
    require_gpu()
    say(f"past the table {kind}")
    s = build(kind, [0, 9], [40, 6], 16, 2, 4, 64, "tree", seed=17)
    s["bits"][[0, 7, 39]] = 0xFFFFFF0000000000          # only bits past the 40 nodes
    s["bits"][41] = 0                                   # sees its prefix
    s["kw"]["mask"] = mask_tensor(s["bits"])
    clean = codes_f64(D.dflash_tree_attention(s["q"], s["cache"], **s["kw"]))
    blind = np.zeros(40, dtype=bool)
    blind[[0, 7, 39]] = True
    assert (clean[:40][blind] == 0).all() and np.isfinite(clean[:46]).all()
    table = s["kw"]["page_table"]
    bad = table.clone()
    bad[0, 2] = -1                                      # a page that is not there
    for t in (table[:, :2].contiguous(), bad):          # or a table that ends at 32 positions
        got = codes_f64(D.dflash_tree_attention(s["q"], s["cache"], **dict(s["kw"], page_table=t)))
        assert (got[:40][blind] == 0).all()
        assert np.isnan(got[:40][~blind]).all()
        np.testing.assert_array_equal(got[40:46], clean[40:46])


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_the_largest_start_that_the_table_holds(kind):
    """Requests 0 and 2 start two positions before the table's end: 0's table
    row has entries of -1 there, 2's has pages, its last rows never written."""
    require_gpu()
    say(f"at the table's end {kind}")
    s = build(kind, [50, 20, 300], [4, 4, 2], 16, 2, 4, 128, "tree", seed=4)
    far = s["host"][0].shape[1] * 16 - 2
    s["host"][1][:] = [far, 20, far]
    s["kw"]["start"] = torch.tensor([far, 20, far], dtype=torch.int32, device=DEV)
    got, want = check(s)
    assert np.isnan(want[:4]).all() and np.isfinite(want[4:8]).all() and np.isnan(want[8:10]).all()
    s["host"][1][2] = far - 2                           # within what was written: as the oracle says
    s["kw"]["start"] = torch.tensor([far, 20, far - 2], dtype=torch.int32, device=DEV)
    tensors = s["cache"]
    for name in ("k", "v"):                             # the last page's rows behind the prefix hold ones
        t = getattr(tensors, name)
        (t.view(torch.uint8) if kind == "e4m3" else t)[int(s["host"][0][2, -1])] = 1
        if kind != "bf16":
            getattr(tensors, name + "_scale")[int(s["host"][0][2, -1])] = 127
    got, want = check(s)
    assert np.isnan(want[:4]).all() and np.isfinite(want[4:10]).all()


@pytest.mark.parametrize("kind", ["bf16", "i8"])
def test_long_runs_of_requests_without_rows(kind):
    """20000 requests of which five have rows, the first and the last among them."""
    require_gpu()
    say(f"empty requests {kind}")
    rows, start = np.zeros(20000, dtype=np.int64), np.zeros(20000, dtype=np.int64)
    for r, n, a in ((0, 2, 30), (1, 1, 0), (9999, 3, 64), (10001, 1, 5), (19999, 4, 17)):
        rows[r], start[r] = n, a
    s = build(kind, start.tolist(), rows.tolist(), 16, 1, 2, 64, "tree", seed=18)
    check(s)
    n = int(s["host"][2][-1])
    outs = D.dflash_kv_read(s["cache"], page_table=s["kw"]["page_table"], start=s["kw"]["start"], offsets=s["kw"]["offsets"], n_rows=n)
    ref = [np.zeros((n, 1, 64)) for _ in "kv"]
    O.read(oracle_cache(*s["tensors"]), *s["host"], ref)
    for o, r in zip(outs, ref):
        np.testing.assert_array_equal(codes_f64(o), r)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("max_nodes", [1, 64, 4096])
def test_room_for_more_nodes_than_sent(kind, max_nodes):
    """max_nodes chooses the kernel's form, never the result beyond its bound."""
    require_gpu()
    say(f"room for {max_nodes} {kind}")
    check(build(kind, [700, 90, 3], [1, 1, 1], 16, 2, 8, 128, "chain", seed=19, max_nodes=max_nodes))
