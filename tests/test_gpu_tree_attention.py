"""GPU tests of the draft-tree attention through the C ABI against the float64
oracle, within a bound derived from the arithmetic (kv_helpers.attention_bound)."""
import numpy as np
import pytest
import torch

import block_draft_proposal_amd as D
from gpu_helpers import DEV, require_gpu, say
from kv_helpers import (TYPES, attention_bound, codes_f64, dead_cache, make_plan, mask_tensor, oracle_cache, rand_rows,
                        tree_mask)
from oracle import kv_oracle as O

pytestmark = pytest.mark.gpu


def build(kind, start, rows, page, heads, group, dim, mask="tree", seed=0, words=None, max_nodes=None, spare=2):
    """Everything one call needs, the cache filled by dflash_kv_write."""
    (table, st, off), host, n_pages, n_rows = make_plan(start, rows, page, seed=seed, spare=spare)
    tensors = dead_cache(kind, n_pages, heads, page, dim)
    cache = D.KVCache(*tensors)
    total = [int(s + n) for s, n in zip(start, rows)]
    every = torch.tensor(np.concatenate([[0], np.cumsum(total)]), dtype=torch.int32, device=DEV)
    n = max(1, int(sum(total)))
    D.dflash_kv_write(cache, rand_rows(n, heads, dim, "bf16", seed + 1), rand_rows(n, heads, dim, "bf16", seed + 2),
                      page_table=table, start=torch.zeros_like(st), offsets=every)
    max_nodes = max_nodes or max(1, max(rows))
    bits = None if mask == "chain" else tree_mask(n_rows, host[2], words or -(-max_nodes // 64), seed, mask)
    return dict(cache=cache, tensors=tensors, host=host, n_rows=n_rows, bits=bits, q=rand_rows(n_rows, heads * group, dim, "bf16", seed + 3),
                kw=dict(page_table=table, start=st, offsets=off, max_nodes=max_nodes, mask=mask_tensor(bits)))


def check(s, scale=None, out=None, want_cache=None):
    dim = s["cache"].head_dim
    out = torch.full(s["q"].shape, 3.0, dtype=torch.bfloat16, device=DEV) if out is None else out
    D.dflash_tree_attention(s["q"], s["cache"], scale=scale, out=out, **s["kw"])
    torch.cuda.synchronize()
    want = np.full(out.shape, 3.0)
    spread, reach = O.tree_attention(codes_f64(s["q"]), want_cache or oracle_cache(*s["tensors"]), s["host"][0], s["host"][1],
                                     s["host"][2], s["bits"], dim ** -0.5 if scale is None else scale, want)
    got = codes_f64(out)
    nan = np.isnan(want)
    np.testing.assert_array_equal(np.isnan(got), nan)
    with np.errstate(invalid="ignore"):
        off = np.abs(got - want) / attention_bound(want, spread, reach, dim)
    off[nan | (got == want)] = 0
    assert off.max() <= 1.0, (off.max(), np.unravel_index(off.argmax(), off.shape))
    return got, want


CASES = [
    # start, rows, page, kv heads, group, dim, mask
    ([0], [1], 16, 1, 1, 64, "chain"),
    ([1], [1], 16, 2, 4, 128, "tree"),
    ([130], [1], 16, 8, 4, 128, "chain"),
    ([63, 64, 65, 0, 127], [1, 2, 3, 4, 0], 16, 2, 3, 64, "tree"),
    ([31, 500, 0, 77], [16, 16, 16, 16], 20, 2, 4, 128, "chain"),
    ([200, 3, 128], [10, 7, 10], 32, 1, 7, 64, "random"),
    ([0, 0, 40], [33, 65, 1], 64, 1, 2, 128, "random"),
    ([300, 50], [60, 61], 64, 2, 8, 128, "tree"),
    ([90, 10], [100, 130], 100, 1, 5, 64, "full"),
    ([257, 31], [9, 20], 8, 2, 2, 256, "tree"),
    ([41], [5], 1, 2, 16, 256, "random"),
    ([70, 2], [3, 3], 16, 1, 64, 128, "random"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"s{c[0][0]}n{max(c[1])}p{c[2]}h{c[3]}g{c[4]}d{c[5]}{c[6]}")
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_against_the_oracle(case, kind):
    require_gpu()
    start, rows, page, heads, group, dim, mask = case
    say(f"tree attention {case} {kind}")
    check(build(kind, start, rows, page, heads, group, dim, mask, seed=sum(start) % 97))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_long_ragged_batch(kind):
    """Contexts of very different lengths in one batch, split over many workgroups."""
    require_gpu()
    say(f"ragged {kind}")
    check(build(kind, [9000, 1, 0, 700, 2111, 0, 64], [4, 4, 0, 1, 3, 2, 4], 16, 2, 3, 128, "tree", seed=5))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_large_scores(kind):
    """A sharp softmax: the running maximum moves often, most weights underflow."""
    require_gpu()
    say(f"large scores {kind}")
    check(build(kind, [700, 200], [6, 9], 16, 2, 4, 128, "tree", seed=8), scale=0.5)


def test_rows_that_see_nothing_are_zero():
    require_gpu()
    say("empty rows")
    s = build("bf16", [0, 0], [5, 3], 16, 2, 2, 64, "random", seed=2)
    s["bits"][:] = 0xFFFFFFFFFFFFFFE0                   # only bits past the nodes
    s["bits"][5:8] = 0
    s["bits"][6] = 1
    s["kw"]["mask"] = mask_tensor(s["bits"])
    got, _ = check(s)
    assert (got[:6] == 0).all() and (got[7] == 0).all() and (got[6] != 0).any()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf"), -3.0e38])
@pytest.mark.parametrize("nodes", [7, 40])
def test_what_a_node_does_not_see_has_no_effect(bad, nodes):
    """One node's K and V hold NaN, infinities or the type's lowest values: the
    nodes that do not see it are as without it."""
    require_gpu()
    say(f"masked {bad} {nodes}")
    s = build("bf16", [37, 100], [nodes, nodes], 16, 2, 4, 128, "tree", seed=6)
    clean = codes_f64(D.dflash_tree_attention(s["q"], s["cache"], **s["kw"]))
    for node, name in ((3, "k"), (3, "v"), (5, "v")):
        for r in range(2):
            t = int(s["host"][1][r]) + node
            getattr(s["cache"], name)[int(s["host"][0][r, t // 16]), :, t % 16] = bad
    dirty = codes_f64(D.dflash_tree_attention(s["q"], s["cache"], **s["kw"]))
    unseen = [i for i in range(2 * nodes) if not int(s["bits"][i, 0]) & 0b101000]
    assert len(unseen) > 4
    np.testing.assert_array_equal(dirty[unseen], clean[unseen])
    if not np.isfinite(bad):
        seen = [i for i in range(2 * nodes) if int(s["bits"][i, 0]) & 0b100000]
        assert not np.isfinite(dirty[seen]).any()


def test_scale_byte_nan_in_a_masked_place():
    require_gpu()
    say("masked NaN scale")
    s = build("e4m3", [20], [6], 16, 2, 2, 64, "tree", seed=3)
    clean = codes_f64(D.dflash_tree_attention(s["q"], s["cache"], **s["kw"]))
    page, slot = int(s["host"][0][0, 24 // 16]), 24 % 16
    s["cache"].k_scale[page, :, slot] = 255
    s["cache"].v_scale[page, :, slot] = 255
    dirty = codes_f64(D.dflash_tree_attention(s["q"], s["cache"], **s["kw"]))
    for i in range(6):
        if int(s["bits"][i, 0]) & 16:
            assert np.isnan(dirty[i]).all()
        else:
            np.testing.assert_array_equal(dirty[i], clean[i])


@pytest.mark.parametrize("kind", ["bf16", "i8"])
def test_positions_without_a_page_make_the_request_nan(kind):
    require_gpu()
    say(f"bad page {kind}")
    s = build(kind, [50, 20, 300], [4, 4, 2], 16, 2, 4, 128, "tree", seed=4)
    clean = codes_f64(D.dflash_tree_attention(s["q"], s["cache"], **s["kw"]))
    table = s["kw"]["page_table"].clone()
    table[0, 1], table[2, 7] = s["cache"].n_pages, -5
    s["kw"]["page_table"] = table
    got = codes_f64(D.dflash_tree_attention(s["q"], s["cache"], **s["kw"]))
    assert np.isnan(got[:4]).all() and np.isnan(got[8:10]).all()
    np.testing.assert_array_equal(got[4:8], clean[4:8])
    s["kw"]["page_table"] = s["kw"]["page_table"][:, :3].contiguous()      # request 2 runs past the table
    got = codes_f64(D.dflash_tree_attention(s["q"], s["cache"], **s["kw"]))
    assert np.isnan(got[8:10]).all()
    np.testing.assert_array_equal(got[4:8], clean[4:8])


def test_padding_and_rows_beyond_max_nodes_are_left():
    require_gpu()
    say("rows left alone")
    s = build("bf16", [20, 5], [6, 9], 16, 1, 2, 64, "chain", seed=5)
    s["kw"]["max_nodes"] = 7
    out = torch.full(s["q"].shape, 3.0, dtype=torch.bfloat16, device=DEV)
    D.dflash_tree_attention(s["q"], s["cache"], out=out, **s["kw"])
    torch.cuda.synchronize()
    left = (out == 3.0).all(-1).all(-1).cpu().numpy()
    assert left.tolist() == [False] * 6 + [False] * 7 + [True] * 2 + [True] * (s["n_rows"] - 15)


def test_same_result_every_time_and_in_a_graph():
    """No order of arrival changes a bit; a captured call replayed over a
    growing context equals eager calls, the workspace shared by two graphs."""
    require_gpu()
    say("repeats and graphs")
    s = build("bf16", [3000, 900], [5, 5], 16, 2, 4, 128, "tree", seed=9)
    size = D.tree_attention_workspace_size(s["cache"], n_req=2, max_nodes=5, n_q_heads=8)
    work = torch.empty(max(1, size), dtype=torch.uint8, device=DEV)
    outs = [torch.zeros(s["q"].shape, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    first = D.dflash_tree_attention(s["q"], s["cache"], **s["kw"]).clone()
    graphs = []
    for i in range(2):
        D.dflash_tree_attention(s["q"], s["cache"], out=outs[i], workspace=work, **s["kw"])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            D.dflash_tree_attention(s["q"], s["cache"], out=outs[i], workspace=work, **s["kw"])
        graphs.append(g)
    start = s["kw"]["start"]
    for step in range(4):
        for g in graphs:
            g.replay()
        work.random_(0, 255)                            # a call relies on nothing that a workspace holds
        graphs[step % 2].replay()
        D.dflash_tree_attention(s["q"], s["cache"], out=outs[2], **s["kw"])
        torch.cuda.synchronize()
        n = int(s["host"][2][-1])
        assert torch.equal(outs[0][:n], outs[2][:n]) and torch.equal(outs[1][:n], outs[2][:n])
        if step == 0:
            assert torch.equal(outs[2][:n], first[:n])
        start -= torch.tensor([700, 1], dtype=torch.int32, device=DEV)


def test_two_calls_at_once_on_two_streams():
    require_gpu()
    say("two streams")
    a, b = (build(kind, [2500, 40], [6, 16], 16, 2, 4, 128, "tree", seed=20 + i) for i, kind in enumerate(("bf16", "i8")))
    ref = [D.dflash_tree_attention(s["q"], s["cache"], **s["kw"]).clone() for s in (a, b)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.zeros(s["q"].shape, dtype=torch.bfloat16, device=DEV) for s in (a, b)]
    works = [torch.empty(max(1, D.tree_attention_workspace_size(s["cache"], n_req=2, max_nodes=16, n_q_heads=8)),
                         dtype=torch.uint8, device=DEV) for s in (a, b)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, w, st in zip((a, b), outs, works, streams):
            D.dflash_tree_attention(s["q"], s["cache"], out=o, workspace=w, stream=st, **s["kw"])
    torch.cuda.synchronize()
    for o, r in zip(outs, ref):
        assert torch.equal(o[:22], r[:22])


@pytest.mark.parametrize("n_req", [300, 1100])
def test_many_requests(n_req):
    require_gpu()
    say(f"{n_req} requests")
    rng = np.random.default_rng(n_req)
    s = build("i8", rng.integers(0, 90, size=n_req).tolist(), rng.integers(0, 4, size=n_req).tolist(), 16, 1, 2, 64, "tree", seed=7)
    check(s)


def test_offsets_beyond_32_bits():
    require_gpu()
    heads, page, dim = 2, 16, 128
    need = heads * page * dim
    pool = torch.empty(2 * (1 << 30) + 1024 * need, dtype=torch.bfloat16, device=DEV)
    k = pool.as_strided((3, heads, page, dim), ((1 << 30) + 64, page * dim, dim, 1))
    v = pool.as_strided((3, heads, page, dim), ((1 << 30) + 64, page * dim, dim, 1), storage_offset=need)
    s = build("bf16", [40], [5], page, heads, 4, dim, "tree", seed=1, spare=0)
    k.copy_(s["cache"].k)
    v.copy_(s["cache"].v)
    say("pages 2 GiB apart")
    far = D.dflash_tree_attention(s["q"], D.KVCache(k, v), **s["kw"])
    near = D.dflash_tree_attention(s["q"], s["cache"], **s["kw"])
    torch.cuda.synchronize()
    assert torch.equal(far[:5], near[:5])


WIDE = [
    # more than 128 rows to a kv head: pairs of 128-row tiles, and odd numbers of them
    ([300, 5, 0], [64, 20, 33], 16, 1, 4, 128, "tree"),
    ([77], [130], 20, 2, 2, 128, "random"),
    ([40, 129], [300, 1], 16, 1, 1, 64, "random"),
    ([1000, 10], [200, 7], 32, 1, 2, 64, "tree"),
    ([129, 0], [16, 2], 16, 1, 64, 128, "random"),
    ([50, 600], [30, 64], 16, 2, 8, 256, "tree"),
    ([5, 260], [140, 100], 1, 1, 2, 128, "chain"),
]


@pytest.mark.parametrize("case", WIDE, ids=lambda c: f"s{c[0][0]}n{max(c[1])}p{c[2]}h{c[3]}g{c[4]}d{c[5]}{c[6]}")
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_many_rows_to_a_kv_head(case, kind):
    require_gpu()
    start, rows, page, heads, group, dim, mask = case
    say(f"tree attention {case} {kind}")
    check(build(kind, start, rows, page, heads, group, dim, mask, seed=sum(start) % 89))


@pytest.mark.parametrize("dim", [64, 128])
def test_a_long_context_in_many_pieces_and_room_for_many_nodes(dim):
    """Items cut into more than eight pieces; max_nodes far above the nodes."""
    require_gpu()
    say(f"many pieces {dim}")
    check(build("e4m3", [9000, 2], [5, 3], 16, 1, 4, dim, "tree", seed=8, max_nodes=4096))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("nodes", [40, 64])
@pytest.mark.parametrize("start", [20, 9000])
def test_unseen_values_of_wide_and_cut_items(kind, nodes, start):
    require_gpu()
    say(f"masked values {kind} {nodes} {start}")
    s = build(kind, [start], [nodes], 16, 1, 8, 128, "tree", seed=11)
    clean = codes_f64(D.dflash_tree_attention(s["q"], s["cache"], **s["kw"]))
    at = start + 5
    v = s["cache"].v.view(torch.uint8) if kind == "e4m3" else s["cache"].v
    v[int(s["host"][0][0, at // 16]), :, at % 16, 3::7] = 0x7F if kind == "e4m3" else float("-inf")
    dirty = codes_f64(D.dflash_tree_attention(s["q"], s["cache"], **s["kw"]))
    seen = np.array([bool(int(s["bits"][i, 0]) & 32) for i in range(nodes)])
    assert 2 < seen.sum() < nodes - 2
    np.testing.assert_array_equal(dirty[:nodes][~seen], clean[:nodes][~seen])
    np.testing.assert_array_equal(np.isfinite(dirty[:nodes][seen][..., 3::7]), False)
    rest = np.arange(128) % 7 != 3
    np.testing.assert_array_equal(dirty[:nodes][seen][..., rest], clean[:nodes][seen][..., rest])


def test_lengths_beyond_the_table_take_one_step():
    """A length that the table does not reach (up to the largest int32) makes
    its request NaN and leaves the others as they are."""
    require_gpu()
    say("lengths beyond the table")
    s = build("i8", [50, 20, 300], [4, 4, 2], 16, 2, 4, 128, "tree", seed=4)
    clean = codes_f64(D.dflash_tree_attention(s["q"], s["cache"], **s["kw"]))
    width = s["host"][0].shape[1]
    for far in (width * 16 - 3, 1 << 30, (1 << 31) - 1):
        s["kw"]["start"] = torch.tensor([far, 20, far], dtype=torch.int32, device=DEV)
        got = codes_f64(D.dflash_tree_attention(s["q"], s["cache"], **s["kw"]))
        assert np.isnan(got[:4]).all()
        assert np.isnan(got[8:10]).all() or far == width * 16 - 3
        np.testing.assert_array_equal(got[4:8], clean[4:8])


def test_strided_table_and_query_without_strides():
    require_gpu()
    say("strided table, expanded query")
    s = build("bf16", [50, 20], [4, 6], 16, 2, 4, 128, "tree", seed=12)
    want = D.dflash_tree_attention(s["q"], s["cache"], **s["kw"])
    table = s["kw"]["page_table"]
    wide = torch.full((2, table.shape[1] + 9), -1, dtype=torch.int32, device=DEV)
    wide[:, 2:2 + table.shape[1]] = table
    s["kw"]["page_table"] = wide[:, 2:-1]
    got = D.dflash_tree_attention(s["q"], s["cache"], **s["kw"])
    assert torch.equal(got[:10], want[:10])
    one = s["q"][:1, :1].expand(s["q"].shape)
    got = D.dflash_tree_attention(one, s["cache"], **s["kw"])
    want = D.dflash_tree_attention(one.contiguous(), s["cache"], **s["kw"])
    assert torch.equal(got[:10], want[:10])


def test_no_rows_and_no_requests():
    require_gpu()
    say("nothing to do")
    s = build("bf16", [50, 20], [4, 6], 16, 2, 4, 64, "chain", seed=13)
    kw = dict(s["kw"], page_table=s["kw"]["page_table"][:0], start=s["kw"]["start"][:0], offsets=s["kw"]["offsets"][:1])
    assert D.dflash_tree_attention(s["q"], s["cache"], **kw).shape == s["q"].shape
    assert D.dflash_tree_attention(s["q"][:0], s["cache"], **s["kw"]).shape[0] == 0
    torch.cuda.synchronize()


def test_new_tensors_of_a_call_on_another_stream_are_its_own():
    """The workspace that a call makes is given to nobody while the call's
    stream still has to run it."""
    require_gpu()
    say("workspace of another stream")
    s = build("bf16", [2500, 40], [6, 16], 16, 2, 4, 128, "tree", seed=21)
    want = D.dflash_tree_attention(s["q"], s["cache"], **s["kw"]).clone()
    size = D.tree_attention_workspace_size(s["cache"], n_req=2, max_nodes=16, n_q_heads=8)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    got = D.dflash_tree_attention(s["q"], s["cache"], stream=side, **s["kw"])
    others = [torch.zeros(size, dtype=torch.uint8, device=DEV) for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got[:22], want[:22]) and not any(x.any() for x in others)
