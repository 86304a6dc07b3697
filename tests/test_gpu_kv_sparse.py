"""GPU parity of the bounds of pages, the choice of blocks and the attention
over them with the float64 oracle."""
import numpy as np
import pytest
import torch

import block_draft_proposal_amd as D
from gpu_helpers import DEV, require_gpu, say
from kv_helpers import attention_bound, codes_f64, dead_cache, make_plan, mask_tensor, oracle_cache, rand_rows, tree_mask
from oracle import sparse_oracle as S

pytestmark = pytest.mark.gpu


def gpu(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.array(x, dtype=dtype))).to(DEV)


def written(kind, start, rows, page, heads, dim, seed=0, spare=2):
    """A cache that holds every request's start + rows positions, dead memory elsewhere."""
    plan, host, n_pages, n_rows = make_plan(start, rows, page, seed=seed, spare=spare)
    tensors = dead_cache(kind, n_pages, heads, page, dim)
    cache = D.KVCache(*tensors)
    total = np.asarray(start) + np.asarray(rows)
    ends = np.concatenate([[0], np.cumsum(total)])
    k, v = rand_rows(int(ends[-1]), heads, dim, "bf16", seed + 1), rand_rows(int(ends[-1]), heads, dim, "bf16", seed + 2)
    D.dflash_kv_write(cache, k, v, page_table=plan[0], start=gpu(np.zeros(len(total))), offsets=gpu(ends))
    return cache, tensors, plan, host, n_rows


# --- bounds ---


def check_bounds(cache, tensors, table, host_table, start, end):
    b = D.KVBounds.empty(cache)
    b.codes.fill_(33)
    b.scale.fill_(44)
    want = np.full(tuple(b.codes.shape), 33, dtype=np.int64), np.full(tuple(b.scale.shape), 44, dtype=np.int64)
    D.dflash_kv_bounds(cache, b, page_table=table, start=gpu(start), end=gpu(end))
    torch.cuda.synchronize()
    S.bounds(oracle_cache(*tensors), *want, host_table, start, end)
    np.testing.assert_array_equal(b.scale.cpu().numpy(), want[1])
    np.testing.assert_array_equal(b.codes.cpu().numpy(), want[0])
    return b


@pytest.mark.parametrize("page", [1, 3, 16, 20, 65])
@pytest.mark.parametrize("kind,dim,heads", [("bf16", 64, 1), ("bf16", 128, 3), ("bf16", 256, 2), ("e4m3", 64, 2), ("e4m3", 128, 8),
                                            ("e4m3", 256, 1), ("i8", 64, 5), ("i8", 128, 2), ("i8", 256, 2)])
def test_bounds(kind, dim, heads, page):
    require_gpu()
    say(f"bounds {kind} {dim} {heads} {page}")
    start, rows = [0, 3 * page, 2 * page + 1, 5 * page - 1, 7, 0], [4 * page, 2 * page, page - 1, 1, 0, page - 1]
    cache, tensors, (table, _, _), host, _ = written(kind, start, rows, page, heads, dim)
    check_bounds(cache, tensors, table, host[0], start, [a + b for a, b in zip(start, rows)])


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_bounds_of_odd_keys(kind):
    """Infinities and NaN, values at the borders of the codes, the smallest and
    the largest, tiny ones beside them, zeros."""
    require_gpu()
    say(f"odd keys {kind}")
    page, heads, dim, pages = 4, 2, 64, 12
    rows = torch.zeros((pages * page, heads, dim), device=DEV)
    x = rows.view(pages, page, heads, dim)
    x[0, 1, 0, 5], x[0, 2, 1, 6] = float("inf"), float("nan")
    x[1, 0] = 127.0
    x[1, 1] = -127.0
    x[2, 0], x[2, 0, :, 3] = 1.0, 127.5
    x[3, 3, :, 7], x[3, 0, :, 8], x[3, 2, :, 9] = 3e38, 1e-38, -1e-38
    x[4, 0, :, 0] = 9.2e-41
    x[5, :, :, ::2], x[5, :, :, 1::2] = -2.0 ** -100, 2.0 ** -101
    x[6, 0] = -0.0
    x[7] = torch.arange(dim, device=DEV) - 31.5
    x[8, 2, 0, 1] = -float("inf")
    x[9, 1] = 448.0 * 2.0 ** 119
    x[10] = 2.0 ** -130
    x[10, 0, 0] = -(2.0 ** 20)
    cache = D.KVCache(*dead_cache(kind, pages + 1, heads, page, dim))
    table = torch.arange(pages, 0, -1, dtype=torch.int32, device=DEV)[None].contiguous()
    D.dflash_kv_write(cache, rows, rows, page_table=table, start=gpu([0]), offsets=gpu([0, pages * page]))
    tensors = [cache.k, cache.v, cache.k_scale, cache.v_scale]
    b = check_bounds(cache, tensors, table, table.cpu().numpy(), [0], [pages * page])
    assert b.scale[pages].tolist() == [255, 255] and (b.scale[:pages] == 255).sum() >= 1


def test_bounds_ignore_what_is_not_there():
    """Ranges that end before they begin, beyond the table, of pages outside the pool."""
    require_gpu()
    say("bounds out of range")
    cache, tensors, (table, _, _), host, _ = written("bf16", [0, 0, 0, 0], [40, 40, 40, 40], 8, 2, 64)
    table, host_table = table.clone(), host[0].copy()
    for b, bad in ((0, -1), (2, 99), (4, -2147483648)):
        table[1, b] = bad
        host_table[1, b] = bad
    check_bounds(cache, tensors, table, host_table, [-5, 0, 16, 2147483647], [24, 40, 8, -2147483648])
    check_bounds(cache, tensors, table, host_table, [39, 0, 0, 8], [2147483647, 7, 0, 8])


@pytest.mark.parametrize("n_req", [300, 2048, 2049])
def test_bounds_of_many_requests(n_req):
    """More requests than threads, and than the line holds; many with nothing to do."""
    require_gpu()
    say(f"bounds of {n_req}")
    rng = np.random.default_rng(n_req)
    page = 4
    start = rng.integers(0, 9, n_req)
    rows = np.where(rng.random(n_req) < 0.4, 0, rng.integers(0, 14, n_req))
    cache, tensors, (table, _, _), host, _ = written("i8", start, rows, page, 2, 64)
    check_bounds(cache, tensors, table, host[0], start, start + rows)


# --- the choice ---


def check_select(q, bounds, plan, host, take, n_first=1, n_last=1, max_nodes=None):
    table, start, offsets = plan
    n_rows = q.shape[0]
    out = torch.full((n_rows, bounds.n_kv_heads, take), -9, dtype=torch.int32, device=DEV)
    most = int((host[2][1:] - host[2][:-1]).max()) if max_nodes is None else max_nodes
    got = D.dflash_kv_select(q, bounds, page_table=table, start=start, offsets=offsets, max_nodes=max(1, most), n_first=n_first,
                             n_last=n_last, out=out)
    torch.cuda.synchronize()
    want = np.full(tuple(out.shape), -9, dtype=np.int64)
    S.select(codes_f64(q), bounds.codes.cpu().numpy(), bounds.scale.cpu().numpy(), bounds.n_pages, bounds.page_size, *host, take,
             n_first, n_last, want)
    if max_nodes is not None:
        for r in range(len(host[1])):
            want[host[2][r] + max_nodes:host[2][r + 1]] = -9
    np.testing.assert_array_equal(got.cpu().numpy(), want)
    return got


def rand_bounds(n_pages, heads, dim, page, seed, wide=127, scales=3):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    ends = torch.randint(-wide, wide + 1, (n_pages, heads, 2, dim), generator=gen, device=DEV)
    scale = torch.randint(120, 120 + scales, (n_pages, heads), generator=gen, device=DEV)
    return D.KVBounds(ends.sort(2).values.to(torch.int8), scale.to(torch.uint8), page_size=page)


@pytest.mark.parametrize("dim,heads,group,page,start,rows,take", [
    (128, 8, 4, 16, [700], [1], 8),
    (128, 2, 1, 16, [700, 33, 0, 15, 16, 4000], [1, 1, 1, 1, 1, 1], 5),
    (64, 1, 7, 20, [999, 3, 640], [2, 2, 1], 9),
    (128, 3, 5, 8, [333, 1000, 0, 77, 5000], [10, 3, 16, 0, 7], 20),
    (256, 2, 8, 32, [3000, 64, 1500], [16, 33, 5], 30),
    (256, 1, 64, 16, [500, 900], [16, 3], 6),
    (64, 2, 16, 1, [300, 70], [9, 1], 33),
    (128, 1, 20, 64, [6400, 64 * 300 + 63], [4, 17], 100),
])
def test_select(dim, heads, group, page, start, rows, take):
    require_gpu()
    say(f"select {dim} {heads} {group} {page} {take}")
    plan, host, n_pages, n_rows = make_plan(start, rows, page, seed=3)
    b = rand_bounds(n_pages, heads, dim, page, 5)
    q = rand_rows(n_rows, heads * group, dim, "bf16", 6)
    check_select(q, b, plan, host, take, n_first=0, n_last=0)
    check_select(q, b, plan, host, take, n_first=2, n_last=3)


@pytest.mark.parametrize("blocks", [4095, 4096, 4097, 9001])
def test_select_of_many_blocks(blocks):
    """More blocks than a segment holds, with few distinct scores."""
    require_gpu()
    say(f"select of {blocks}")
    plan, host, n_pages, n_rows = make_plan([blocks, blocks // 2], [1, 2], 1, seed=4)
    b = rand_bounds(n_pages, 1, 64, 1, 7, wide=1, scales=1)
    q = (rand_rows(n_rows, 2, 64, "bf16", 8) > 1).to(torch.bfloat16)
    check_select(q, b, plan, host, 130)
    check_select(q, b, plan, host, blocks - 1, n_first=0, n_last=0)


def test_select_ties_go_to_the_lower_block():
    require_gpu()
    say("ties")
    plan, host, n_pages, n_rows = make_plan([40, 41], [3, 1], 1, seed=9)
    b = rand_bounds(n_pages, 2, 64, 1, 7)
    b.codes.zero_()
    b.scale.fill_(127)
    q = rand_rows(n_rows, 4, 64, "bf16", 8)
    got = check_select(q, b, plan, host, 10, n_first=0, n_last=2)
    assert got[0, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 38, 39]
    b.codes.fill_(-3)
    b.codes[:, :, 1] = 100
    check_select(q, b, plan, host, 10)


def test_select_broken_blocks_and_queries():
    """Pages outside the pool and bounds of odd keys come before any score; a
    row with an infinity or a NaN scores 0 everywhere; smallest and largest scales."""
    require_gpu()
    say("broken blocks")
    plan, host, n_pages, n_rows = make_plan([320, 320, 320], [5, 1, 2], 16, seed=2)
    table, host_table = plan[0].clone(), host[0].copy()
    for r, blk, bad in ((0, 7, -1), (1, 12, n_pages), (2, 1, 2147483647)):
        table[r, blk] = bad
        host_table[r, blk] = bad
    b = rand_bounds(n_pages, 2, 128, 16, 7)
    b.scale.random_(27, 250)
    b.scale[::5, 0] = 255
    q = rand_rows(n_rows, 6, 128, "bf16", 8)
    q[1, 0, 3], q[2, 4, 7], q[3] = float("inf"), float("nan"), 0.0
    q[4] = 3e38
    q[5] = 1e-40
    check_select(q, b, (table, *plan[1:]), (host_table, *host[1:]), 9)
    check_select(q, b, (table, *plan[1:]), (host_table, *host[1:]), 2, n_first=1, n_last=1)
    check_select(q, b, (table, *plan[1:]), (host_table, *host[1:]), 40, n_first=20, n_last=20)


@pytest.mark.parametrize("blocks", [900, 5000])
def test_select_any_scale_byte(blocks):
    """Scores over the whole range of the bytes, which no other kernel writes:
    finite, and in order."""
    require_gpu()
    say(f"scale bytes {blocks}")
    plan, host, n_pages, n_rows = make_plan([blocks, blocks - 7], [3, 2], 1, seed=6)
    b = rand_bounds(n_pages, 2, 64, 1, 7)
    b.scale.random_(25, 256)
    b.scale[b.scale == 255] = 254                        # so that none is broken
    b.codes[::3] = b.codes.amin(2, keepdim=True)[::3]    # scores of either sign
    q = rand_rows(n_rows, 4, 64, "bf16", 8)
    for take in (3, 400, blocks - 9):
        check_select(q, b, plan, host, take, n_first=0, n_last=0)
    b.scale.random_(0, 25)
    low = D.KVBounds(b.codes, torch.full_like(b.scale, 25), page_size=1)
    kw = dict(page_table=plan[0], start=plan[1], offsets=plan[2], max_nodes=3, n_take=400)
    assert torch.equal(D.dflash_kv_select(q, b, **kw)[:host[2][-1]], D.dflash_kv_select(q, low, **kw)[:host[2][-1]])


@pytest.mark.parametrize("dim,heads,group,page,nodes,n_req", [(64, 8, 2, 16, 16, 19), (128, 16, 5, 8, 8, 15), (256, 8, 3, 16, 12, 20), (128, 8, 4, 1, 6, 25)])
def test_select_of_enough_rows_for_one_launch(dim, heads, group, page, nodes, n_req):
    """Tiles that hold parts of several requests, requests without rows or without
    blocks, and padding."""
    require_gpu()
    say(f"one launch {dim} {heads} {nodes}")
    rng = np.random.default_rng(dim + nodes)
    rows = rng.integers(0, nodes + 1, n_req)
    rows[:3] = nodes, 0, nodes
    start = rng.integers(0, 40 * page, n_req)
    start[5:8] = 0, page - 1, 40 * page
    plan, host, n_pages, n_rows = make_plan(start, rows, page, seed=3)
    b = rand_bounds(n_pages, heads, dim, page, 5)
    b.scale[::11] = 255
    q = rand_rows(n_rows, heads * group, dim, "bf16", 6)
    check_select(q, b, plan, host, 7, max_nodes=nodes)
    check_select(q, b, plan, host, 12, n_first=3, n_last=2, max_nodes=nodes)
    check_select(q, b, plan, host, 5, max_nodes=nodes - 1)


@pytest.mark.parametrize("scores", ["spread", "few", "one", "wide"])
@pytest.mark.parametrize("dim,nodes,n_req,blocks,take", [(128, 16, 18, 2000, 128), (64, 8, 33, 2300, 2200), (256, 16, 17, 700, 65), (64, 16, 40, 70, 64)])
def test_a_batch_chooses_as_its_requests_alone(dim, nodes, n_req, blocks, take, scores):
    """One launch for the batch's tiles, two for a request's few."""
    require_gpu()
    say(f"batch and alone {dim} {nodes} {blocks} {scores}")
    rng = np.random.default_rng(blocks)
    rows, start = np.full(n_req, nodes), rng.integers(blocks // 2, blocks + 1, n_req)
    rows[1::3] = nodes // 2 + 1
    start[0] = blocks
    plan, host, n_pages, n_rows = make_plan(start, rows, 1, seed=4)
    heads = 8
    b = rand_bounds(n_pages, heads, dim, 1, 7, wide=1 if scores == "few" else 127, scales=1 if scores == "few" else 3)
    if scores == "wide":
        b.scale.random_(27, 250)
    if scores == "one":
        b.codes.fill_(3)
        b.scale.fill_(127)
    q = rand_rows(n_rows, heads, dim, "bf16", 8)
    if scores == "few":
        q = (q > 1).to(torch.bfloat16)
    table, begin, offsets = plan
    got = D.dflash_kv_select(q, b, page_table=table, start=begin, offsets=offsets, max_nodes=nodes, n_take=take)
    for r in range(n_req):
        lo, hi = int(host[2][r]), int(host[2][r + 1])
        alone = D.dflash_kv_select(q[lo:hi], b, page_table=table[r:r + 1], start=begin[r:r + 1], offsets=gpu([0, hi - lo]),
                                   max_nodes=nodes, n_take=take)
        assert torch.equal(got[lo:hi], alone), r


def test_select_leaves_the_rest_alone():
    """Rows beyond max_nodes and padding keep what they held; lengths out of range."""
    require_gpu()
    say("select rest")
    plan, host, n_pages, n_rows = make_plan([64, 200, 32], [7, 2, 20], 16, seed=2)
    b = rand_bounds(n_pages, 1, 64, 16, 7)
    q = rand_rows(n_rows, 3, 64, "bf16", 8)
    for most in (1, 2, 5, 16, 19):
        check_select(q, b, plan, host, 3, max_nodes=most)
    start = gpu([-7, 2147483647, 31])
    check_select(q, b, (plan[0], start, plan[2]), (host[0], np.array([-7, 2147483647, 31]), host[2]), 3)


# --- attention over blocks ---


def pick(host, n_rows, heads, page, take, seed, kind="some"):
    """blocks [n_rows, heads, take] ascending, -1 behind."""
    rng = np.random.default_rng(seed)
    table, start, offsets = host
    out = np.full((n_rows, heads, take), -1, dtype=np.int32)
    for r in range(len(start)):
        full = S.n_blocks(start[r], page, table.shape[1])
        for row in range(offsets[r], offsets[r + 1]):
            for h in range(heads):
                m = min(full, take if kind == "all" else int(rng.integers(0, take + 1)))
                out[row, h, :m] = np.sort(rng.choice(full, m, replace=False)) if m else []
    return out


def check_sparse(cache, tensors, plan, host, n_rows, group, blocks, mask=None, seed=0, scale=None, max_nodes=None, q=None):
    heads, dim = cache.n_kv_heads, cache.head_dim
    q = rand_rows(n_rows, heads * group, dim, "bf16", seed + 9) if q is None else q
    most = max(1, int((host[2][1:] - host[2][:-1]).max())) if max_nodes is None else max_nodes
    out = torch.full((n_rows, heads * group, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    kw = dict(page_table=plan[0], start=plan[1], offsets=plan[2], max_nodes=most, mask=mask_tensor(mask), scale=scale)
    D.dflash_sparse_attention(q, cache, gpu(blocks), out=out, **kw)
    torch.cuda.synchronize()
    want = np.full(tuple(out.shape), 7.0)
    spread, reach = S.sparse_attention(codes_f64(q), oracle_cache(*tensors), *host, blocks, mask,
                                       dim ** -0.5 if scale is None else scale, want)
    got = codes_f64(out)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    off = np.abs(got - want)[ok] - attention_bound(want, spread, reach, dim)[ok]
    assert (off <= 0).all(), off.max()
    n = int(host[2][-1])
    assert (got[n:] == 7.0).all()
    return q, out, kw


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("dim,heads,group,page,start,rows,take,shape", [
    (128, 2, 4, 16, [200], [1], 5, None),
    (64, 1, 1, 1, [90, 0, 1], [1, 1, 1], 40, None),
    (128, 3, 7, 20, [333, 19, 0, 20, 100], [3, 1, 9, 0, 5], 6, "tree"),
    (256, 2, 5, 32, [300, 64], [6, 2], 4, "random"),
    (64, 2, 17, 8, [77, 200], [2, 3], 9, "full"),
    (128, 1, 40, 64, [500], [3], 6, "tree"),
    (256, 1, 64, 16, [130, 40], [2, 1], 7, None),
    (128, 1, 33, 33, [70, 3], [70, 1], 2, "random"),
    (128, 1, 4, 16, [200, 77, 0], [70, 33, 64], 6, "tree"),
    (64, 2, 1, 16, [300, 9], [40, 64], 9, "random"),
    (128, 2, 8, 16, [300, 500, 31], [16, 10, 8], 9, None),
    (256, 1, 4, 16, [300, 100], [16, 9], 9, "tree"),
    (128, 2, 3, 16, [120], [5], 3, "full"),
    (64, 1, 2, 1, [3000], [6], 500, "tree"),
])
def test_sparse(kind, dim, heads, group, page, start, rows, take, shape):
    require_gpu()
    say(f"sparse {kind} {dim} {heads} {group} {page} {shape}")
    cache, tensors, plan, host, n_rows = written(kind, start, rows, page, heads, dim)
    blocks = pick(host, n_rows, heads, page, take, 1)
    mask = None if shape is None else tree_mask(n_rows, host[2], -(-max(rows) // 64), kind=shape)
    check_sparse(cache, tensors, plan, host, n_rows, group, blocks, mask)


@pytest.mark.parametrize("kind,n_req,rows", [("bf16", 1, 1), ("i8", 2, 1), ("e4m3", 3, 1), ("e4m3", 3, 4), ("bf16", 1, 7), ("i8", 2, 3), ("i8", 40, 5), ("bf16", 150, 4)])
def test_sparse_splits(kind, n_req, rows):
    """From one item, split over many workgroups, to more than the chip holds."""
    require_gpu()
    say(f"splits {kind} {n_req}")
    most = 1300 if n_req <= 3 else 400                   # up to 1040 keys: four workgroups to an item
    start = [most - 13 * r if r % 3 == 0 else 40 * r for r in range(n_req)]
    cache, tensors, plan, host, n_rows = written(kind, start, [rows] * n_req, 16, 2, 64)
    blocks = pick(host, n_rows, 2, 16, 64 if n_req <= 3 else 24, 2, kind="all" if n_req <= 3 else "some")
    check_sparse(cache, tensors, plan, host, n_rows, 3, blocks)


@pytest.mark.parametrize("kind,dim,heads,n_req,rows", [
    ("bf16", 128, 16, 18, 1), ("bf16", 128, 16, 40, 1), ("bf16", 128, 16, 80, 1), ("i8", 64, 16, 50, 1), ("e4m3", 128, 32, 70, 1), ("bf16", 256, 16, 20, 1),
    ("bf16", 256, 16, 40, 1), ("i8", 256, 16, 20, 1), ("bf16", 128, 16, 20, 2), ("e4m3", 64, 32, 40, 3), ("i8", 128, 16, 70, 2), ("bf16", 256, 16, 33, 2)])
def test_sparse_of_fewer_waves_to_a_workgroup(kind, dim, heads, n_req, rows):
    """More items than workgroups run at once: four, two and one wave to each."""
    require_gpu()
    say(f"waves {kind} {dim} {heads} {n_req} {rows}")
    start = [170 - 7 * r % 150 for r in range(n_req)]
    cache, tensors, plan, host, n_rows = written(kind, start, [rows] * n_req, 16, heads, dim)
    check_sparse(cache, tensors, plan, host, n_rows, 2, pick(host, n_rows, heads, 16, 6, 2))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_all_blocks_are_the_whole_prefix(kind):
    """With every block chosen, it is the tree attention over the prefix."""
    require_gpu()
    say(f"all blocks {kind}")
    cache, tensors, plan, host, n_rows = written(kind, [100, 0, 31, 640], [5, 9, 1, 12], 16, 2, 128)
    blocks = pick(host, n_rows, 2, 16, 40, 3, kind="all")
    mask = tree_mask(n_rows, host[2], 1)
    q, out, kw = check_sparse(cache, tensors, plan, host, n_rows, 4, blocks, mask)
    dense = torch.full_like(out, 7.0)
    D.dflash_tree_attention(q, cache, out=dense, **kw)
    n = int(host[2][-1])
    # each is within half a step (2^-8) of weights and of the result of the same number
    assert ((out - dense)[:n].float().norm() <= 2.0 ** -7 * dense[:n].float().norm())


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_rows_that_see_nothing_and_blocks_that_name_nothing(kind):
    require_gpu()
    say(f"nothing {kind}")
    page, heads = 16, 2
    cache, tensors, plan, host, n_rows = written(kind, [0, 32, 48, 15], [3, 2, 2, 2], page, heads, 64)
    blocks = np.full((n_rows, heads, 4), -1, dtype=np.int32)
    blocks[3, 0] = [5, -7, 2, 2147483647]                # beyond the prefix's full pages
    blocks[4, 1] = [-1, -1, 0, -1]                       # a gap before an entry
    blocks[5, 0] = [2, 2, 0, 1]                          # not above the entry before: named once, and not at all
    mask = np.zeros((n_rows, 1), dtype=np.uint64)
    mask[1, 0] = 0b100
    mask[5, 0] = 0xfffffffffffffff0                       # bits past the nodes
    check_sparse(cache, tensors, plan, host, n_rows, 4, blocks, mask)
    check_sparse(cache, tensors, plan, host, n_rows, 4, blocks[:, :, :0], mask)


@pytest.mark.parametrize("rows", [[4, 6], [1, 1]])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("start", [[50, 20], [900, 700]])
def test_what_is_not_seen_has_no_effect(kind, rows, start):
    """Every row in turn, with NaN in all blocks that it has not chosen and in
    all nodes that it does not see, which other rows of its request do see."""
    require_gpu()
    say(f"unseen {kind} {rows} {start}")
    page, heads, dim = 8, 2, 128
    cache, tensors, plan, host, n_rows = written(kind, start, rows, page, heads, dim)
    blocks = pick(host, n_rows, heads, page, max(start) // page // 3, 5)
    mask = tree_mask(n_rows, host[2], 1)
    q, out, kw = check_sparse(cache, tensors, plan, host, n_rows, 4, blocks, mask)
    clean = oracle_cache(*tensors)
    want = np.full(tuple(out.shape), 7.0)
    spread, reach = S.sparse_attention(codes_f64(q), clean, *host, blocks, mask, dim ** -0.5, want)
    bound = attention_bound(want, spread, reach, dim)
    names = ("k", "v") if kind != "i8" else ("k_scale", "v_scale")
    bad = {"bf16": 0xff, "e4m3": 0x7f, "i8": 255}[kind]
    for r in range(2):
        n, full = int(host[2][r + 1] - host[2][r]), int(host[1][r]) // page
        for i in range(n):
            row = int(host[2][r]) + i
            for h in range(heads):
                keep = [getattr(cache, name).clone() for name in names]
                used = {int(b) for b in blocks[row, h]}
                for name in names:
                    t = getattr(cache, name).view(torch.uint8)
                    t[host[0][r, [b for b in range(full) if b not in used]].tolist()] = bad
                    for j in range(n):
                        if not (int(mask[row, 0]) >> j) & 1:
                            p = int(host[1][r]) + j
                            t[int(host[0][r, p // page]), :, p % page] = bad
                got = codes_f64(D.dflash_sparse_attention(q, cache, gpu(blocks), **kw))
                at = np.s_[row, 4 * h:4 * h + 4]
                assert (np.abs(got[at] - want[at]) <= bound[at]).all(), (row, h)
                # rows that see what is broken are NaN
                others = [x for x in range(int(host[2][r]), int(host[2][r + 1]))
                          if {int(b) for b in blocks[x, h] if b >= 0} - used or int(mask[x, 0]) & ~int(mask[row, 0]) & ((1 << n) - 1)]
                for x in others:
                    assert np.isnan(got[x, 4 * h:4 * h + 4]).any(), (row, x, h)
                for name, was in zip(names, keep):
                    getattr(cache, name).view(torch.uint8).copy_(was.view(torch.uint8))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("start", [40, 700])
def test_infinities_that_one_node_sees(kind, start):
    require_gpu()
    say(f"infinity {kind} {start}")
    page, heads, dim = 8, 1, 64
    cache, tensors, plan, host, n_rows = written(kind, [start], [3], page, heads, dim)
    full = start // page                                 # 87 blocks: keys for two workgroups
    blocks = np.full((n_rows, heads, full), -1, dtype=np.int32)
    blocks[0, 0], blocks[1, 0, :full - 1] = range(full), [b for b in range(full) if b != 1]
    p = int(host[0][0, 1])
    if kind == "bf16":
        cache.v[p, 0, 3, 5], cache.v[p, 0, 4, 6] = float("inf"), -float("inf")
    else:
        cache.v.view(torch.uint8)[p, 0, 3, 5] = 0x7f
    q, out, kw = check_sparse(cache, tensors, plan, host, n_rows, 3, np.where(blocks == 1, -1, blocks))
    got = D.dflash_sparse_attention(q, cache, gpu(blocks), **kw).float()
    assert not torch.isfinite(got[0, :, 5]).any() and torch.isfinite(got[0, :, 7:]).all() and torch.isfinite(got[1:3]).all()
    if kind == "bf16":
        assert (got[0, :, 5] == float("inf")).all() and (got[0, :, 6] == -float("inf")).all()


def test_pages_outside_the_pool_and_lengths_beyond_the_table():
    require_gpu()
    say("outside")
    page, heads = 8, 1
    cache, tensors, plan, host, n_rows = written("bf16", [40, 40, 20, 16], [2, 2, 2, 2], page, heads, 64)
    table, host_table = plan[0].clone(), host[0].copy()
    for r, b, bad in ((0, 1, -1), (1, 5, cache.n_pages), (2, 2, -5)):
        table[r, b] = bad
        host_table[r, b] = bad
    blocks = np.full((n_rows, heads, 2), -1, dtype=np.int32)
    blocks[0, 0], blocks[1, 0], blocks[3, 0] = [0, 1], [0, 2], [3, 4]
    # row 0 sees a page that is none, row 1 does not; the nodes of request 1 and the tail of 2 have no page
    q, out, kw = check_sparse(cache, tensors, (table, *plan[1:]), (host_table, *host[1:]), n_rows, 2, blocks)
    assert [bool(torch.isnan(out[i].float()).any()) for i in range(8)] == [True, False, True, True, True, True, False, False]
    far = dict(kw, start=gpu([2147483647, 47, 40, -3]))
    got = D.dflash_sparse_attention(q, cache, gpu(blocks), **far)
    assert torch.isnan(got[:2].float()).all() and torch.isnan(got[2:4].float()).all()     # 47 + 2 is past the table's 48
    assert not torch.isnan(got[6:8].float()).any()                                        # no prefix


def test_strided_queries_scales_and_streams():
    require_gpu()
    say("strides")
    cache, tensors, plan, host, n_rows = written("bf16", [100, 37], [3, 4], 16, 2, 64)
    blocks = pick(host, n_rows, 2, 16, 5, 6)
    wide = torch.randn((n_rows, 3, 8, 64), device=DEV).bfloat16()
    q = wide[:, 1].transpose(0, 1).contiguous().transpose(0, 1)       # heads apart, rows next to each other
    check_sparse(cache, tensors, plan, host, n_rows, 4, blocks, q=q, scale=1.0)
    check_sparse(cache, tensors, plan, host, n_rows, 4, blocks, q=wide[:, 2], scale=0.01)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    kw = dict(page_table=plan[0], start=plan[1], offsets=plan[2], max_nodes=4)
    want = D.dflash_sparse_attention(q, cache, gpu(blocks), **kw)
    at = gpu(blocks)
    torch.cuda.synchronize()
    got = D.dflash_sparse_attention(q, cache, at, stream=side, **kw)
    side.synchronize()
    assert torch.equal(got[:7], want[:7])


def test_rows_beyond_max_nodes_are_left_alone():
    require_gpu()
    say("beyond max_nodes")
    cache, tensors, plan, host, n_rows = written("i8", [100, 37], [3, 9], 16, 2, 64)
    blocks = pick(host, n_rows, 2, 16, 5, 6)
    q = rand_rows(n_rows, 4, 64, "bf16", 3)
    out = torch.full((n_rows, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    kw = dict(page_table=plan[0], start=plan[1], offsets=plan[2])
    D.dflash_sparse_attention(q, cache, gpu(blocks), max_nodes=5, out=out, **kw)
    want = D.dflash_sparse_attention(q, cache, gpu(blocks), max_nodes=9, **kw)
    assert torch.equal(out[:8], want[:8]) and (out[8:] == 7).all()


def test_one_workspace_serves_calls_of_any_size():
    require_gpu()
    say("one workspace")
    cache, tensors, plan, host, n_rows = written("e4m3", [400, 37, 90], [3, 9, 1], 16, 2, 64)
    blocks = pick(host, n_rows, 2, 16, 20, 6)
    q = rand_rows(n_rows, 8, 64, "bf16", 3)
    size = D.sparse_attention_workspace_size(cache, n_rows=n_rows, n_take=20, max_nodes=9, n_q_heads=8)
    work = torch.empty(size, dtype=torch.uint8, device=DEV)
    for n_req in (3, 2, 1):
        n = int(host[2][n_req])
        kw = dict(page_table=plan[0][:n_req], start=plan[1][:n_req], offsets=plan[2][:n_req + 1], max_nodes=9)
        got = D.dflash_sparse_attention(q[:n], cache, gpu(blocks[:n]), workspace=work, **kw)
        want = D.dflash_sparse_attention(q[:n], cache, gpu(blocks[:n]), **kw)
        assert torch.equal(got, want)


def test_a_step_from_write_to_commit_and_its_graph():
    """Write a prompt, bounds, choose, attend, commit, bounds of what became
    full; then the same calls captured, replayed on new rows."""
    require_gpu()
    say("whole step")
    page, heads, dim, n, nodes, take = 16, 2, 128, 3, 6, 4
    width, n_pages = 16, 60
    states = []
    for _ in range(2):
        cache = D.KVCache(*(torch.zeros((n_pages, heads, page, dim), dtype=torch.bfloat16, device=DEV) for _ in "kv"))
        b = D.KVBounds.empty(cache)
        table = torch.randperm(n_pages, generator=torch.Generator().manual_seed(1))[:n * width].view(n, width).int().to(DEV)
        lens = [130, 64, 7]
        ends = np.concatenate([[0], np.cumsum(lens)])
        rows = rand_rows(int(ends[-1]), heads, dim, "bf16", 1)
        D.dflash_kv_write(cache, rows, rows, page_table=table, start=gpu([0] * n), offsets=gpu(ends))
        D.dflash_kv_bounds(cache, b, page_table=table, start=gpu([0] * n), end=gpu(lens))
        states.append(dict(cache=cache, bounds=b, table=table, lens=gpu(lens)))
    offsets = gpu(np.arange(n + 1) * nodes)
    k, v = rand_rows(n * nodes, heads, dim, "bf16", 2, packed=False), rand_rows(n * nodes, heads, dim, "bf16", 3, packed=False)
    q = rand_rows(n * nodes, heads * 4, dim, "bf16", 4, packed=False)
    paths, kept = gpu([[0, 2, 5, 0, 0, 0], [0, 1, 2, 3, 4, 5], [0, 0, 0, 0, 0, 0]]), gpu([3, 6, 1])

    def step(s):
        batch = dict(page_table=s["table"], start=s["lens"], offsets=offsets)
        D.dflash_kv_write(s["cache"], k, v, **batch)
        blocks = D.dflash_kv_select(q, s["bounds"], max_nodes=nodes, n_take=take, **batch)
        out = D.dflash_sparse_attention(q, s["cache"], blocks, max_nodes=nodes, **batch)
        D.dflash_kv_commit(s["cache"], page_table=s["table"], start=s["lens"], paths=paths, path_lens=kept)
        end = s["lens"] + kept
        D.dflash_kv_bounds(s["cache"], s["bounds"], page_table=s["table"], start=s["lens"], end=end)
        s["lens"].copy_(end)
        return blocks, out

    s, e = states
    for x in states:
        step(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(s)
    for i in range(6):
        for x, seed in ((k, 70), (v, 80), (q, 90)):
            x.copy_(rand_rows(x.shape[0], x.shape[1], dim, "bf16", seed + i, packed=False))
        graph.replay()
        want = step(e)
        torch.cuda.synchronize()
        for a, b in zip((*got, s["lens"]), (*want, e["lens"])):
            assert torch.equal(a, b), i
        np.testing.assert_array_equal(s["bounds"].codes[s["table"][1, :4].long()].cpu().numpy(), e["bounds"].codes[e["table"][1, :4].long()].cpu().numpy())
    # and the choice is that of the oracle, the attention too
    host = (s["table"].cpu().numpy(), s["lens"].cpu().numpy(), offsets.cpu().numpy())
    b = s["bounds"]
    plan = (s["table"], s["lens"], offsets)
    blocks = check_select(q, b, plan, host, take)
    check_sparse(s["cache"], [s["cache"].k, s["cache"].v, None, None], plan, host, n * nodes, 4, blocks.cpu().numpy(), q=q)


def test_idle_calls_and_refusals():
    require_gpu()
    say("idle, refusals")
    cache, tensors, plan, host, n_rows = written("bf16", [100], [3], 16, 2, 64)
    b = D.KVBounds.empty(cache)
    q = rand_rows(n_rows, 4, 64, "bf16", 3)
    kw = dict(page_table=plan[0], start=plan[1], offsets=plan[2], max_nodes=3)
    assert D.dflash_kv_select(q[:0], b, n_take=3, **kw).shape == (0, 2, 3)
    assert D.dflash_sparse_attention(q[:0], cache, gpu(np.zeros((0, 2, 3))), **kw).shape == (0, 4, 64)
    none = dict(page_table=plan[0][:0], start=plan[1][:0])
    D.dflash_kv_bounds(cache, b, end=plan[1][:0], **none)
    with pytest.raises(ValueError, match="blocks"):
        D.dflash_sparse_attention(q, cache, gpu(np.zeros((n_rows, 1, 3))), **kw)
    with pytest.raises(ValueError, match="blocks"):
        D.dflash_sparse_attention(q, cache, gpu(np.zeros((n_rows, 2, 3))).long(), **kw)
    with pytest.raises(ValueError, match="out"):
        D.dflash_kv_select(q, b, n_take=3, out=gpu(np.zeros((n_rows, 2, 4))), **kw)
    with pytest.raises(ValueError, match="n_take"):
        D.dflash_kv_select(q, b, **kw)
    with pytest.raises(ValueError, match="end"):
        D.dflash_kv_bounds(cache, b, page_table=plan[0], start=plan[1], end=gpu([1, 2]))
    with pytest.raises(D.DFlashError, match="n_first"):
        D.dflash_kv_select(q, b, n_take=3, n_first=2, n_last=2, **kw)
    with pytest.raises(D.DFlashError, match="bounds"):
        D.dflash_kv_bounds(cache, D.KVBounds(b.codes[:3].contiguous(), b.scale[:3].contiguous(), page_size=16),
                           page_table=plan[0], start=plan[1], end=plan[1])
    with pytest.raises(D.DFlashError, match="workspace"):
        D.dflash_sparse_attention(q, cache, gpu(np.zeros((n_rows, 2, 3))), workspace=torch.empty(16, dtype=torch.uint8, device=DEV), **kw)
