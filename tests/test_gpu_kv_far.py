"""GPU tests at the far ends of the ranges: positions and lengths near 2^31, the
longest table of the choice, and caches whose pages hold K, V and scales in one
pool."""
import numpy as np
import pytest
import torch

import block_draft_proposal_amd as D
from gpu_helpers import DEV, require_gpu, say
from kv_helpers import TYPES, oracle_cache, rand_rows
from oracle import sparse_oracle as S
from test_gpu_kv_pages import Books, gpu
from test_gpu_kv_sparse import rand_bounds

pytestmark = pytest.mark.gpu
MOST = 0x7fffffff - (1 << 17)                            # start plus nodes


def rand_cache(kind, n_pages, heads, page, dim, seed):
    """(cache, its tensors), every row written."""
    cache = D.KVCache.empty(n_pages, heads, page, dim, TYPES[kind])
    k, v = (rand_rows(n_pages * page, heads, dim, "bf16", seed + i) for i in range(2))
    D.dflash_kv_write(cache, k, v, page_table=gpu([range(n_pages)]), start=gpu([0]), offsets=gpu([0, n_pages * page]))
    return cache, [cache.k, cache.v, cache.k_scale, cache.v_scale]


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("page,total,nodes", [(65536, MOST, 3), (65536, 1 << 30, 3), (4096, (1 << 30) + 5, 1), (128, MOST, 1), (128, MOST, 5)])
def test_positions_up_to_the_largest(kind, page, total, nodes):
    """A request of `total` positions on a few pages that its table repeats: the
    same blocks, tail and nodes as near the start give the same bits."""
    require_gpu()
    say(f"far positions {kind} {page} {total} {nodes}")
    heads, dim, group = 2, 64, 3
    cache, _ = rand_cache(kind, 6, heads, page, dim, 3)
    start = total - nodes
    full, tail = start // page, start % page
    width = -(-total // page)
    table = torch.zeros((2, width), dtype=torch.int32, device=DEV)
    table[0] = torch.randint(0, 6, (width,), dtype=torch.int32, device=DEV, generator=torch.Generator(device=DEV).manual_seed(5))
    ids = [0, full // 2, full - 1]                        # blocks of the far request; 0, 1, 2 of the near one
    table[1, :3] = table[0, ids]
    rest = width - full                                  # pages of the tail and the nodes
    table[1, 3:3 + rest] = table[0, full:]
    q = rand_rows(nodes, heads * group, dim, "bf16", 4)
    take = 3 if nodes == 1 else 4
    far, near = np.full((nodes, heads, take), -1), np.full((nodes, heads, take), -1)
    for i in range(nodes):
        for h in range(heads):
            some = [x for x in range(3) if (i + h + x) % 3 or x == 2]
            far[i, h, :len(some)], near[i, h, :len(some)] = [ids[x] for x in some], some
    kw = dict(offsets=gpu([0, nodes]), max_nodes=nodes)
    got = D.dflash_sparse_attention(q, cache, gpu(far), page_table=table[:1], start=gpu([start]), **kw)
    want = D.dflash_sparse_attention(q, cache, gpu(near), page_table=table[1:], start=gpu([3 * page + tail]), **kw)
    assert torch.isfinite(got.float()).all() and torch.equal(got, want)
    # a node more is too far
    if total == MOST:
        over = D.dflash_sparse_attention(q, cache, gpu(far), page_table=table[:1], start=gpu([start + 1]), **kw)
        assert torch.isnan(over.float()).all()


@pytest.mark.parametrize("kind", ["bf16", "i8"])
def test_bounds_of_far_pages(kind):
    """The last pages of lengths near 2^31."""
    require_gpu()
    say(f"far bounds {kind}")
    page, heads, dim = 128, 2, 64
    cache, tensors = rand_cache(kind, 4, heads, page, dim, 3)
    width = (1 << 31) // page - 1
    table = torch.full((1, width), 3, dtype=torch.int32, device=DEV)
    table[0, -3:] = gpu([2, 0, 1])
    b = D.KVBounds.empty(cache)
    b.codes.fill_(33)
    b.scale.fill_(44)
    want = np.full(tuple(b.codes.shape), 33, dtype=np.int64), np.full(tuple(b.scale.shape), 44, dtype=np.int64)
    start, end = (width - 3) * page + 1, 0x7fffffff
    D.dflash_kv_bounds(cache, b, page_table=table, start=gpu([start]), end=gpu([end]))
    torch.cuda.synchronize()
    S.bounds(oracle_cache(*tensors), *want, table.cpu().numpy(), [start], [end])
    np.testing.assert_array_equal(b.scale.cpu().numpy(), want[1])
    np.testing.assert_array_equal(b.codes.cpu().numpy(), want[0])
    assert (want[1][3] == 44).all() and (want[1][:3] != 44).all()


@pytest.mark.parametrize("take", [1000, 65536])
def test_the_longest_table_of_the_choice(take):
    """2^24 blocks of few distinct scores: the first ones of the best pages."""
    require_gpu()
    say(f"2^24 blocks {take}")
    width, heads = 1 << 24, 2
    b = rand_bounds(7, heads, 64, 128, 5)
    rng = np.random.default_rng(1)
    pages = rng.choice(7, width, p=[0.0001, 0.0009, 0.009, 0.09, 0.3, 0.3, 0.3]).astype(np.int32)
    q = rand_rows(1, heads, 64, "bf16", 6)
    got = D.dflash_kv_select(q, b, page_table=gpu([pages]), start=gpu([0x7fffffff]), offsets=gpu([0, 1]), max_nodes=1, n_take=take,
                             n_first=1, n_last=2).cpu().numpy()
    blocks = min(width, 0x7fffffff // 128)
    x = q.float().cpu().double().numpy()
    forced = {0, blocks - 2, blocks - 1}
    for h in range(heads):
        score = []
        for p in range(7):
            c = S.query_codes(x[0, h:h + 1])[0]
            edge = np.where(c > 0, b.codes[p, h, 1].cpu().numpy().astype(np.int64), b.codes[p, h, 0].cpu().numpy().astype(np.int64))
            score.append(np.ldexp(float((c * edge).sum()), int(b.scale[p, h]) - 127))
        left, chosen = take - len(forced), set(forced)
        for s in sorted(set(score), reverse=True):
            at = np.nonzero(np.isin(pages[:blocks], [p for p in range(7) if score[p] == s]))[0]
            at = [int(a) for a in at[:left + 3] if int(a) not in forced][:left]
            chosen.update(at)
            left -= len(at)
            if not left:
                break
        assert got[0, h].tolist() == sorted(chosen), h


def test_lengths_up_to_the_largest():
    """2^31 - 1 positions on pages of 65536, shared and copied."""
    require_gpu()
    say("largest lengths")
    n_pages, width, page = 40000, 33000, 65536
    b = Books(np.zeros(n_pages, dtype=np.int32), np.full((3, width), -1), [0, 0, 0], page)
    most = 0x7fffffff
    assert b.resize([most - 5, 7, 0]) == 0
    b.fork([0, 1, 0])
    b.resize([most, 65537, most - 5])                    # the first copies its last page
    b.resize([0, 65537, most])
    b.compact(100)
    b.fork([2, 2, 2])
    b.resize([most, 1, 65536])


def pooled(kind, n_pages, heads, page, dim, gap):
    """A cache whose pages hold K, V and both scales in one allocation."""
    size = 2 if kind == "bf16" else 1
    codes, scales = heads * page * dim * size, 0 if kind == "bf16" else heads * page
    whole = -(-(2 * codes + 2 * scales) // 16) * 16 + gap
    pool = torch.randint(0, 256, (n_pages * whole,), device=DEV, generator=torch.Generator(device=DEV).manual_seed(8)).to(torch.uint8)
    k, v = (pool.view(TYPES[kind]).as_strided((n_pages, heads, page, dim), (whole // size, page * dim, dim, 1), i * codes // size) for i in range(2))
    if kind == "bf16":
        return D.KVCache(k, v), pool
    return D.KVCache(k, v, *(pool.as_strided((n_pages, heads, page), (whole, page, 1), 2 * codes + i * scales) for i in range(2))), pool


@pytest.mark.parametrize("gap", [0, 48])
@pytest.mark.parametrize("kind,dim,page", [("bf16", 128, 16), ("e4m3", 64, 20), ("i8", 128, 16), ("e4m3", 256, 7)])
def test_one_pool_of_all(kind, dim, page, gap):
    """Bounds, attention and copies on such a cache are those on one of separate
    tensors; nothing between its pages changes."""
    require_gpu()
    say(f"one pool {kind} {dim} {gap}")
    n_pages, heads, group = 30, 3, 2
    a, pool = pooled(kind, n_pages, heads, page, dim, gap)
    k, v = (rand_rows(n_pages * page, heads, dim, "bf16", 3 + i) for i in range(2))
    every = dict(page_table=gpu([range(n_pages)]), start=gpu([0]), offsets=gpu([0, n_pages * page]))
    D.dflash_kv_write(a, k, v, **every)
    b = D.KVCache(*(None if t is None else t.contiguous() for t in (a.k, a.v, a.k_scale, a.v_scale)))
    table = gpu([np.random.default_rng(1).permutation(n_pages)])
    bounds = [D.KVBounds.empty(x) for x in (a, b)]
    for x, y in zip((a, b), bounds):
        D.dflash_kv_bounds(x, y, page_table=table, start=gpu([0]), end=gpu([n_pages * page]))
    assert torch.equal(bounds[0].codes, bounds[1].codes) and torch.equal(bounds[0].scale, bounds[1].scale)
    for nodes in (1, 4):
        q = rand_rows(nodes, heads * group, dim, "bf16", 9)
        kw = dict(page_table=table, start=gpu([(n_pages - 2) * page + 3]), offsets=gpu([0, nodes]), max_nodes=nodes)
        blocks = D.dflash_kv_select(q, bounds[0], n_take=6, **kw)
        x, y = (D.dflash_sparse_attention(q, c, blocks, **kw) for c in (a, b))
        assert torch.isfinite(x.float()).all() and torch.equal(x, y)
    pairs = gpu([(3, 29), (0, 1), (28, 2)])
    used = torch.zeros(pool.numel(), dtype=torch.bool, device=DEV)
    size = 2 if kind == "bf16" else 1
    for t in (a.k, a.v, a.k_scale, a.v_scale):
        if t is not None:
            s = size if t.dim() == 4 else 1
            used.as_strided((n_pages, t[0].numel() * s), (t.stride(0) * s, 1), t.storage_offset() * s).fill_(True)
    between = pool[~used].clone()
    for c, y in zip((a, b), bounds):
        D.dflash_kv_copy_pages(c, pairs, bounds=y)
    for s, t in zip((a.k, a.v, a.k_scale, a.v_scale), (b.k, b.v, b.k_scale, b.v_scale)):
        assert s is None or torch.equal(s.contiguous().view(torch.uint8), t.view(torch.uint8))
    assert torch.equal(pool[~used], between)
    assert torch.equal(bounds[0].codes, bounds[1].codes) and torch.equal(bounds[0].codes[29], bounds[0].codes[3])
