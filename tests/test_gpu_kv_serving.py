"""The operators on pages and over chosen pages together, as a server uses them:
prompts, their samples, drafted nodes, accepted paths and a packed pool."""
import numpy as np
import pytest
import torch

import block_draft_proposal_amd as D
from gpu_helpers import DEV, require_gpu, say
from kv_helpers import attention_bound, codes_f64, dead_cache, mask_tensor, oracle_cache, rand_rows, tree_mask
from oracle import pages_oracle as P
from oracle import sparse_oracle as S

pytestmark = pytest.mark.gpu


def gpu(x):
    return torch.from_numpy(np.ascontiguousarray(np.array(x, dtype=np.int32))).to(DEV)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_prompts_samples_trees_and_a_packed_pool(kind):
    require_gpu()
    say(f"serving {kind}")
    page, heads, group, dim, n, width, n_pages, nodes, take = 16, 2, 4, 64, 8, 20, 150, 6, 4
    tensors = dead_cache(kind, n_pages, heads, page, dim)
    cache = D.KVCache(*tensors)
    bounds = D.KVBounds.empty(cache)
    bounds.codes.zero_()
    bounds.scale.fill_(255)
    table = torch.full((n, width + 5), -1, dtype=torch.int32, device=DEV)[:, 2:width + 2]      # rows apart
    refs, lens = gpu(np.zeros(n_pages)), gpu(np.zeros(n))
    pool = D.KVPool(refs, page)
    books = dict(page_table=table, lens=lens)
    prompts = [137, 0, 0, 0, 250, 0, 0, 0]

    def grow(want):
        before = lens.clone()
        copies, counts = D.dflash_kv_resize(pool, want=gpu(want), **books)
        D.dflash_kv_copy_pages(cache, copies, counts, bounds=bounds)
        assert int(counts[1]) == 0
        return before

    before = grow(prompts)
    ends = gpu(np.concatenate([[0], np.cumsum(prompts)]))
    k, v = rand_rows(sum(prompts), heads, dim, "bf16", 1), rand_rows(sum(prompts), heads, dim, "bf16", 2)
    D.dflash_kv_write(cache, k, v, page_table=table, start=before, offsets=ends)
    D.dflash_kv_bounds(cache, bounds, page_table=table, start=before, end=lens)
    D.dflash_kv_fork(pool, parents=gpu([0, 0, 0, 0, 4, 4, -1, 4]), **books)
    offsets = gpu([0, 6, 12, 18, 24, 30, 36, 36, 42])
    for step in range(4):
        start = lens.clone()
        live = np.diff(offsets.cpu().numpy())        # the nodes of each, none where a sample has ended
        grow(start.cpu().numpy() + live)                 # parts shared pages, takes room for the nodes
        rows = int(offsets[-1])
        batch = dict(page_table=table, start=start, offsets=offsets)
        D.dflash_kv_write(cache, rand_rows(rows, heads, dim, "bf16", 10 + step), rand_rows(rows, heads, dim, "bf16", 20 + step), **batch)
        q, mask = rand_rows(rows, heads * group, dim, "bf16", 30 + step), tree_mask(rows, offsets.cpu().numpy(), 1, seed=step)
        host = (table.cpu().numpy(), start.cpu().numpy(), offsets.cpu().numpy())
        blocks = D.dflash_kv_select(q, bounds, max_nodes=nodes, n_take=take, **batch)
        want = np.full(tuple(blocks.shape), -9, dtype=np.int64)
        S.select(codes_f64(q), bounds.codes.cpu().numpy(), bounds.scale.cpu().numpy(), n_pages, page, *host, take, 1, 1, want)
        np.testing.assert_array_equal(blocks.cpu().numpy(), want)
        out = D.dflash_sparse_attention(q, cache, blocks, max_nodes=nodes, mask=mask_tensor(mask), **batch)
        ref = np.zeros(tuple(out.shape))
        spread, reach = S.sparse_attention(codes_f64(q), oracle_cache(*tensors), *host, want, mask, dim ** -0.5, ref)
        assert (np.abs(codes_f64(out) - ref) <= attention_bound(ref, spread, reach, dim)).all(), step
        # the path of a node is accepted, its rows move up, the rest is let go
        paths, kept = np.zeros((n, nodes), dtype=np.int32), np.zeros(n, dtype=np.int32)
        for r in range(n):
            if live[r]:
                bits = int(mask[int(offsets[r]) + (r + step) % nodes, 0])
                path = [j for j in range(nodes) if bits >> j & 1]
                paths[r, :len(path)], kept[r] = path, len(path)
        D.dflash_kv_commit(cache, page_table=table, start=start, paths=gpu(paths), path_lens=gpu(kept))
        grow(start.cpu().numpy() + kept)
        D.dflash_kv_bounds(cache, bounds, page_table=table, start=start, end=lens)
        if step == 1:                                    # samples end, and others are forked from those that are left
            D.dflash_kv_fork(pool, parents=gpu([0, 1, 1, -1, 5, 5, -1, 7]), **books)
            offsets = gpu([0, 6, 12, 18, 18, 24, 30, 30, 36])
        # a packed pool answers as before
        q = rand_rows(int(offsets[-1]), heads * group, dim, "bf16", 50 + step)
        ask = dict(page_table=table, start=lens, offsets=offsets)
        chosen = D.dflash_kv_select(q, bounds, max_nodes=nodes, n_take=take, **ask)
        copies, counts, _ = D.dflash_kv_compact(pool, **books)
        D.dflash_kv_copy_pages(cache, copies, counts, bounds=bounds)
        held = int(counts[1])
        assert (refs[:held] > 0).all() and not refs[held:].any()
        assert torch.equal(chosen, D.dflash_kv_select(q, bounds, max_nodes=nodes, n_take=take, **ask))
    t, l = table.cpu().numpy(), lens.cpu().numpy()
    count = np.zeros(n_pages, dtype=np.int32)        # the counts are those of the tables
    for r in range(n):
        for j in range(P.entries(int(l[r]), page, width)):
            count[t[r, j]] += 1
    np.testing.assert_array_equal(refs.cpu().numpy(), count)


def test_pages_beyond_four_gigabytes():
    """Rows whose offsets pass 32 bits, in bytes and in elements: copies, bounds
    and attention equal those on a small pool."""
    require_gpu()
    say("far pages")
    page, heads, dim, n_pages = 16, 8, 128, 300_000           # 9.8 GB of K, as much of V
    big = D.KVCache.empty(n_pages, heads, page, dim, torch.bfloat16)
    small = D.KVCache.empty(12, heads, page, dim, torch.bfloat16)
    far = torch.tensor([299_999, 270_001, 140_000, 3, 131_072, 262_143, 299_998, 65_536, 200_000, 1], dtype=torch.int32, device=DEV)
    near = torch.arange(10, dtype=torch.int32, device=DEV)
    start, offsets = gpu([150]), gpu([0, 4])
    k, v, q = (rand_rows(154, h, dim, "bf16", i) for i, h in ((1, heads), (2, heads), (3, 32)))
    outs = []
    for cache, table in ((big, far[None]), (small, near[None])):
        D.dflash_kv_write(cache, k, v, page_table=table, start=gpu([0]), offsets=gpu([0, 154]))
        moved = table.clone()
        to = 299_997 if cache is big else 11
        D.dflash_kv_copy_pages(cache, torch.stack([table[0, 4], torch.full_like(table[0, 4], to)])[None].contiguous())
        moved[0, 4] = to
        b = D.KVBounds.empty(cache)
        D.dflash_kv_bounds(cache, b, page_table=moved, start=gpu([0]), end=start)
        batch = dict(page_table=moved, start=start, offsets=offsets, max_nodes=4)
        blocks = D.dflash_kv_select(q[:4], b, n_take=5, **batch)
        out = D.dflash_sparse_attention(q[:4], cache, blocks, **batch)
        one = D.dflash_sparse_attention(q[:1], cache, blocks[:1], **dict(batch, offsets=gpu([0, 1]), max_nodes=1))
        outs.append((b.codes[moved[0, :9].long()], b.scale[moved[0, :9].long()], blocks, out, one))
    torch.cuda.synchronize()
    for x, y in zip(*outs):
        assert torch.equal(x, y)


@pytest.mark.parametrize("nodes", [1, 5])
def test_two_streams_with_workspaces_of_their_own(nodes):
    """The same calls on two streams at once give what they give alone."""
    require_gpu()
    say(f"two streams {nodes}")
    page, heads, dim, n = 16, 2, 128, 12
    cache = D.KVCache.empty(400, heads, page, dim, torch.bfloat16)
    table = torch.randperm(400, generator=torch.Generator().manual_seed(1))[:n * 32].view(n, 32).int().to(DEV)
    ends = np.concatenate([[0], np.cumsum([500] * n)])
    k = rand_rows(500 * n, heads, dim, "bf16", 1)
    D.dflash_kv_write(cache, k, k, page_table=table, start=gpu(np.zeros(n)), offsets=gpu(ends))
    b = D.KVBounds.empty(cache)
    D.dflash_kv_bounds(cache, b, page_table=table, start=gpu(np.zeros(n)), end=gpu([480] * n))
    batch = dict(page_table=table, start=gpu([480] * n), offsets=gpu(np.arange(n + 1) * nodes), max_nodes=nodes)
    qs = [rand_rows(n * nodes, heads * 4, dim, "bf16", 5 + i) for i in range(2)]

    def ask(q, stream=None):
        blocks = D.dflash_kv_select(q, b, n_take=9, stream=stream, **batch)
        return blocks, D.dflash_sparse_attention(q, cache, blocks, stream=stream, **batch)

    want = [ask(q) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [ask(q, s) for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


@pytest.mark.parametrize("n,nodes,heads", [(20, 16, 8), (2, 5, 2), (40, 1, 8)])
def test_a_captured_choice_and_attention(n, nodes, heads):
    """Enough tiles for one launch of the choice, few tiles that are split, and
    single rows: replays over new queries, with eager calls and waits between."""
    require_gpu()
    say(f"captured {n} {nodes}")
    page, dim, length = 16, 128, 1000
    width = -(-(length + nodes) // page)
    cache = D.KVCache.empty(n * width, heads, page, dim, torch.bfloat16)
    table = torch.randperm(n * width, generator=torch.Generator().manual_seed(2)).view(n, width).int().to(DEV)
    k = rand_rows((length + nodes) * n, heads, dim, "bf16", 1)
    D.dflash_kv_write(cache, k, k, page_table=table, start=gpu(np.zeros(n)), offsets=gpu(np.arange(n + 1) * (length + nodes)))
    b, start = D.KVBounds.empty(cache), gpu(length - 7 * np.arange(n))
    D.dflash_kv_bounds(cache, b, page_table=table, start=gpu(np.zeros(n)), end=start)
    batch = dict(page_table=table, start=start, offsets=gpu(np.arange(n + 1) * nodes), max_nodes=nodes)
    q = rand_rows(n * nodes, heads * 4, dim, "bf16", 5)

    def ask():
        blocks = D.dflash_kv_select(q, b, n_take=12, **batch)
        return blocks, D.dflash_sparse_attention(q, cache, blocks, **batch)

    ask()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ask()
    for seed in range(4):
        q.copy_(rand_rows(n * nodes, heads * 4, dim, "bf16", 10 + seed))
        want = ask()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), seed
