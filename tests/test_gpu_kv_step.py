"""The operators in the order a serving loop uses them, beside the draft path:
a prompt goes into the cache, trees of drafted nodes are written and attended
to, a path is accepted and committed, and the next step starts behind it."""
import numpy as np
import pytest
import torch

import block_draft_proposal_amd as D
from gpu_helpers import DEV, require_gpu, say
from kv_helpers import TYPES, attention_bound, codes_f64, mask_tensor, oracle_cache, rand_rows, tree_mask
from oracle import kv_oracle as O

pytestmark = pytest.mark.gpu


def test_chain_of_the_verified_block_then_the_next_step():
    """dflash_verify's accepted counts drive a chain: the kept tokens' rows are
    in place already, so only start advances."""
    require_gpu()
    say("verify with a chain")
    R, S, V, heads, dim, page = 3, 5, 97, 2, 64, 16
    gen = torch.Generator(device=DEV).manual_seed(1)
    logits = torch.randn((R, S + 1, V + 7), generator=gen, device=DEV)[..., :V]
    cand = torch.stack([torch.randperm(V, device=DEV)[:4] for _ in range(R * S)]).view(R, S, 4)
    q = torch.full((R, S, 4), 0.25, device=DEV)
    accepted, committed = D.dflash_verify(logits, cand, q, cand[..., 0].contiguous(), torch.rand((R, S), generator=gen, device=DEV),
                                          torch.rand(R, generator=gen, device=DEV), torch.ones(R, device=DEV),
                                          torch.zeros(R, dtype=torch.uint8, device=DEV))
    cache = D.KVCache.empty(12, heads, page, dim)
    table = torch.randperm(12, device=DEV, dtype=torch.int32).view(R, 4)
    start = torch.tensor([7, 0, 20], dtype=torch.int32, device=DEV)
    full = torch.arange(R + 1, dtype=torch.int32, device=DEV) * 30
    kw = dict(page_table=table)
    D.dflash_kv_write(cache, rand_rows(90, heads, dim, "bf16", 1), rand_rows(90, heads, dim, "bf16", 2),
                      start=torch.zeros_like(start), offsets=full, **kw)
    block = torch.arange(R + 1, dtype=torch.int32, device=DEV) * (S + 1)
    start = start + accepted + 1                        # the accepted tokens and the one committed after them
    rows = R * (S + 1)
    D.dflash_kv_write(cache, rand_rows(rows, heads, dim, "bf16", 3), rand_rows(rows, heads, dim, "bf16", 4), start=start, offsets=block, **kw)
    x = rand_rows(rows, 4, dim, "bf16", 5)
    out = D.dflash_tree_attention(x, cache, start=start, offsets=block, max_nodes=S + 1, **kw)
    torch.cuda.synchronize()
    want = np.zeros(out.shape)
    spread, reach = O.tree_attention(codes_f64(x), oracle_cache(cache.k, cache.v), table.cpu().numpy(), start.cpu().numpy(),
                                     block.cpu().numpy(), None, dim ** -0.5, want)
    assert (np.abs(codes_f64(out) - want) <= attention_bound(want, spread, reach, dim)).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_prompt_trees_and_commits(kind):
    require_gpu()
    say(f"three steps {kind}")
    R, heads, group, dim, page, nodes = 3, 2, 4, 128, 16, 12
    tensors = [torch.zeros((40, heads, page, dim), dtype=torch.uint8 if kind == "e4m3" else TYPES[kind], device=DEV).view(TYPES[kind]) for _ in "kv"]
    tensors += [None, None] if kind == "bf16" else [torch.zeros((40, heads, page), dtype=torch.uint8, device=DEV) for _ in "kv"]
    cache, model = D.KVCache(*tensors), oracle_cache(*tensors)
    table = torch.randperm(40, device=DEV, dtype=torch.int32)[:36].view(R, 12).contiguous()
    host_table = table.cpu().numpy()
    start = np.zeros(R, dtype=np.int32)
    lens = np.array([50, 1, 100], dtype=np.int32)       # the prompts
    gpu = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731

    def write(first, counts, seed):
        offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        k, v = (rand_rows(int(offsets[-1]), heads, dim, "bf16", seed + i) for i in range(2))
        D.dflash_kv_write(cache, k, v, page_table=table, start=gpu(first), offsets=gpu(offsets))
        O.write(model, kind, codes_f64(k), codes_f64(v), host_table, first, offsets)
        return offsets

    write(start, lens, 10)
    start = lens.copy()
    for step in range(3):
        offsets = write(start, np.full(R, nodes), 30 + 10 * step)
        bits = tree_mask(int(offsets[-1]), offsets, 1, seed=step)
        x = rand_rows(int(offsets[-1]), heads * group, dim, "bf16", 70 + step)
        out = D.dflash_tree_attention(x, cache, page_table=table, start=gpu(start), offsets=gpu(offsets), max_nodes=nodes,
                                      mask=mask_tensor(bits))
        torch.cuda.synchronize()
        want = np.zeros(out.shape)
        spread, reach = O.tree_attention(codes_f64(x), model, host_table, start, offsets, bits, dim ** -0.5, want)
        assert (np.abs(codes_f64(out) - want) <= attention_bound(want, spread, reach, dim)).all(), step
        # accept the path of a node: the bits of its row, in ascending order
        paths, kept = np.zeros((R, nodes), dtype=np.int32), np.zeros(R, dtype=np.int32)
        for r in range(R):
            row = int(bits[offsets[r] + (5 + 3 * r + step) % nodes, 0])
            path = [j for j in range(nodes) if row >> j & 1]
            paths[r, :len(path)], kept[r] = path, len(path)
        D.dflash_kv_commit(cache, page_table=table, start=gpu(start), paths=gpu(paths), path_lens=gpu(kept))
        O.commit(model, host_table, start, paths, kept)
        start = start + kept
    ends = np.concatenate([[0], np.cumsum(start)]).astype(np.int32)
    got = D.dflash_kv_read(cache, page_table=table, start=gpu(np.zeros(R, dtype=np.int32)), offsets=gpu(ends),
                           n_rows=int(ends[-1]), dtype=torch.float32)
    ref = [np.zeros((int(ends[-1]), heads, dim)) for _ in "kv"]
    O.read(model, host_table, np.zeros(R, dtype=np.int32), ends, ref)
    for a, b in zip(got, ref):
        np.testing.assert_array_equal(a.double().cpu().numpy(), b)
