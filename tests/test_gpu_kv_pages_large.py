"""GPU tests of pools whose chunks' sums take several rounds of a workgroup: more
than 2^20 pages, against numpy forms of the definitions."""
import numpy as np
import pytest
import torch

import block_draft_proposal_amd as D
from gpu_helpers import require_gpu, say
from test_gpu_kv_pages import gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n_pages", [(1 << 20) + 1, (1 << 21) + 1025, 5_000_003])
@pytest.mark.parametrize("share", [0.0005, 0.3, 1.0])
def test_resize_of_a_pool_of_more_chunks_than_threads(n_pages, share):
    """Free pages few and far apart, many and all of them; requests that grow and
    shrink at once, and a call that is a page short."""
    require_gpu()
    say(f"large pool {n_pages} {share}")
    rng = np.random.default_rng(n_pages)
    n, page = 300, 4
    refs = np.where(rng.random(n_pages) < share, 0, -1).astype(np.int32)
    refs[[0, -1]] = 0
    width = int(max(4, (refs == 0).sum() // 150))
    want = rng.integers(0, page * max(2, (refs == 0).sum() // 400), n)
    want[:2] = 0
    pool, table, lens = D.KVPool(gpu(refs), page), gpu(np.full((n, width), -1)), gpu(np.zeros(n))
    rows, held = np.full((n, width), -1), np.zeros(n, dtype=np.int64)

    def step(want):
        copies, counts = D.dflash_kv_resize(pool, page_table=table, lens=lens, want=gpu(want))
        need = -(-want // page)
        for r in np.nonzero(need < held)[0]:
            refs[rows[r, need[r]:held[r]]] -= 1
            rows[r, need[r]:held[r]] = -1
        free, more = np.nonzero(refs == 0)[0], np.maximum(need - held, 0)
        short = max(0, int(more.sum()) - len(free))
        now = np.minimum(need, held) if short else need
        at = 0
        for r in np.nonzero(more)[0] if not short else ():
            rows[r, held[r]:need[r]] = free[at:at + more[r]]
            at += more[r]
        refs[free[:at]] = 1
        held[:] = now
        assert counts.tolist() == [0, short]
        np.testing.assert_array_equal(table.cpu().numpy(), rows)
        np.testing.assert_array_equal(pool.refs.cpu().numpy(), refs)
        return short

    assert step(want) == 0
    assert step(np.where(rng.random(n) < 0.5, 0, want)) == 0
    assert step(want[::-1].copy()) == 0
    left = int((refs == 0).sum())
    most = np.zeros(n, dtype=np.int64)
    if left < width:                                     # the last pages of the pool, and one too many
        most[0] = page * left
        assert step(np.maximum(want[::-1], most)) == 0
        most[1] = page
        assert step(np.maximum(want[::-1], most)) == 1
    else:
        assert step(want[::-1] + page * (left // n + 1)) == n * (left // n + 1) - left


@pytest.mark.parametrize("n_pages,most", [((1 << 20) + 1, None), ((1 << 21) + 1025, 1_000_000), (3_000_001, 2049)])
def test_compact_of_a_pool_of_more_chunks_than_threads(n_pages, most):
    require_gpu()
    say(f"large compact {n_pages}")
    rng = np.random.default_rng(n_pages)
    refs = rng.choice(np.array([0, 0, 1, 3, -1], dtype=np.int32), n_pages)
    n, page = 40, 2
    held = np.nonzero(refs > 0)[0]
    entries = rng.choice(held, (n, 5000))
    lens = rng.integers(0, 2 * 5000 + 1, n)
    pool, table = D.KVPool(gpu(refs), page), gpu(entries)
    most = n_pages // 2 if most is None else most
    copies = torch.full((most, 2), -7, dtype=torch.int32, device="cuda")
    copies, counts, page_map = D.dflash_kv_compact(pool, page_table=table, lens=gpu(lens), copies=copies)
    free, down = np.nonzero(refs == 0)[0], held[::-1]
    m = min(len(free), len(held), most)
    m = int((down[:m] > free[:m]).sum())                 # sources fall and targets rise
    moved = np.arange(n_pages)
    moved[refs == 0] = -1
    moved[down[:m]] = free[:m]
    want = refs.copy()
    want[free[:m]], want[down[:m]] = refs[down[:m]], 0
    assert counts.tolist() == [m, len(held)]
    np.testing.assert_array_equal(copies.cpu().numpy()[:m], np.stack([down[:m], free[:m]], 1))
    assert (copies[m:] == -7).all()
    np.testing.assert_array_equal(page_map.cpu().numpy(), moved)
    np.testing.assert_array_equal(pool.refs.cpu().numpy(), want)
    inside = np.arange(5000) < -(-lens // page)[:, None]
    np.testing.assert_array_equal(table.cpu().numpy(), np.where(inside, moved[entries], entries))
