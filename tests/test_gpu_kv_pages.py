"""GPU tests of the page tables against the plain oracle: random lives of
requests that grow, shrink, fork and end, a pool that is packed, and the ends of
the ranges."""
import numpy as np
import pytest
import torch

import block_draft_proposal_amd as D
from gpu_helpers import DEV, require_gpu, say
from kv_helpers import dead_cache
from oracle import pages_oracle as P

pytestmark = pytest.mark.gpu


def gpu(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(np.array(x, dtype=dtype))).to(DEV)


class Books:
    """The oracle's lists and the same on the GPU (rows of the table apart)."""

    def __init__(self, refs, table, lens, page):
        self.refs, self.table, self.lens, self.page = list(refs), [list(r) for r in table], list(lens), page
        self.n, self.width = len(lens), len(table[0])
        wide = torch.full((self.n, self.width + 3), 12345, dtype=torch.int32, device=DEV)
        self.g_table = wide[:, :self.width]
        self.g_table.copy_(gpu(table))
        self.wide = wide
        self.g_refs, self.g_lens = gpu(refs), gpu(lens)
        self.pool = D.KVPool(self.g_refs, page)

    def kw(self):
        return dict(page_table=self.g_table, lens=self.g_lens)

    def check(self, what):
        torch.cuda.synchronize()
        np.testing.assert_array_equal(self.g_lens.cpu().numpy(), self.lens, err_msg=what)
        np.testing.assert_array_equal(self.g_table.cpu().numpy(), self.table, err_msg=what)
        np.testing.assert_array_equal(self.g_refs.cpu().numpy(), self.refs, err_msg=what)
        assert (self.wide[:, self.width:] == 12345).all()

    def resize(self, want, **kw):
        pairs, missing = P.resize(self.refs, self.table, self.lens, want, self.page)
        copies = torch.full((self.n, 2), -7, dtype=torch.int32, device=DEV)
        copies, counts = D.dflash_kv_resize(self.pool, want=gpu(want), copies=copies, **self.kw(), **kw)
        self.check(f"resize {want}")
        assert counts.tolist() == [len(pairs), missing]
        assert copies.tolist() == [list(p) for p in pairs] + [[-7, -7]] * (self.n - len(pairs))
        return missing

    def fork(self, parents):
        P.fork(self.refs, self.table, self.lens, parents, self.page)
        D.dflash_kv_fork(self.pool, parents=gpu(parents), **self.kw())
        self.check(f"fork {parents}")

    def compact(self, most):
        pairs, held, page_map = P.compact(self.refs, self.table, self.lens, self.page, most)
        copies = torch.full((most, 2), -7, dtype=torch.int32, device=DEV)
        copies, counts, got = D.dflash_kv_compact(self.pool, copies=copies, **self.kw())
        self.check(f"compact {most}")
        assert counts.tolist() == [len(pairs), held]
        assert got.tolist() == page_map
        assert copies.tolist() == [list(p) for p in pairs] + [[-7, -7]] * (most - len(pairs))


def empty(n_pages, n, width, page, reserved=()):
    refs = np.zeros(n_pages, dtype=np.int32)
    refs[list(reserved)] = -1
    return Books(refs, np.full((n, width), -1), [0] * n, page)


@pytest.mark.parametrize("seed,n_pages,n,width,page", [(0, 40, 6, 9, 4), (1, 300, 33, 20, 16), (2, 5000, 7, 900, 1), (3, 64, 1, 30, 20),
                                                       (4, 9000, 300, 40, 7), (5, 12, 5, 3, 65536),
                                                       (6, 8300, 41, 900, 1), (7, 8192, 1024, 32, 16), (8, 8192, 1025, 3, 5), (9, 100, 3, 20000, 1)])
def test_random_lives(seed, n_pages, n, width, page):
    require_gpu()
    say(f"random lives {seed}")
    rng = np.random.default_rng(seed)
    b = empty(n_pages, n, width, page, reserved=rng.integers(0, n_pages, 3))
    most = min(width * page, 2 ** 31 - 1)
    short = 0
    for step in range(14):
        what = rng.integers(0, 4)
        if what <= 1:
            want = [int(x) if rng.random() < 0.7 else y for x, y in zip(rng.integers(0, most + 1, n), b.lens)]
            if rng.random() < 0.5:                       # steps of a few positions
                want = [min(most, max(0, x + int(d))) for x, d in zip(b.lens, rng.integers(-page, page + 3, n))]
            short += b.resize(want) > 0
        elif what == 2:
            b.fork([int(x) if rng.random() < 0.5 else r for r, x in enumerate(rng.integers(-1, n, n))])
        else:
            b.compact(int(rng.integers(0, n_pages // 2 + 1)))
    b.resize([0] * n)
    assert all(c <= 0 for c in b.refs)


def test_copy_on_write():
    """Holders of a partly filled page: one grows (copies), all grow (the first
    keeps it), one of two grows after the other shrank away."""
    require_gpu()
    say("copy on write")
    b = empty(30, 5, 6, 10)
    b.resize([25, 0, 0, 0, 0])
    b.fork([0, 0, 0, -1, 4])
    b.resize([25, 26, 25, 0, 0])                         # one of three copies
    b.resize([27, 26, 28, 0, 0])                         # the two others grow at once
    b.fork([0, 0, 0, 0, 0])
    b.resize([30, 30, 30, 30, 30])                       # fills the page up: four copies, one stays
    b.fork([0, 0, 0, 0, 0])
    b.resize([30, 31, 30, 30, 30])                       # a full page is shared on
    b.resize([25, 0, 25, 0, 5])                          # shrunk into shared pages
    b.resize([26, 0, 30, 0, 6])


def test_pages_let_go_are_given_again_in_the_same_call():
    require_gpu()
    say("let go and given")
    b = empty(10, 3, 10, 4)
    b.resize([40, 0, 0])
    assert b.resize([20, 20, 1]) == 1                    # one page short: the first shrinks, nobody grows
    assert b.resize([0, 20, 20]) == 0


def test_all_or_nothing_and_out_of_range():
    require_gpu()
    say("out of range")
    b = empty(8, 4, 5, 4)
    b.resize([4, 8, 0, 0])
    b.resize([21, -1, 20, -5])                           # beyond the table and below zero: left alone
    assert b.resize([8, 8, 20, 4]) == 2                   # 1 + 2 + 5 of 8 pages are held, two more are wanted
    b.lens[1] = -3
    b.g_lens[1] = -3
    b.resize([8, 4, 0, 0])                               # a broken length is left alone too
    b.fork([1, 1, 0, 4])                                 # a parent of a broken length, one that is no request
    b.fork([0, 0, 2, 3])                                 # and gets a parent


def test_entries_outside_the_pool_hold_nothing():
    require_gpu()
    say("entries outside")
    b = Books([0, 1, 0, 1, 0, 0], [[1, 77, 3, -1], [-2147483648, 2147483647, -1, -1], [-1] * 4], [9, 5, 0], 3)
    b.fork([0, 1, 0])
    b.resize([9, 6, 11])                                 # the second grows into a page that is none: no copy
    b.compact(3)
    b.resize([0, 0, 0])


def test_full_and_empty_pools():
    require_gpu()
    say("full and empty")
    b = empty(7, 2, 7, 2)
    b.compact(3)
    assert b.resize([14, 1]) == 1
    b.resize([14, 0])
    b.compact(3)
    b.resize([4, 0])
    b.compact(3)
    b.resize([14, 0])


def test_negative_counts_stay():
    require_gpu()
    say("reserved pages")
    b = empty(20, 2, 12, 1, reserved=(0, 3, 19))
    b.resize([8, 8])
    b.resize([0, 8])
    b.compact(10)
    assert b.resize([10, 8]) == 1
    assert b.resize([9, 8]) == 0


def test_many_requests_and_a_large_pool():
    """More requests than a round of the sums holds, and more chunks: against
    the sizes alone (the oracle walks lists)."""
    require_gpu()
    say("many requests")
    n, width, page, n_pages = 5000, 40, 16, 300_001
    rng = np.random.default_rng(7)
    refs, table, lens = gpu(np.zeros(n_pages)), gpu(np.full((n, width), -1)), gpu(np.zeros(n))
    pool = D.KVPool(refs, page)
    for step in range(3):
        want = rng.integers(0, width * page + 1, n)
        copies, counts = D.dflash_kv_resize(pool, page_table=table, lens=lens, want=gpu(want))
        assert counts.tolist() == [0, 0] and lens.cpu().numpy().tolist() == want.tolist()
        t, need = table.cpu().numpy(), -(-want // page)
        held = t[np.arange(width) < need[:, None]]
        assert (t[np.arange(width) >= need[:, None]] == -1).all()
        assert len(np.unique(held)) == len(held) and held.min() >= 0 and held.max() < n_pages
        np.testing.assert_array_equal(np.bincount(held, minlength=n_pages), refs.cpu().numpy())
    before = table.clone()
    copies, counts, page_map = D.dflash_kv_compact(pool, page_table=table, lens=lens)
    m, used = counts.tolist()
    assert used == len(held) and (refs[:used] == 1).all() and not refs[used:].any()
    live = before >= 0
    assert torch.equal(table[live], page_map[before[live].long()]) and (table[~live] == -1).all()
    pairs = copies[:m].cpu().numpy()
    assert (pairs[:, 0] > pairs[:, 1]).all() and len(np.unique(pairs)) == 2 * m


@pytest.mark.parametrize("kind,dim,heads,page", [("bf16", 64, 1, 1), ("bf16", 128, 8, 16), ("e4m3", 128, 3, 20), ("i8", 256, 2, 33), ("i8", 64, 5, 7)])
@pytest.mark.parametrize("with_bounds", [False, True])
def test_copies_of_pages(kind, dim, heads, page, with_bounds):
    require_gpu()
    say(f"copy pages {kind} {dim} {heads} {page}")
    n_pages = 24
    tensors = dead_cache(kind, n_pages, heads, page, dim)
    for t in tensors:
        if t is not None:
            t.view(torch.uint8).random_(0, 256)
    cache = D.KVCache(*tensors)
    bounds = None
    if with_bounds:
        bounds = D.KVBounds.empty(cache)
        bounds.codes.random_(-127, 128)
        bounds.scale.random_(0, 256)
    held = [t for t in tensors if t is not None] + ([bounds.codes, bounds.scale] if with_bounds else [])
    want = [t.view(torch.uint8).clone() for t in held]
    # one source twice, pages outside the pool, a page onto itself
    pairs = [(3, 9), (3, 0), (17, 23), (5, 5), (-1, 4), (4, 24), (24, 8), (2147483647, 1), (11, 2), (12, 13)]
    n = 9
    for w in want:
        for a, b in pairs[:n]:
            if 0 <= a < n_pages and 0 <= b < n_pages:
                w[b] = w[a]
    D.dflash_kv_copy_pages(cache, gpu(pairs), gpu([n, 99]), bounds=bounds)
    torch.cuda.synchronize()
    for t, w in zip(held, want):
        assert torch.equal(t.view(torch.uint8), w)
    for w in want:
        w[13] = w[12]
    D.dflash_kv_copy_pages(cache, gpu(pairs), bounds=bounds)       # all of them
    D.dflash_kv_copy_pages(cache, gpu(pairs)[:0], bounds=bounds)
    D.dflash_kv_copy_pages(cache, gpu(pairs), gpu([-4, 0]), bounds=bounds)
    torch.cuda.synchronize()
    for t, w in zip(held, want):
        assert torch.equal(t.view(torch.uint8), w)


def test_contents_follow_the_tables():
    """A prompt, its samples, and a packed pool: every request reads what it
    wrote."""
    require_gpu()
    say("contents follow")
    heads, page, dim, n = 2, 8, 64, 6
    cache = D.KVCache.empty(60, heads, page, dim, torch.bfloat16)
    refs, table, lens = gpu(np.zeros(60)), gpu(np.full((n, 9), -1)), gpu(np.zeros(n))
    pool = D.KVPool(refs, page)
    model = [torch.zeros((0, heads, dim), dtype=torch.bfloat16, device=DEV) for _ in range(n)]

    def grow(counts, seed):
        have = [len(m) for m in model]
        want = [h + c for h, c in zip(have, counts)]
        copies, got = D.dflash_kv_resize(pool, page_table=table, lens=lens, want=gpu(want))
        D.dflash_kv_copy_pages(cache, copies, got)
        offsets = np.concatenate([[0], np.cumsum(counts)])
        k = torch.randn((int(offsets[-1]), heads, dim), generator=torch.Generator(device=DEV).manual_seed(seed), device=DEV).bfloat16()
        D.dflash_kv_write(cache, k, k, page_table=table, start=gpu(have), offsets=gpu(offsets))
        for r in range(n):
            model[r] = torch.cat([model[r], k[offsets[r]:offsets[r + 1]]])

    def check():
        ends = np.concatenate([[0], np.cumsum([len(m) for m in model])])
        k, v = D.dflash_kv_read(cache, page_table=table, start=gpu(np.zeros(n)), offsets=gpu(ends), n_rows=int(ends[-1]))
        assert torch.equal(k, torch.cat(model)) and torch.equal(k, v)

    def fork(parents):
        D.dflash_kv_fork(pool, page_table=table, lens=lens, parents=gpu(parents))
        model[:] = [model[p] if p >= 0 else model[0][:0] for p in parents]

    grow([21, 0, 0, 16, 0, 3], 0)
    check()
    fork([0, 0, 0, 3, 3, 5])
    grow([2, 5, 0, 1, 9, 1], 1)
    check()
    fork([1, 0, 2, 4, -1, 3])
    grow([1, 1, 1, 1, 7, 1], 2)
    check()
    fork([-1, 1, 2, -1, 4, 5])
    for most in (2, 30):
        copies, counts, _ = D.dflash_kv_compact(pool, page_table=table, lens=lens,
                                                copies=torch.empty((most, 2), dtype=torch.int32, device=DEV))
        D.dflash_kv_copy_pages(cache, copies, counts)
        check()
    held = int((refs > 0).sum())
    assert (refs[:held] > 0).all()
    grow([30, 1, 1, 5, 1, 1], 3)
    check()


def test_captured_lives():
    """Fork, resize and copies in one graph; replays on new parents and lengths
    equal eager calls, other work of the program in between."""
    require_gpu()
    say("captured lives")
    n, width, page, n_pages = 8, 20, 4, 200

    def make():
        cache = D.KVCache(torch.zeros((n_pages, 1, page, 64), dtype=torch.int8, device=DEV).random_(-99, 99, generator=torch.Generator(device=DEV).manual_seed(3)),
                          torch.ones((n_pages, 1, page, 64), dtype=torch.int8, device=DEV),
                          *(torch.full((n_pages, 1, page), 127, dtype=torch.uint8, device=DEV) for _ in "kv"))
        s = dict(cache=cache, refs=gpu(np.zeros(n_pages)), table=gpu(np.full((n, width), -1)), lens=gpu(np.zeros(n)),
                 copies=gpu(np.zeros((n, 2))), counts=gpu([0, 0]))
        s["pool"] = D.KVPool(s["refs"], page)
        return s

    parents, want = gpu(range(n)), gpu([9] * n)

    def step(s):
        kw = dict(page_table=s["table"], lens=s["lens"])
        D.dflash_kv_fork(s["pool"], parents=parents, **kw)
        D.dflash_kv_resize(s["pool"], want=want, copies=s["copies"], counts=s["counts"], **kw)
        D.dflash_kv_copy_pages(s["cache"], s["copies"], s["counts"])
        D.dflash_kv_compact(s["pool"], **kw)

    s, e = make(), make()
    for x in (s, e):
        step(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s)
    rng = np.random.default_rng(0)
    for i in range(5):
        parents.copy_(gpu(rng.integers(-1, n, n)))
        want.copy_(gpu(rng.integers(0, width * page + 1, n)))
        graph.replay()
        step(e)
        torch.cuda.synchronize()
        for name in ("refs", "table", "lens", "copies", "counts"):
            assert torch.equal(s[name], e[name]), (i, name)
        assert torch.equal(s["cache"].k, e["cache"].k)


def test_idle_calls_and_other_streams():
    require_gpu()
    say("idle calls, streams")
    b = empty(10, 2, 4, 4)
    none = dict(page_table=b.g_table[:0], lens=b.g_lens[:0])
    copies, counts = D.dflash_kv_resize(b.pool, want=gpu([]), **none)
    assert counts.tolist() == [0, 0] and copies.shape == (0, 2)
    D.dflash_kv_fork(b.pool, parents=gpu([]), **none)
    _, counts, page_map = D.dflash_kv_compact(b.pool, **none)
    assert counts.tolist() == [0, 0] and page_map.tolist() == [-1] * 10
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    P.resize(b.refs, b.table, b.lens, [13, 3], 4)
    want = gpu([13, 3])
    torch.cuda.synchronize()
    _, counts = D.dflash_kv_resize(b.pool, want=want, stream=side, **b.kw())
    side.synchronize()
    assert counts.tolist() == [0, 0]
    b.check("side stream")


def test_binding_refuses():
    require_gpu()
    say("binding refusals")
    b = empty(10, 2, 4, 4)
    with pytest.raises(ValueError, match="refs"):
        D.KVPool(b.g_refs.long(), 4)
    with pytest.raises(ValueError, match="want"):
        D.dflash_kv_resize(b.pool, want=gpu([1, 2, 3]), **b.kw())
    with pytest.raises(ValueError, match="copies"):
        D.dflash_kv_resize(b.pool, want=gpu([1, 2]), copies=gpu([[0, 0]]), **b.kw())
    with pytest.raises(ValueError, match="parents"):
        D.dflash_kv_fork(b.pool, parents=gpu([1, 2]).long(), **b.kw())
    with pytest.raises(D.DFlashError, match="overlaps"):
        D.dflash_kv_resize(b.pool, want=b.g_lens, **b.kw())
    with pytest.raises(D.DFlashError, match="workspace"):
        D.dflash_kv_fork(b.pool, parents=gpu([0, 0]), workspace=torch.empty(256, dtype=torch.uint8, device=DEV), **b.kw())
    cache = D.KVCache.empty(10, 1, 4, 64)
    other = D.KVCache.empty(10, 1, 8, 64)
    with pytest.raises(D.DFlashError, match="bounds"):
        D.dflash_kv_copy_pages(cache, gpu([[0, 1]]), bounds=D.KVBounds.empty(other))
    b.check("nothing has changed")


@pytest.mark.parametrize("n", [2047, 2048, 2049, 5000])
def test_pages_to_the_first_and_the_last_of_many_requests(n):
    """Requests between them that take nothing, more than a workgroup keeps."""
    require_gpu()
    say(f"first and last of {n}")
    page, width, n_pages = 4, 5, 20_000
    refs, table, lens = gpu(np.zeros(n_pages)), gpu(np.full((n, width), -1)), gpu(np.zeros(n))
    refs[::2] = -1
    want = np.zeros(n)
    want[0], want[1], want[n // 2], want[n - 1] = 9, 20, 1, 17
    copies, counts = D.dflash_kv_resize(D.KVPool(refs, page), page_table=table, lens=lens, want=gpu(want))
    assert counts.tolist() == [0, 0]
    rows = table.cpu().numpy()
    free = 1
    for r, need in ((0, 3), (1, 5), (n // 2, 1), (n - 1, 5)):
        assert rows[r].tolist() == [free + 2 * i for i in range(need)] + [-1] * (width - need), r
        free += 2 * need
    assert int((table >= 0).sum()) == 14 and int((refs == 1).sum()) == 14
