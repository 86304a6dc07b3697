"""GPU tests of the paged KV cache: write, read and commit through the C ABI
against the float64 oracle.  Codes, scales and values read back are exact, so
every comparison is for equality."""
import numpy as np
import pytest
import torch

import block_draft_proposal_amd as D
from gpu_helpers import DEV, require_gpu, say
from kv_helpers import TYPES, codes_f64, dead_cache, make_plan, oracle_cache, rand_rows
from oracle import kv_oracle as O

pytestmark = pytest.mark.gpu

SHAPES = [
    # start, rows, page, heads, dim
    ([0], [1], 16, 1, 64),
    ([0, 5, 31], [1, 0, 7], 16, 2, 128),
    ([3, 0, 17, 40, 0], [10, 33, 1, 5, 0], 20, 3, 64),
    ([0, 100], [129, 2], 1, 1, 128),
    ([7, 64, 65, 1], [70, 64, 3, 9], 64, 5, 256),
]


def _same(got, ref, name):
    np.testing.assert_array_equal(got, ref, err_msg=name)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"r{len(s[0])}p{s[2]}h{s[3]}d{s[4]}")
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_write_then_read(shape, kind, io):
    require_gpu()
    start, rows, page, heads, dim = shape
    (table, st, off), host, n_pages, n_rows = make_plan(start, rows, page, seed=len(rows))
    say(f"write/read {shape} {kind} {io}")
    k, v = rand_rows(n_rows, heads, dim, io, 1), rand_rows(n_rows, heads, dim, io, 2)
    k[0, 0], v[-4, -1] = 0, 1e-38                       # rows of zeros and of tiny values
    tensors = dead_cache(kind, n_pages, heads, page, dim)
    want = oracle_cache(*tensors)
    cache = D.KVCache(*tensors)
    D.dflash_kv_write(cache, k, v, page_table=table, start=st, offsets=off)
    torch.cuda.synchronize()
    src = [codes_f64(x.to(torch.bfloat16) if kind == "bf16" else x) for x in (k, v)]
    O.write(want, kind, *src, *host)
    for name, t in zip(("k", "v"), tensors):
        _same(codes_f64(t), want[name], name)
    for name, t in zip(("k_scale", "v_scale"), tensors[2:]):
        if t is not None:
            _same(t.cpu().numpy(), want[name], name)
    outs = [torch.full((n_rows, heads, dim), -5.0, dtype=TYPES[io], device=DEV) for _ in "kv"]
    D.dflash_kv_read(cache, page_table=table, start=st, offsets=off, k_out=outs[0], v_out=outs[1])
    torch.cuda.synchronize()
    ref = [np.full((n_rows, heads, dim), -5.0) for _ in "kv"]
    O.read(want, *host, ref)
    for o, r, name in zip(outs, ref, "kv"):
        r = torch.from_numpy(r).to(torch.float32).to(TYPES[io]).double().numpy()
        _same(codes_f64(o), r, f"{name} read back")     # padding rows stay -5


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_rows_with_infinities_read_as_nan_and_leave_their_neighbours(kind):
    require_gpu()
    (table, st, off), host, n_pages, n_rows = make_plan([2], [6], 8)
    say(f"non-finite rows {kind}")
    k, v = rand_rows(n_rows, 2, 64, "f32", 3, packed=False), rand_rows(n_rows, 2, 64, "f32", 4, packed=False)
    k[1, 0, 5], k[3, 1, 63], v[0, 1, 0] = float("inf"), float("nan"), float("-inf")
    cache = D.KVCache.empty(n_pages, 2, 8, 64, TYPES[kind])
    D.dflash_kv_write(cache, k, v, page_table=table, start=st, offsets=off)
    ko, vo = D.dflash_kv_read(cache, page_table=table, start=st, offsets=off, n_rows=n_rows, dtype=torch.float32)
    torch.cuda.synchronize()
    bad_k, bad_v = (torch.isnan(x[:6]).all(-1).cpu().numpy() for x in (ko, vo))
    assert {tuple(map(int, x)) for x in np.argwhere(bad_k)} == {(1, 0), (3, 1)}
    assert {tuple(map(int, x)) for x in np.argwhere(bad_v)} == {(0, 1)}
    assert int(torch.isnan(ko[:6]).sum()) == 2 * 64


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_every_rounding_case_of_a_code(kind):
    """Midpoints between neighbouring codes, and values a step of fp32 beside them."""
    require_gpu()
    top = O.TOP[kind]
    grid = np.arange(-127, 128.0) if kind == "i8" else np.unique(O.nearest_code(np.linspace(-448, 448, 1 << 16), kind))
    if kind == "e4m3":
        grid = np.unique(np.concatenate([grid, np.arange(-64, 65) * 2.0 ** -9]))
    mids = ((grid[1:] + grid[:-1]) / 2).astype(np.float32)
    x = np.concatenate([mids, np.nextafter(mids, np.float32(np.inf)), np.nextafter(mids, np.float32(-np.inf))])
    x = np.resize(x, (-(-x.size // 63), 63))
    x = np.concatenate([np.full((len(x), 1), top, dtype=np.float32), x], axis=1)    # the first element fixes the scale at 1
    n = len(x)
    rows = torch.from_numpy(x[:, None].copy()).to(DEV)
    (table, st, off), host, n_pages, n_rows = make_plan([0], [n], 16, pad=0)
    say(f"midpoints {kind} {n} rows")
    cache = D.KVCache.empty(n_pages, 1, 16, 64, TYPES[kind])
    D.dflash_kv_write(cache, rows, -rows, page_table=table, start=st, offsets=off)
    ko, vo = D.dflash_kv_read(cache, page_table=table, start=st, offsets=off, n_rows=n, dtype=torch.float32)
    torch.cuda.synchronize()
    want = O.nearest_code(x.astype(np.float64), kind)
    _same(ko[:, 0].double().cpu().numpy(), want, "k")
    _same(vo[:, 0].double().cpu().numpy(), -want, "v")


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 20), (256, 1)])
def test_commit(kind, dim, page):
    require_gpu()
    nodes, heads = 40, 3
    paths_list = [[0, 1, 2, 3], [0, 5, 6, 20, 39], [], [7], [0] + list(range(2, 40)), list(range(40))]
    start = [0, 13, 5, 64, 31, 2]
    (table, st, off), host, n_pages, n_rows = make_plan(start, [nodes] * len(start), page, seed=9)
    say(f"commit {kind} d{dim} p{page}")
    tensors = dead_cache(kind, n_pages, heads, page, dim)
    cache = D.KVCache(*tensors)
    everything = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0] * len(start), np.cumsum([0] + [s + nodes for s in start]))]
    total = int(everything[1][-1])
    D.dflash_kv_write(cache, rand_rows(total, heads, dim, "bf16", 5), rand_rows(total, heads, dim, "bf16", 6),
                      page_table=table, start=everything[0], offsets=everything[1])
    torch.cuda.synchronize()
    want = oracle_cache(*tensors)
    width = max(map(len, paths_list)) + 2
    paths = np.full((len(start), width), 10 ** 6, dtype=np.int32)
    for r, p in enumerate(paths_list):
        paths[r, :len(p)] = p
    lens = np.array([len(p) for p in paths_list], dtype=np.int32)
    D.dflash_kv_commit(cache, page_table=table, start=st, paths=torch.from_numpy(paths).to(DEV),
                       path_lens=torch.from_numpy(lens).to(DEV))
    torch.cuda.synchronize()
    O.commit(want, host[0], host[1], paths, lens)
    for name, t in zip(("k", "v", "k_scale", "v_scale"), tensors):
        if t is not None:
            _same(codes_f64(t) if "scale" not in name else t.cpu().numpy(), want[name], name)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_positions_without_a_page(kind):
    """Pages outside the pool and positions past the table: not written, read
    as NaN, not moved; everything else as usual."""
    require_gpu()
    heads, page, dim = 2, 8, 64
    table = torch.tensor([[3, -1, 1], [0, 2, 999]], dtype=torch.int32, device=DEV)
    st = torch.tensor([4, 10], dtype=torch.int32, device=DEV)
    off = torch.tensor([0, 30, 50], dtype=torch.int32, device=DEV)     # request 0 runs past its 24 positions
    host = tuple(x.cpu().numpy() for x in (table, st, off))
    say(f"bad pages {kind}")
    tensors = dead_cache(kind, 4, heads, page, dim)
    for t in tensors[:2]:
        (t if kind == "bf16" else t.view(torch.uint8)).fill_(1)
    want = oracle_cache(*tensors)
    cache = D.KVCache(*tensors)
    k, v = rand_rows(52, heads, dim, "bf16", 7), rand_rows(52, heads, dim, "bf16", 8)
    D.dflash_kv_write(cache, k, v, page_table=table, start=st, offsets=off)
    outs = D.dflash_kv_read(cache, page_table=table, start=st, offsets=off, n_rows=52, dtype=torch.float32)
    torch.cuda.synchronize()
    O.write(want, kind, codes_f64(k), codes_f64(v), *host)
    for name, t in zip("kv", tensors):
        _same(codes_f64(t), want[name], name)
    ref = [np.zeros((52, heads, dim)) for _ in "kv"]
    O.read(want, *host, ref)
    for o, r in zip(outs, ref):
        _same(o[:50].double().cpu().numpy(), r[:50], "read")
        assert np.isnan(r).any()
    paths = np.array([[1, 5, 12, 25], [1, 3, 9, 13]], dtype=np.int32)
    lens = np.array([4, 4], dtype=np.int32)
    D.dflash_kv_commit(cache, page_table=table, start=st, paths=torch.from_numpy(paths).to(DEV),
                       path_lens=torch.from_numpy(lens).to(DEV))
    torch.cuda.synchronize()
    O.commit(want, host[0], host[1], paths, lens)
    for name, t in zip("kv", tensors):
        _same(codes_f64(t), want[name], name + " after commit")


def test_offsets_beyond_32_bits_and_one_pool_for_k_and_v():
    """K and V interleaved in one pool whose pages lie 2 GiB apart, so that a
    page's byte offset passes 32 bits."""
    require_gpu()
    heads, page, dim = 2, 16, 128
    need = heads * page * dim
    pool = torch.empty(2 * (1 << 31) + 4096 * need, dtype=torch.int8, device=DEV)
    k = pool.as_strided((3, heads, page, dim), ((1 << 31) + 64, page * dim, dim, 1))
    v = pool.as_strided((3, heads, page, dim), ((1 << 31) + 64, page * dim, dim, 1), storage_offset=need)
    scales = [torch.zeros((3, heads, page), dtype=torch.uint8, device=DEV) for _ in "kv"]
    (table, st, off), host, _, n_rows = make_plan([0], [40], page)
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    say("pages 2 GiB apart")
    cache = D.KVCache(k, v, *scales)
    x, y = rand_rows(n_rows, heads, dim, "bf16", 11), rand_rows(n_rows, heads, dim, "bf16", 12)
    D.dflash_kv_write(cache, x, y, page_table=table, start=st, offsets=off)
    outs = D.dflash_kv_read(cache, page_table=table, start=st, offsets=off, n_rows=n_rows, dtype=torch.float32)
    torch.cuda.synchronize()
    for src, o in zip((x, y), outs):
        codes, b = O.quantise_rows(codes_f64(src)[:40], "i8")
        _same(o[:40].double().cpu().numpy(), codes * O.scale_value(b)[..., None], "values")


def test_many_requests_empty_ones_among_them():
    require_gpu()
    rng = np.random.default_rng(4)
    rows = rng.integers(0, 3, size=5000)
    (table, st, off), host, n_pages, n_rows = make_plan(rng.integers(0, 40, size=5000), rows, 16, seed=5)
    say("5000 requests")
    cache = D.KVCache.empty(n_pages, 1, 16, 64)
    k, v = rand_rows(n_rows, 1, 64, "bf16", 13), rand_rows(n_rows, 1, 64, "bf16", 14)
    D.dflash_kv_write(cache, k, v, page_table=table, start=st, offsets=off)
    ko, vo = D.dflash_kv_read(cache, page_table=table, start=st, offsets=off, n_rows=n_rows)
    torch.cuda.synchronize()
    n = int(host[2][-1])
    assert torch.equal(ko[:n], k[:n]) and torch.equal(vo[:n], v[:n])
    for r in (0, 17, 2500, 4999):
        for i in range(int(rows[r])):
            t = int(host[1][r]) + i
            assert torch.equal(cache.k[host[0][r, t // 16], :, t % 16], k[int(host[2][r]) + i])


def test_capture_and_another_stream():
    """A captured write, commit and read, replayed on changed inputs, against
    eager calls; the eager calls on a side stream."""
    require_gpu()
    (table, st, off), host, n_pages, n_rows = make_plan([3, 0], [20, 12], 16)
    k, v = rand_rows(n_rows, 2, 128, "bf16", 15, packed=False), rand_rows(n_rows, 2, 128, "bf16", 16, packed=False)
    paths = torch.tensor([[0, 4, 9], [1, 2, 5]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([3, 2], dtype=torch.int32, device=DEV)

    def step(cache, outs, stream=None):
        kw = dict(page_table=table, start=st, stream=stream)
        D.dflash_kv_write(cache, k, v, offsets=off, **kw)
        D.dflash_kv_commit(cache, paths=paths, path_lens=lens, **kw)
        D.dflash_kv_read(cache, k_out=outs[0], v_out=outs[1], offsets=off, **kw)

    make = lambda: (D.KVCache(*dead_cache("e4m3", n_pages, 2, 16, 128)), [torch.zeros((n_rows, 2, 128), device=DEV) for _ in "kv"])  # noqa: E731
    captured, eager = make(), make()
    say("captured write, commit, read")
    step(*captured)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*captured)
    side = torch.cuda.Stream()
    for i in range(4):
        k.copy_(rand_rows(n_rows, 2, 128, "bf16", 20 + i, packed=False))
        paths[0, 2] = 9 + i
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        step(*eager, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        for a, b in zip(captured[1], eager[1]):
            assert torch.equal(a, b)
        assert torch.equal(captured[0].k.view(torch.uint8), eager[0].k.view(torch.uint8))


@pytest.mark.parametrize("dim,heads", [(64, 9), (128, 8), (256, 5)])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_large_batches_equal_small_ones(dim, heads, kind, io):
    """Many rows at once, several (head, K or V) pairs to a thread, against the
    same rows a few requests at a time, and K's rows against the oracle."""
    require_gpu()
    say(f"large batch {dim} {heads} {kind} {io}")
    rng = np.random.default_rng(dim)
    rows = rng.integers(0, 300, size=56)
    (table, st, off), host, n_pages, n_rows = make_plan(rng.integers(0, 40, size=56), rows, 16, seed=3)
    k, v = rand_rows(n_rows, heads, dim, io, 31), rand_rows(n_rows, heads, dim, io, 32)
    large, small = (dead_cache(kind, n_pages, heads, 16, dim) for _ in range(2))
    D.dflash_kv_write(D.KVCache(*large), k, v, page_table=table, start=st, offsets=off)
    for r in range(0, 56, 4):
        a, b = int(host[2][r]), int(host[2][r + 4])
        if b > a:
            D.dflash_kv_write(D.KVCache(*small), k[a:b], v[a:b], page_table=table[r:r + 4], start=st[r:r + 4], offsets=off[r:r + 5] - a)
    torch.cuda.synchronize()
    for x, y in zip(large, small):
        assert x is None or torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    want = oracle_cache(*(t[:, :1] if t is not None else None for t in dead_cache(kind, n_pages, 1, 16, dim)))
    one = [codes_f64((x.to(torch.bfloat16) if kind == "bf16" else x)[:, -1:]) for x in (k, v)]
    O.write(want, kind, *one, *host)
    _same(codes_f64(large[0][:, -1:]), want["k"], "k of the last head")
    ko, vo = D.dflash_kv_read(D.KVCache(*large), page_table=table, start=st, offsets=off, n_rows=n_rows, dtype=TYPES[io])
    ref = [np.zeros((n_rows, 1, dim)) for _ in "kv"]
    O.read(want, *host, ref)
    n = int(host[2][-1])
    for o, r, name in zip((ko, vo), ref, "kv"):
        _same(codes_f64(o[:n, -1:]), torch.from_numpy(r[:n]).to(torch.float32).to(TYPES[io]).double().numpy(), name)
