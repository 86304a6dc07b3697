"""CPU checks of what the write and the commit say to caches whose parts
overlap: two unordered writers on the same bytes.  Caches that are taken are
told by the next refusal, so that nothing is launched."""
import pytest

from block_draft_proposal_amd import binding as B
from block_draft_proposal_amd import kv as K
from test_abi_kv import CACHE, SCALED, _commit, _read, _tree, _write

EXTENT = 8 * 16 * 128                                   # elements of a page of CACHE; a page's scales are 128 bytes
AT = CACHE["k"]
CALLS = [lambda c: _write(cache=c, k=None), lambda c: _commit(cache=c, paths=None)]


def _said(call, cache):
    assert call(cache) == -1
    return B.last_error()


def _cache(k=0, v=0, stride=2 * EXTENT, pages=10, dtype=B.DFLASH_BF16, ks=None, vs=None, scale_stride=0):
    """Addresses from one pool's start, in bytes; stride in elements."""
    at = lambda x: None if x is None else AT + x  # noqa: E731
    return dict(k=AT + k, v=AT + v, page_stride=stride, n_pages=pages, dtype=dtype, k_scale=at(ks), v_scale=at(vs), scale_page_stride=scale_stride)


BYTES = 2 * EXTENT                                      # of a bf16 page
OVERLAPPING = [
    _cache(v=0), _cache(v=16), _cache(v=16 * 128 * 2), _cache(v=BYTES - 16), _cache(v=BYTES + 16), _cache(v=2 * BYTES - 16),
    _cache(k=16), _cache(k=BYTES + 16), _cache(k=3 * BYTES + 16), _cache(v=2 * BYTES * 9), _cache(v=2 * BYTES * 9 + BYTES - 16),
    _cache(v=BYTES, stride=EXTENT), _cache(v=16, stride=EXTENT), _cache(v=BYTES - 16, pages=1),
    _cache(v=BYTES, stride=EXTENT + 8),                 # a gap that is too small
]
APART = [
    _cache(v=BYTES), _cache(k=BYTES), _cache(v=3 * BYTES), _cache(v=2 * BYTES * 9 + BYTES), _cache(v=10 * BYTES, stride=EXTENT),
    _cache(v=BYTES + 16, stride=2 * EXTENT + 8), _cache(v=BYTES, pages=1), _cache(v=BYTES, stride=1 << 30, pages=1),
]
# int8: [K | V | K's scales | V's scales] in each page of one pool
E, F = EXTENT, 8 * 16
WHOLE = 2 * E + 2 * F
ONE_POOL = dict(v=E, stride=WHOLE, dtype=K.DFLASH_I8, ks=2 * E, vs=2 * E + F, scale_stride=WHOLE)
SCALES_OVERLAP = [
    {**ONE_POOL, "vs": 2 * E}, {**ONE_POOL, "vs": 2 * E + 1}, {**ONE_POOL, "vs": 2 * E + F + 1}, {**ONE_POOL, "ks": 2 * E - 1},
    {**ONE_POOL, "ks": E}, {**ONE_POOL, "ks": 5}, {**ONE_POOL, "scale_stride": WHOLE + 16}, {**ONE_POOL, "ks": 7 * WHOLE + E - F},
]
SCALES_APART = [
    ONE_POOL, {**ONE_POOL, "ks": 7 * WHOLE + 2 * E}, {**ONE_POOL, "ks": 20 * WHOLE, "vs": 20 * WHOLE + 10 * F, "scale_stride": F},
    {**ONE_POOL, "ks": 20 * WHOLE, "vs": 20 * WHOLE + F, "scale_stride": 2 * F}, {**ONE_POOL, "scale_stride": F, "pages": 1},
]


@pytest.mark.parametrize("call", CALLS, ids=["write", "commit"])
def test_parts_that_overlap_are_refused(call):
    for c in OVERLAPPING:
        assert "overlap" in _said(call, c), c
    for c in SCALES_OVERLAP:
        assert "overlap" in _said(call, _cache(**c)), c
    for c in (dict(v=AT), {**SCALED, "v_scale": SCALED["k_scale"] + 1}, {**SCALED, "k_scale": AT + 64}, {**SCALED, "v_scale": 2 * AT + 64}):
        assert "overlap" in _said(call, c), c


@pytest.mark.parametrize("call", CALLS, ids=["write", "commit"])
def test_parts_in_each_others_gaps_are_taken(call):
    for c in APART + [_cache(**c) for c in SCALES_APART] + [dict(), SCALED]:
        assert "null" in _said(call, c), (c, B.last_error())


def test_against_every_byte_of_small_pools():
    """The rule, counted out: 3 pages of 4 kinds of stride, V's and the scales'
    offsets a step of 16 (1 for scales) apart."""
    dim, heads, page = 64, 1, 1
    small = dict(head_dim=dim, n_kv_heads=heads, page_size=page, n_pages=3, dtype=K.DFLASH_I8)
    far = 1 << 20
    for stride in (64, 80, 128, 160):
        pages = lambda at, n, s: {at + i * s + j for i in range(3) for j in range(n)}  # noqa: E731
        for off in range(-3 * stride, 3 * stride + 1, 16):
            c = dict(small, k=AT, v=AT + off, page_stride=stride, k_scale=AT + far, v_scale=AT + 2 * far, scale_page_stride=stride)
            meet = bool(pages(0, dim, stride) & pages(off, dim, stride))
            assert ("overlap" in _said(CALLS[0], c)) == meet, (stride, off)
        for off in range(-3 * stride, 3 * stride + 1):
            c = dict(small, k=AT, v=AT + far, page_stride=stride, k_scale=AT + off, v_scale=AT + 2 * far, scale_page_stride=stride)
            meet = bool(pages(0, dim, stride) & pages(off, 1, stride))
            assert ("overlap" in _said(CALLS[0], c)) == meet, (stride, off)


def test_calls_that_only_read_take_such_a_cache():
    for c in OVERLAPPING:
        assert _read(cache=c, k=None) == -1 and "null output" in B.last_error()
        assert _tree(cache=c, q=None) == -1 and "null q" in B.last_error()
