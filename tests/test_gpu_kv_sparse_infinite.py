"""GPU tests of the attention over chosen pages with infinite keys: in the rows
that see them, by the definition, and in no others."""
import numpy as np
import pytest

import block_draft_proposal_amd as D
from gpu_helpers import require_gpu, say
from kv_helpers import codes_f64, rand_rows
from test_gpu_kv_sparse import gpu, written

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [[1, 1], [3, 2]])
@pytest.mark.parametrize("start", [40, 700])
@pytest.mark.parametrize("group", [3, 33])
def test_infinite_keys(rows, start, group):
    """A key whose product with the query is -infinity has weight 0; where it is
    +infinity or a NaN, the row is NaN.  By head and row, in every form."""
    require_gpu()
    say(f"infinite keys {rows} {start} {group}")
    page, heads, dim = 8, 1, 64
    cache, tensors, plan, host, n_rows = written("bf16", [start, start], rows, page, heads, dim)
    full = start // page
    blocks = np.full((n_rows, heads, full), -1, dtype=np.int32)
    blocks[:sum(rows)] = np.arange(full)
    q = rand_rows(n_rows, heads * group, dim, "bf16", 4).clone()
    q[..., 5] = q[..., 5].abs() + 1
    q[:, 1, 5] *= -1                                     # one head of the opposite sign
    q[:, 2, 5] = 0
    n = sum(rows)
    kw = dict(page_table=plan[0], start=plan[1], offsets=plan[2], max_nodes=max(rows))
    page_of = int(host[0][0, 2])                         # of the first request; the second has none of this
    was = cache.k[page_of, 0, 3].clone()
    for sign in (-1, 1):
        cache.k[page_of, 0, 3, 5] = sign * float("inf")
        got = codes_f64(D.dflash_sparse_attention(q, cache, gpu(blocks), **kw))
        weightless = [h for h in range(group) if (h != 1) == (sign < 0) and h != 2]
        nan = [h for h in range(group) if h not in weightless]
        assert np.isnan(got[:rows[0], nan]).all() and np.isfinite(got[:rows[0], weightless]).all()
        assert np.isfinite(got[rows[0]:n]).all()
        # the same as with a key so far below the others that its weight is 0 in fp32
        cache.k[page_of, 0, 3, 5] = sign * 3e4
        far = codes_f64(D.dflash_sparse_attention(q, cache, gpu(blocks), **kw))
        np.testing.assert_array_equal(got[:rows[0], weightless], far[:rows[0], weightless])
        cache.k[page_of, 0, 3] = was
    # who does not see the key keeps its result, whatever it is
    without = gpu(np.where(blocks == 2, -1, blocks))
    clean = codes_f64(D.dflash_sparse_attention(q, cache, without, **kw))
    cache.k[page_of, 0, 3, 5] = float("inf")
    got = codes_f64(D.dflash_sparse_attention(q, cache, without, **kw))
    np.testing.assert_array_equal(got[:n], clean[:n])


@pytest.mark.parametrize("rows", [[1], [3]])
def test_only_keys_of_minus_infinity(rows):
    """No key has a weight: NaN, as the definition's 0 / 0."""
    require_gpu()
    say(f"only -infinity {rows}")
    cache, tensors, plan, host, n_rows = written("bf16", [16], rows, 8, 1, 64)
    cache.k[..., 0] = -float("inf")
    q = rand_rows(n_rows, 2, 64, "bf16", 4).clone()
    q[..., 0] = 1
    got = codes_f64(D.dflash_sparse_attention(q, cache, gpu(np.full((n_rows, 1, 1), 1)), page_table=plan[0], start=plan[1], offsets=plan[2],
                                              max_nodes=rows[0]))
    assert np.isnan(got[:rows[0]]).all()
