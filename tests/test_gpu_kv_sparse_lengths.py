"""GPU tests of the attention over chosen pages where a request's length is
beyond its table: rows that see something are NaN, rows that see nothing zeros."""
import numpy as np
import pytest
import torch

import block_draft_proposal_amd as D
from gpu_helpers import DEV, require_gpu, say
from kv_helpers import codes_f64, mask_tensor, rand_rows
from test_gpu_kv_sparse import gpu, written

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("take", [4, 300])
@pytest.mark.parametrize("kind,dim,group,rows", [("bf16", 64, 2, 5), ("e4m3", 128, 4, 5), ("i8", 256, 1, 5), ("bf16", 128, 33, 5), ("i8", 64, 64, 5),
                                                 ("e4m3", 64, 3, 1), ("bf16", 256, 20, 1)])
def test_rows_that_see_nothing_beyond_the_table(kind, dim, group, rows, take):
    """Rows together and by themselves, few enough to be split over workgroups
    and not."""
    require_gpu()
    say(f"nothing beyond the table {kind} {dim} {group} {rows} {take}")
    page, heads = 16, 2
    cache, tensors, plan, host, n_rows = written(kind, [48] * rows + [20], [rows] * rows + [rows], page, heads, dim)
    kw = dict(page_table=plan[0][:, :3], start=plan[1], offsets=plan[2], max_nodes=rows)   # 48 + rows is past 3 pages
    blocks = np.full((n_rows, heads, take), -1, dtype=np.int32)
    mask = np.full((n_rows, 1), 0xffffffffffffffe0 if rows == 5 else 0xfffffffffffffffe, dtype=np.uint64)   # bits past the nodes
    sees = np.zeros((n_rows, heads), dtype=bool)
    for r in range(rows):
        at = int(host[2][r]) + r                          # another node of each request: of row 0, 1, ...
        what = r % 5 if rows == 5 else 2
        if what == 0:
            mask[at, 0] |= 1 << (rows - 1)                # a node
            sees[at] = True
        elif what == 1:
            blocks[at, 1, take - 1] = 2                   # a block, the last entry, for one of the heads
            sees[at, 1] = True
        elif what == 2:
            blocks[at, 0, :4] = [3, 0, -7, 2147483647]    # names nothing: beyond the prefix, and below the entry before
        elif what == 3:
            blocks[at, 0, :4] = [-1, -1, 0, 0]
            sees[at, 0] = True
    q = rand_rows(n_rows, heads * group, dim, "bf16", 5)
    last = int(host[2][rows])
    out = torch.full((n_rows, heads * group, dim), 7.0, dtype=torch.bfloat16, device=DEV)
    D.dflash_sparse_attention(q, cache, gpu(blocks), mask=mask_tensor(mask), out=out, **kw)
    got = codes_f64(out).reshape(n_rows, heads, group, dim)
    assert np.isnan(got[:last][sees[:last]]).all()
    assert (got[:last][~sees[:last]] == 0).all()
    assert np.isfinite(got[last:int(host[2][-1])]).all()   # the request within the table
    assert (got[int(host[2][-1]):] == 7).all()
    # without a mask every row sees itself
    D.dflash_sparse_attention(q, cache, gpu(blocks), out=out, **kw)
    assert torch.isnan(out[:last].float()).all()


@pytest.mark.parametrize("group", [2, 33])
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_nodes_beyond_the_table_are_those_of_the_tree_attention(kind, group):
    """No prefix, more nodes than the table's one page."""
    require_gpu()
    say(f"nodes beyond the table {kind} {group}")
    heads, dim, rows = 2, 64, 20
    cache, tensors, plan, host, n_rows = written(kind, [0, 0], [rows, 3], 16, heads, dim)
    mask = np.zeros((n_rows, 1), dtype=np.uint64)
    mask[::3, 0] = 1
    mask[1, 0] = 0xfffffffffff00000                       # bits past the nodes
    q = rand_rows(n_rows, heads * group, dim, "bf16", 5)
    kw = dict(page_table=plan[0][:, :1], start=plan[1], offsets=plan[2], max_nodes=rows, mask=mask_tensor(mask))
    got = codes_f64(D.dflash_sparse_attention(q, cache, gpu(np.zeros((n_rows, heads, 0))), **kw))
    want = codes_f64(D.dflash_tree_attention(q, cache, **kw))
    n = int(host[2][-1])
    for x in (got, want):
        assert np.isnan(x[:rows:3]).all() and (x[1:rows:3] == 0).all() and (x[2:rows:3] == 0).all()
        assert np.isfinite(x[rows:n]).all()
