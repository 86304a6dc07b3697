"""GPU tests of the forms of the attention over chosen pages: which one a call
takes, by its launches, and each against the float64 oracle."""
import numpy as np
import pytest
import torch

import block_draft_proposal_amd as D
from gpu_helpers import DEV, require_gpu, say
from kv_helpers import mask_tensor, rand_rows, tree_mask
from launch_helpers import launches
from test_gpu_kv_sparse import check_sparse, gpu, pick, written

pytestmark = pytest.mark.gpu
TYPE = {"bf16": 1, "e4m3": 2, "i8": 3}


def kernels(cache, plan, n_rows, group, blocks, max_nodes, mask=None):
    """[(kernel, workgroups, threads of one)] of the call that check_sparse makes."""
    heads, dim = cache.n_kv_heads, cache.head_dim
    q = rand_rows(n_rows, heads * group, dim, "bf16", 1)
    out = torch.empty((n_rows, heads * group, dim), dtype=torch.bfloat16, device=DEV)
    at, bits = gpu(blocks), mask_tensor(mask)
    work = torch.empty(D.sparse_attention_workspace_size(cache, n_rows=n_rows, n_take=blocks.shape[2], max_nodes=max_nodes, n_q_heads=heads * group),
                       dtype=torch.uint8, device=DEV)
    return launches(lambda: D.dflash_sparse_attention(q, cache, at, page_table=plan[0], start=plan[1], offsets=plan[2], max_nodes=max_nodes,
                                                      mask=bits, out=out, workspace=work))


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("dim,group,tiles", [(64, 3, 1), (64, 20, 2), (64, 40, 4), (64, 64, 4), (128, 4, 1), (128, 20, 2), (128, 33, 4), (128, 64, 4),
                                             (256, 4, 1), (256, 20, 2), (256, 33, 2), (256, 64, 2)])
def test_few_single_rows_are_split(kind, dim, group, tiles):
    """Single rows over up to 2000 chosen keys: partial sums of several
    workgroups, of more than 16 heads and of more than one tile of them."""
    require_gpu()
    say(f"split rows {kind} {dim} {group}")
    heads, page, take = 2, 16, 125
    cache, tensors, plan, host, n_rows = written(kind, [2007, 300, 1999], [1, 1, 1], page, heads, dim)
    blocks = pick(host, n_rows, heads, page, take, 2, kind="all")
    blocks[2, 1, 7:] = -1                                # a short list: most of its workgroups have no keys
    ran = kernels(cache, plan, n_rows, group, blocks, 1)
    assert [x[0] for x in ran] == [f"sparse_attention_kernel<{TYPE[kind]}, {dim}, {tiles}>", f"sparse_join_kernel<{dim}, {tiles}>"], ran
    items = n_rows * heads * -(-group // (16 * tiles))
    assert ran[0][1] % items == 0 and ran[0][1] > items, ran
    check_sparse(cache, tensors, plan, host, n_rows, group, blocks, max_nodes=1)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("dim,group,tiles", [(64, 20, 2), (64, 40, 4), (128, 20, 2), (128, 33, 4), (256, 20, 2), (256, 64, 2)])
def test_single_rows_of_many_heads_whole(kind, dim, group, tiles):
    """Few keys: an item to a workgroup, no join."""
    require_gpu()
    say(f"whole rows {kind} {dim} {group}")
    cache, tensors, plan, host, n_rows = written(kind, [77, 0, 20, 130], [1, 1, 1, 1], 16, 2, dim)
    blocks = pick(host, n_rows, 2, 16, 4, 2)
    ran = kernels(cache, plan, n_rows, group, blocks, 1)
    assert [x[0] for x in ran] == [f"sparse_attention_kernel<{TYPE[kind]}, {dim}, {tiles}>"], ran
    check_sparse(cache, tensors, plan, host, n_rows, group, blocks, max_nodes=1)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("n_req", [2, 150])
def test_single_rows_of_more_blocks_than_are_read_at_once(kind, n_req):
    """Lists of more than 256 entries, named ones at both ends, and the last one
    alone behind many that name nothing."""
    require_gpu()
    say(f"long lists {kind} {n_req}")
    page, heads, take = 1, 8 if n_req > 2 else 2, 600
    start = [900 - 5 * (r % 40) for r in range(n_req)]
    cache, tensors, plan, host, n_rows = written(kind, start, [1] * n_req, page, heads, 64)
    blocks = pick(host, n_rows, heads, page, take, 3)
    blocks[0, 0] = -1
    blocks[0, 0, 599] = 800
    blocks[0, 1] = -1
    blocks[0, 1, 300:303] = [1, 5, 7]
    blocks[1, 0] = -1
    blocks[1, 0, 255:257] = [2, 894]
    blocks[1, 1, :] = np.arange(600)
    ran = kernels(cache, plan, n_rows, 2, blocks, 1)
    assert [x[0] for x in ran] == [f"sparse_attention_kernel<{TYPE[kind]}, 64, 1>"] + (["sparse_join_kernel<64, 1>"] if n_req == 2 else []), ran
    check_sparse(cache, tensors, plan, host, n_rows, 2, blocks, max_nodes=1)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
@pytest.mark.parametrize("dim,group,nodes,tiles", [(64, 4, 4, 1), (64, 4, 8, 2), (64, 4, 16, 4), (64, 1, 32, 2), (128, 4, 3, 1), (128, 2, 16, 2),
                                                   (128, 8, 7, 4), (256, 2, 8, 1), (256, 16, 2, 2)])
@pytest.mark.parametrize("split", [False, True])
def test_rows_together(kind, dim, group, nodes, tiles, split):
    """Trees whose rows fill one, two and four tiles of 16, whole and split."""
    require_gpu()
    say(f"tiles {kind} {dim} {group} {nodes} {split}")
    page, heads, take = 16, 2, 60 if split else 2
    cache, tensors, plan, host, n_rows = written(kind, [1100, 333], [nodes, nodes // 2 + 1], page, heads, dim)
    blocks = pick(host, n_rows, heads, page, take, 2, kind="all" if split else "some")
    mask = tree_mask(n_rows, host[2], 1)
    ran = kernels(cache, plan, n_rows, group, blocks, nodes, mask)
    main = f"<{TYPE[kind]}, {dim}, {tiles}>"
    assert [x[0] for x in ran] == ["sparse_union_kernel", "sparse_tile_kernel" + main] + (["sparse_tile_join_kernel" + main] if split else []), ran
    check_sparse(cache, tensors, plan, host, n_rows, group, blocks, mask)


@pytest.mark.parametrize("width,form", [(16384, "sparse_union_kernel"), (16385, "sparse_attention_kernel<3, 64, 1>")])
def test_the_longest_table_of_rows_together(width, form):
    """A word for each block of the table in LDS, and one block too many."""
    require_gpu()
    say(f"table of {width}")
    cache, tensors, plan, host, n_rows = written("i8", [width - 3, 90], [3, 2], 1, 1, 64)
    blocks = pick(host, n_rows, 1, 1, 40, 3, kind="all")
    blocks[0, 0, -1], blocks[1, 0, 0] = width - 4, 0
    ran = kernels(cache, plan, n_rows, 2, blocks, 3)
    assert ran[0][0] == form, ran
    check_sparse(cache, tensors, plan, host, n_rows, 2, blocks)
