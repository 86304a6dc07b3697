"""GPU tests that the operators on pages and chosen blocks write nothing outside
their outputs and the workspace that they asked for, and nothing in rows that are
no request's."""
import numpy as np
import pytest
import torch

import block_draft_proposal_amd as D
from gpu_helpers import DEV, require_gpu, say
from kv_helpers import attention_bound, codes_f64, make_plan, mask_tensor, oracle_cache, rand_rows, tree_mask
from launch_helpers import launches
from oracle import sparse_oracle as S
from test_gpu_kv_sparse import gpu, pick, rand_bounds, written

pytestmark = pytest.mark.gpu
EDGE = 4096


class Guarded:
    """Tensors with EDGE bytes on either side that have to stay."""

    def __init__(self):
        self.held = []

    def __call__(self, shape, dtype=torch.uint8):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        whole = torch.full((2 * EDGE + n,), 0xA5, dtype=torch.uint8, device=DEV)
        self.held.append((whole, n))
        return whole[EDGE:EDGE + n].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for whole, n in self.held:
            assert (whole[:EDGE] == 0xA5).all() and (whole[EDGE + n:] == 0xA5).all()


@pytest.mark.parametrize("n_pages,n,width,page", [(50, 5, 9, 4), (8192, 1024, 32, 16), (8193, 1024, 32, 16), (9000, 3, 12000, 1), (30000, 2000, 17, 3)])
def test_page_tables(n_pages, n, width, page):
    require_gpu()
    say(f"guarded pages {n_pages} {n} {width}")
    rng = np.random.default_rng(n)
    g = Guarded()
    refs, table, lens, want = g((n_pages,), torch.int32), g((n, width), torch.int32), g((n,), torch.int32), g((n,), torch.int32)
    copies, counts, page_map = g((n, 2), torch.int32), g((2,), torch.int32), g((n_pages,), torch.int32)
    moves = g((n_pages // 2, 2), torch.int32)
    refs.zero_(), table.fill_(-1), lens.zero_()
    pool = D.KVPool(refs, page)
    work = g((D.kv_pages_workspace_size(pool, n_req=n, table_width=width),))
    books = dict(page_table=table, lens=lens, workspace=work)
    for step in range(4):
        want.copy_(gpu(rng.integers(0, min(width, n_pages // n) * page + 1, n)))
        D.dflash_kv_resize(pool, want=want, copies=copies, counts=counts, **books)
        D.dflash_kv_fork(pool, parents=gpu(rng.integers(-1, n, n)), **books)
        D.dflash_kv_compact(pool, copies=moves, counts=counts, page_map=page_map, **books)
    g.check()
    t, need = table.cpu().numpy(), -(-lens.cpu().numpy() // page)
    held = t[np.arange(width) < need[:, None]]
    np.testing.assert_array_equal(np.bincount(held, minlength=n_pages), refs.cpu().numpy())


@pytest.mark.parametrize("dim,heads,group,nodes,n_req,blocks,take,form", [
    (64, 2, 3, 1, 3, 700, 33, "select_take_wave_kernel<18>"), (128, 1, 4, 5, 2, 3000, 7, "select_take_wave_kernel<68>"),
    (64, 2, 1, 2, 2, 9000, 900, "select_take_kernel<1024, 8>"), (128, 8, 2, 16, 17, 90, 64, "select_fused_kernel<128, 16>"),
    (256, 16, 2, 8, 9, 40, 50, "select_fused_kernel<256, 8>")])
def test_choice(dim, heads, group, nodes, n_req, blocks, take, form):
    """Rows before the first request, behind the last and between two of them, and
    strides of the table, too."""
    require_gpu()
    say(f"guarded choice {dim} {nodes} {blocks}")
    plan, host, n_pages, n_rows = make_plan([blocks - 3 * r for r in range(n_req)], [nodes] * n_req, 1, seed=3)
    b = rand_bounds(n_pages, heads, dim, 1, 5)
    q = rand_rows(n_rows + 7, heads * group, dim, "bf16", 6)
    g = Guarded()
    offsets, out = g((n_req + 1,), torch.int32), g((n_rows + 7, heads, take), torch.int32)
    table = g((n_req, plan[0].shape[1] + 5), torch.int32)
    table[:, :plan[0].shape[1]].copy_(plan[0])
    offsets.copy_(plan[2] + 4)
    out.fill_(-9)
    work = g((D.kv_select_workspace_size(b, n_rows=n_rows + 7, table_width=plan[0].shape[1]),))

    def call():
        D.dflash_kv_select(q, b, page_table=table[:, :plan[0].shape[1]], start=plan[1], offsets=offsets, max_nodes=nodes, out=out, workspace=work)

    assert launches(call)[-1][0] == form
    call()
    g.check()
    rows = n_req * nodes
    want = D.dflash_kv_select(q[4:4 + rows], b, page_table=plan[0], start=plan[1], offsets=plan[2], max_nodes=nodes, n_take=take)
    assert torch.equal(out[4:4 + rows], want) and (out[:4] == -9).all() and (out[4 + rows:] == -9).all()


@pytest.mark.parametrize("kind,dim,heads,group,nodes,start,take", [
    ("bf16", 128, 2, 4, 1, 2000, 120), ("e4m3", 256, 2, 33, 1, 1500, 90), ("i8", 64, 1, 40, 1, 1900, 118), ("bf16", 64, 2, 2, 1, 60, 2),
    ("bf16", 128, 2, 4, 16, 900, 50), ("e4m3", 64, 1, 2, 33, 1500, 90), ("i8", 256, 2, 4, 8, 700, 40), ("e4m3", 128, 8, 2, 9, 60, 3)])
def test_attention(kind, dim, heads, group, nodes, start, take):
    """Masks of more words than needed, rows before the first request and behind
    the last."""
    require_gpu()
    say(f"guarded attention {kind} {dim} {group} {nodes}")
    page = 16
    cache, tensors, plan, host, n_rows = written(kind, [start, start // 2, 0], [nodes, nodes, nodes // 2], page, heads, dim)
    last = int(host[2][-1])
    blocks = pick(host, n_rows, heads, page, take, 2, kind="all")
    mask = tree_mask(n_rows, host[2], 3)
    q = rand_rows(n_rows + 4, heads * group, dim, "bf16", 9)
    g = Guarded()
    out, chosen, bits = g((n_rows + 4, heads * group, dim), torch.bfloat16), g((n_rows + 4, heads, take), torch.int32), g((n_rows + 4, 3), torch.int64)
    out.fill_(7)
    chosen.fill_(0x7fffffff), bits.fill_(-1)
    chosen[4:].copy_(gpu(blocks)), bits[4:].copy_(mask_tensor(mask))
    work = g((D.sparse_attention_workspace_size(cache, n_rows=n_rows + 4, n_take=take, max_nodes=nodes, n_q_heads=heads * group),))
    D.dflash_sparse_attention(q, cache, chosen, page_table=plan[0], start=plan[1], offsets=plan[2] + 4, max_nodes=nodes, mask=bits, out=out, workspace=work)
    g.check()
    want = np.full((n_rows, heads * group, dim), 7.0)
    spread, reach = S.sparse_attention(codes_f64(q[4:]), oracle_cache(*tensors), *host, blocks, mask, dim ** -0.5, want)
    got = codes_f64(out)
    assert (got[:4] == 7).all() and (got[4 + last:] == 7).all()
    assert (np.abs(got[4:] - want) <= attention_bound(want, spread, reach, dim)).all()
