"""GPU tests of the forms of the choice of blocks: which one a call takes, by its
launches, and each against the definition, on both sides of the sizes that
decide."""
import numpy as np
import pytest
import torch

import block_draft_proposal_amd as D
from gpu_helpers import DEV, require_gpu, say
from kv_helpers import codes_f64, make_plan, rand_rows
from launch_helpers import launches
from oracle import sparse_oracle as S
from test_gpu_kv_sparse import check_select, rand_bounds

pytestmark = pytest.mark.gpu


def choose(q, bounds, host, take, n_first, n_last, max_nodes, out):
    """The oracle's choice with the scores of a request's rows and blocks in one
    product of whole numbers (below 2^22: exact in float64)."""
    codes, scale = bounds.codes.cpu().numpy(), bounds.scale.cpu().numpy().astype(np.int64)
    table, start, offsets = host
    heads, group = codes.shape[1], q.shape[1] // codes.shape[1]
    for r in range(len(start)):
        blocks, first = S.n_blocks(start[r], bounds.page_size, table.shape[1]), int(offsets[r])
        n = min(int(offsets[r + 1]) - first, max_nodes)
        pages, b = table[r, :blocks], np.arange(blocks)
        lost = (pages < 0) | (pages >= bounds.n_pages)
        at, forced = np.where(lost, 0, pages), (b < n_first) | (b >= blocks - n_last)
        for h in range(heads if n else 0):
            low, high = codes[at, h, 0].astype(np.float64), codes[at, h, 1].astype(np.float64)
            c = np.concatenate([S.query_codes(q[first + i, h * group:(h + 1) * group]) for i in range(n)]).astype(np.float64)
            sums = (np.maximum(c, 0) @ high.T + np.minimum(c, 0) @ low.T).reshape(n, group, blocks).max(1)
            key = np.where(forced, np.inf, np.where(lost | (scale[at, h] == 255), 1e300, np.ldexp(sums, scale[at, h] - 127)))
            best = np.sort(np.argsort(-key, axis=1, kind="stable")[:, :take], axis=1)   # ties: the lower block
            out[first:first + n, h, :best.shape[1]], out[first:first + n, h, best.shape[1]:] = best, -1


def check(q, b, plan, host, max_nodes, take, n_first, n_last, want_launches=None):
    out = torch.full((q.shape[0], b.n_kv_heads, take), -9, dtype=torch.int32, device=DEV)
    work = torch.empty(D.kv_select_workspace_size(b, n_rows=q.shape[0], table_width=plan[0].shape[1]), dtype=torch.uint8, device=DEV)

    def call():
        D.dflash_kv_select(q, b, page_table=plan[0], start=plan[1], offsets=plan[2], max_nodes=max_nodes, n_first=n_first, n_last=n_last,
                           out=out, workspace=work)

    if want_launches is not None:
        ran = launches(call)
        assert [x[0] for x in ran] == want_launches, ran
    call()
    torch.cuda.synchronize()
    want = np.full(tuple(out.shape), -9, dtype=np.int64)
    choose(codes_f64(q), b, host, take, n_first, n_last, max_nodes, want)
    np.testing.assert_array_equal(out.cpu().numpy(), want)


def spoil(b, q, scores):
    if scores == "few":
        b.codes.clamp_(-1, 1)
        b.scale.fill_(127)
        return (q > 1).to(torch.bfloat16)
    if scores == "wide":
        b.scale.random_(27, 250)
        b.scale[::13] = 255
    return q


def test_the_definition_in_products():
    """choose() against the oracle's loops, through the same calls."""
    require_gpu()
    say("definition")
    plan, host, n_pages, n_rows = make_plan([90, 31, 0], [5, 2, 3], 3, seed=2)
    b = rand_bounds(n_pages, 2, 64, 3, 7)
    b.scale[::5] = 255
    q = rand_rows(n_rows, 6, 64, "bf16", 8)
    check_select(q, b, plan, host, 7, n_first=2, n_last=1)
    check(q, b, plan, host, 5, 7, 2, 1)


@pytest.mark.parametrize("scores", ["spread", "few", "wide"])
@pytest.mark.parametrize("dim,tile,nodes,heads,group,blocks", [
    (64, 16, 16, 8, 2, 2000), (64, 16, 9, 8, 5, 60), (64, 8, 8, 8, 4, 2290), (64, 8, 5, 16, 1, 300),
    (128, 16, 16, 8, 4, 900), (128, 16, 13, 8, 16, 1400), (128, 8, 8, 16, 1, 2290), (128, 8, 6, 8, 7, 65),
    (256, 16, 16, 8, 8, 1400), (256, 16, 11, 16, 1, 700), (256, 8, 8, 8, 3, 2290), (256, 8, 7, 8, 16, 900)])
def test_score_and_choice_in_one_launch(dim, tile, nodes, heads, group, blocks, scores):
    """At least 128 tiles; requests of fewer rows, and without any, among them."""
    require_gpu()
    say(f"one launch {dim} {tile} {heads} {group} {blocks} {scores}")
    rng = np.random.default_rng(dim + blocks)
    rows, start = [], []
    while (sum(rows) + 3) // tile * heads < 128:
        rows.append(int(rng.choice([nodes, nodes, nodes // 2 + 1, 0])))
        start.append(int(rng.integers(blocks // 3, blocks + 1)))
    rows[0], start[0], start[1] = nodes, blocks, 0
    rows += [nodes, nodes]
    start += [blocks, min(blocks, 70)]
    plan, host, n_pages, n_rows = make_plan(start, rows, 1, seed=3)
    b = rand_bounds(n_pages, heads, dim, 1, 5)
    q = spoil(b, rand_rows(n_rows, heads * group, dim, "bf16", 6), scores)
    fused = [f"select_fused_kernel<{dim}, {tile}>"]
    for take, n_first, n_last in ((blocks // 16 + 1, 1, 1), (blocks - 1, 3, 2)):
        check(q, b, plan, host, nodes, take, n_first, n_last, fused)
    check(q, b, plan, host, tile // 2 + 1, 5, 0, 1, fused)         # rows beyond max_nodes


@pytest.mark.parametrize("scores", ["spread", "few", "wide"])
@pytest.mark.parametrize("width,form", [(1152, "select_take_wave_kernel<18>"), (1153, "select_take_wave_kernel<36>"), (2304, "select_take_wave_kernel<36>"),
                                        (2305, "select_take_wave_kernel<68>"), (4352, "select_take_wave_kernel<68>"),
                                        (4353, "select_take_kernel<1024, 8>"), (8192, "select_take_kernel<1024, 8>"),
                                        (8193, "select_take_kernel<1024, 8>"), (20001, "select_take_kernel<1024, 8>")])
@pytest.mark.parametrize("nodes", [1, 3])
def test_score_and_choice_apart(width, form, nodes, scores):
    """A table of `width` pages: all of them, one less and few; beyond 8192 the
    keys do not stay in registers."""
    require_gpu()
    say(f"two launches {width} {nodes} {scores}")
    start, rows = [width - nodes, max(0, width - 64 * nodes), 200], [nodes, 1, nodes]
    plan, host, n_pages, n_rows = make_plan(start, rows, 1, seed=4)
    assert host[0].shape[1] == width
    if width % 2:                                        # blocks up to the table's end: the nodes have no page then
        start[0] = width
        host = (host[0], np.array(start, dtype=np.int32), host[2])
        plan = (plan[0], torch.tensor(start, dtype=torch.int32, device=DEV), plan[2])
    b = rand_bounds(n_pages, 2, 64, 1, 7)
    q = spoil(b, rand_rows(n_rows, 6, 64, "bf16", 8), scores)
    tile = 1 if nodes == 1 else 4
    for take, n_first, n_last in ((3, 0, 0), (700, 2, 3), (width - nodes - 1, 1, 1)):
        check(q, b, plan, host, nodes, take, n_first, n_last, [f"select_score_kernel<64, {tile}>", form])


@pytest.mark.parametrize("dim,group,tile", [(64, 20, 16), (128, 33, 4), (256, 64, 2), (256, 20, 4), (128, 64, 4)])
def test_tiles_of_many_heads(dim, group, tile):
    """Fewer rows to a tile where the group's operands would not fit LDS."""
    require_gpu()
    say(f"many heads {dim} {group}")
    plan, host, n_pages, n_rows = make_plan([500, 3, 300], [16, 0, 7], 1, seed=5)
    b = rand_bounds(n_pages, 2, dim, 1, 7)
    q = rand_rows(n_rows, 2 * group, dim, "bf16", 8)
    check(q, b, plan, host, 16, 40, 1, 1, [f"select_score_kernel<{dim}, {tile}>", "select_take_wave_kernel<18>"])
