"""CPU checks of the attention's workspace size: a server that keeps one
workspace for its largest tree passes it with smaller ones too."""
import pytest

from block_draft_proposal_amd import kv as K
from test_abi_kv import SCALED, _structs, _tree

KINDS = {"bf16": {}, "e4m3": SCALED, "i8": {**SCALED, "dtype": K.DFLASH_I8}}


def _sizes(cache, nodes, hq, n_req=2):
    ref = _structs(cache)[0]
    return [K._fns().dflash_tree_attention_workspace_size(ref, n_req, n, hq) for n in nodes]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kind", list(KINDS))
def test_the_size_never_falls_with_more_nodes_heads_or_requests(kind, dim):
    cache = dict(KINDS[kind], head_dim=dim, page_stride=8 * 16 * dim)
    nodes = list(range(1, 600)) + list(range(600, 4097, 13)) + [4096]
    by_group = []
    for group in (1, 2, 3, 4, 7, 8, 16, 64):
        sizes = _sizes(cache, nodes, 8 * group)
        assert min(sizes) > 0 and sizes == sorted(sizes), group
        by_group.append(sizes)
    for fewer, more in zip(by_group, by_group[1:]):
        assert all(a <= b for a, b in zip(fewer, more))
    assert _sizes(cache, [20], 32, 1) <= _sizes(cache, [20], 32, 5000)


def test_a_workspace_for_64_nodes_is_accepted_with_20():
    """Refused by its size before, the call now gets as far as the overlap that
    is put there on purpose: nothing is launched."""
    large, = _sizes({}, [64], 32)
    assert _tree(nodes=20, ws=1 << 40, ws_bytes=large) == -1
    assert _tree(nodes=64, ws=1 << 40, ws_bytes=large) == -1
    need, = _sizes({}, [4], 32)
    assert need > 0
    assert _tree(ws_bytes=need - 1) == -3 and _tree(ws=None) == -3 and _tree(ws=(10 << 40) + 16) == -1
