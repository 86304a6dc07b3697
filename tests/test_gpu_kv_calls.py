"""GPU tests of calls of the KV cache's operators at the ends of what they
allow: idle steps, kept workspaces, layouts and sizes beside the usual ones."""
import pytest
import torch

import block_draft_proposal_amd as D
from gpu_helpers import DEV, require_gpu, say
from test_gpu_tree_attention import build

pytestmark = pytest.mark.gpu


def test_an_idle_step_with_a_tree_mask():
    require_gpu()
    say("no rows, a mask of none")
    s = build("bf16", [50, 20], [4, 6], 16, 2, 4, 64, "tree", seed=13)
    kw = dict(s["kw"], mask=s["kw"]["mask"][:0])
    assert kw["mask"].shape[1] == 1
    assert D.dflash_tree_attention(s["q"][:0], s["cache"], **kw).shape == (0, 8, 64)
    with pytest.raises(ValueError, match="words"):
        D.dflash_tree_attention(s["q"], s["cache"], **dict(s["kw"], mask=s["kw"]["mask"][:, :0].contiguous()))
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("i8", 64), ("bf16", 256)])
def test_one_workspace_for_the_largest_tree_serves_every_smaller_one(kind, dim):
    require_gpu()
    say(f"kept workspace {kind} {dim}")
    s = build(kind, [300, 20], [64, 30], 16, 2, 4, dim, "tree", seed=14)
    size = D.tree_attention_workspace_size(s["cache"], n_req=2, max_nodes=64, n_q_heads=8)
    work = torch.empty(size, dtype=torch.uint8, device=DEV)
    off = s["kw"]["offsets"]
    for nodes in (64, 33, 20, 16, 9, 8, 1):
        kw = dict(s["kw"], max_nodes=nodes, offsets=torch.stack([off[0], off[0] + nodes, off[0] + nodes + min(nodes, 30)]))
        out = D.dflash_tree_attention(s["q"], s["cache"], workspace=work, **kw)
        want = D.dflash_tree_attention(s["q"], s["cache"], **kw)
        n = nodes + min(nodes, 30)
        assert torch.equal(out[:n], want[:n]), nodes
