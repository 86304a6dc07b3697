"""GPU tests of calls of the KV cache's operators at the ends of what they
allow: idle steps, kept workspaces, layouts and sizes beside the usual ones."""
import pytest
import torch

import block_draft_proposal_amd as D
from gpu_helpers import require_gpu, say
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
