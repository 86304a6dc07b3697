"""CPU checks of empty masks: a tensor without elements has a null address, as
no mask has, and the two must not be taken for each other."""
import types

import pytest
import torch

import block_draft_proposal_amd as D
from test_abi_kv import _tree


def test_an_idle_step_with_a_mask_of_no_rows_is_no_error():
    assert torch.empty((3, 2), dtype=torch.int64)[:0].data_ptr() == 0
    assert _tree(batch=dict(n_rows=0), mask=None, words=1) == 0
    assert _tree(batch=dict(n_req=0, page_table=None, start=None, offsets=None), mask=None, words=1) == 0
    assert _tree(mask=None, words=1) == -1              # with rows to do, words without a mask stay refused


@pytest.mark.parametrize("nodes,words", [(1, 0), (64, 0), (65, 1), (4096, 63)])
@pytest.mark.parametrize("rows", [0, 6])
def test_a_mask_of_too_few_words_is_refused(nodes, words, rows):
    """Not taken for a chain when it has no words at all."""
    cpu = torch.device("cpu")
    cache = types.SimpleNamespace(device=cpu, head_dim=64, n_kv_heads=1)
    kw = dict(page_table=torch.zeros((1, 4), dtype=torch.int32), start=torch.zeros(1, dtype=torch.int32),
              offsets=torch.zeros(2, dtype=torch.int32), max_nodes=nodes)
    q = torch.zeros((rows, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="words"):
        D.dflash_tree_attention(q, cache, mask=torch.zeros((rows, words), dtype=torch.int64), **kw)
