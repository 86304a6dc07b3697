"""CPU test of how a call of the KV binding finds the current GPU: by torch's
public function, which also refuses a GPU that a forked process has inherited."""
import types

import pytest
import torch

from block_draft_proposal_amd import kv as K

CACHE = types.SimpleNamespace(device=torch.device("cuda:0"))
STREAM = types.SimpleNamespace(device=torch.device("cuda:0"), cuda_stream=7)


def test_a_call_on_the_current_gpu(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    got = []
    K._call(lambda *args: got.append(args), CACHE, STREAM, 1, 2)
    assert got == [(1, 2, 7)]


def test_torchs_refusal_reaches_the_caller(monkeypatch):
    def refuse():
        raise RuntimeError("Cannot re-initialize CUDA in forked subprocess")

    monkeypatch.setattr(torch.cuda, "current_device", refuse)
    with pytest.raises(RuntimeError, match="forked"):
        K._call(lambda *args: pytest.fail("called"), CACHE, STREAM)
