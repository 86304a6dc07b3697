"""CPU checks of outputs and workspaces that lie over the batch's own arrays or
the mask.  The attention's workgroups each work out the whole batch's plan from
start and offsets: if one changes them while another still reads, the plans
differ, and with them the places of the workspace that the join reads."""
from block_draft_proposal_amd import binding as B
from block_draft_proposal_amd import kv as K
from test_abi_kv import BATCH, _read, _structs, _tree

N = BATCH["n_req"]
ENDS = {"page_table": ((N - 1) * BATCH["table_stride"] + BATCH["table_width"]) * 4, "start": N * 4, "offsets": (N + 1) * 4}
MASK = 11 << 40                                         # uint64 [8, 1]


def _over(bytes_before, at):
    """16-byte aligned places around an array: the last before it that a span
    of so many bytes reaches it from, and the first inside."""
    return at - bytes_before + 16, at


def test_workspace_and_output_of_the_attention():
    need = K._fns().dflash_tree_attention_workspace_size(_structs()[0], N, 4, 32)
    out = 8 * 32 * 128 * 2
    for name in ENDS:
        for p in (BATCH[name], BATCH[name] - (need - 1) // 256 * 256):
            assert _tree(ws=p, ws_bytes=1 << 60) == -1 and "batch" in B.last_error(), name
        for p in _over(out, BATCH[name]):
            assert _tree(out=p) == -1 and "batch" in B.last_error(), name
    for p in (MASK, MASK - (need - 1) // 256 * 256):
        assert _tree(mask=MASK, words=1, ws=p) == -1 and "mask" in B.last_error()
    for p in _over(out, MASK):
        assert _tree(mask=MASK, words=1, out=p) == -1 and "mask" in B.last_error()


def test_outputs_of_the_read():
    size = 8 * 8 * 128 * 2
    for name in ENDS:
        for p in _over(size, BATCH[name]):
            for which in "kv":
                assert _read(**{which: p}) == -1 and "batch" in B.last_error(), name


def test_right_beside_is_allowed():
    """The next refusal is reached: the output's last byte is the one before
    the array, or its first the one behind (aligned up)."""
    out = 8 * 32 * 128 * 2
    for name, size in ENDS.items():
        for p in (BATCH[name] - out, BATCH[name] + -(-size // 16) * 16):
            assert _tree(out=p, ws=None) == -3, name
    for p in (MASK - out, MASK + 8 * 8):
        assert _tree(mask=MASK, words=1, out=p, ws=None) == -3
