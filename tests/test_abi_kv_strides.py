"""CPU checks of tables and paths whose rows lie farther apart than offsets
can say: the products of request and stride must not pass 2^63."""
from block_draft_proposal_amd import binding as B
from test_abi_kv import _commit, _read, _tree, _write


def test_table_strides():
    for call in (_write, _read, _commit, _tree):
        for n_req, stride in ((2, 1 << 60), (3, (1 << 63) - 1), (1 << 20, 1 << 40)):
            assert call(batch=dict(n_req=n_req, table_stride=stride)) == -1, (n_req, stride)
            assert "page_table" in B.last_error()


def test_path_strides():
    for n_req, stride in ((2, 1 << 60), (3, (1 << 63) - 1), (1 << 20, 1 << 40)):
        assert _commit(batch=dict(n_req=n_req), stride=stride) == -1, (n_req, stride)
        assert "paths" in B.last_error()


def test_the_stride_of_a_single_row_is_any():
    """It is never used: the next refusal is reached."""
    one = dict(n_req=1, table_stride=(1 << 63) - 1)
    assert _write(batch=one, k=None) == -1 and "null k" in B.last_error()
    assert _commit(batch=one, stride=(1 << 63) - 1, paths=None) == -1 and "null pointer" in B.last_error()
    assert _tree(batch=one, q=None) == -1 and "null q" in B.last_error()
