"""CPU pins of the KV cache oracle: the 8-bit formats against torch's own
casts, scales against their definition, attention against torch's softmax."""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as O


def test_e4m3_rounding_matches_the_type():
    torch.manual_seed(0)
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64)
    every = every[every.isfinite()].sort().values
    mids = (every[1:] + every[:-1]) / 2                       # exact ties
    x = torch.cat([every, mids, (torch.rand(4000, dtype=torch.float64) - 0.5) * 896, torch.randn(4000, dtype=torch.float64) * 0.01])
    x = x.to(torch.float32)
    want = x.to(torch.float8_e4m3fn).to(torch.float64).numpy()
    np.testing.assert_array_equal(O.nearest_code(x.double().numpy(), "e4m3"), want)


def test_int8_rounding_ties_to_even():
    np.testing.assert_array_equal(O.nearest_code(np.array([0.5, 1.5, -0.5, -2.5, 126.5]), "i8"), [0, 2, -0.0, -2, 126])


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_scale_is_the_smallest_power_of_two_that_fits(kind):
    top = O.TOP[kind]
    amax = np.array([top, top * 1.001, top / 2, 1.0, 1e-30, 0.0, 2.0 ** -140, 3.0e38])
    codes, b = O.quantise_rows(amax[:, None], kind)
    e = b.astype(int) - 127
    for a, x in zip(amax, e):
        assert a * 2.0 ** -float(x) <= top
        assert x == O.MIN_EXP or a * 2.0 ** -float(x - 1) > top
    codes, b = O.quantise_rows(np.array([[1.0, np.nan], [np.inf, 0.0]]), kind)
    assert (b == 255).all() and (codes == 0).all() and np.isnan(O.scale_value(b)).all()


def test_attention_is_softmax_over_what_a_node_sees():
    rng = np.random.default_rng(1)
    cache = dict(k=rng.standard_normal((3, 2, 4, 8)), v=rng.standard_normal((3, 2, 4, 8)), k_scale=None, v_scale=None)
    table, start, offsets = np.array([[2, 0]]), np.array([5]), np.array([0, 3])
    q = rng.standard_normal((4, 4, 8))
    mask = np.array([[1], [0], [5], [0]], dtype=np.uint64)
    out = np.full((4, 4, 8), 7.0)
    O.tree_attention(q, cache, table, start, offsets, mask, 0.3, out)
    k = torch.tensor(np.concatenate([cache["k"][2], cache["k"][0]], axis=1))       # [heads, 8, dim]
    v = torch.tensor(np.concatenate([cache["v"][2], cache["v"][0]], axis=1))
    for i, extra in enumerate(([0], [], [0, 2])):
        seen = list(range(5)) + [5 + j for j in extra]
        for h in range(4):
            w = torch.softmax(0.3 * (k[h // 2, seen] @ torch.tensor(q[i, h])), 0)
            np.testing.assert_allclose(out[i, h], (w @ v[h // 2, seen]).numpy(), rtol=1e-12, atol=1e-12)
    assert (out[3] == 7.0).all()


def test_a_node_that_sees_nothing_is_zero_and_unseen_values_do_not_matter():
    cache = dict(k=np.full((1, 1, 4, 2), np.nan), v=np.full((1, 1, 4, 2), np.inf), k_scale=None, v_scale=None)
    cache["k"][0, 0, 1], cache["v"][0, 0, 1] = 1.0, 2.0
    out = np.full((2, 1, 2), 9.0)
    O.tree_attention(np.ones((2, 1, 2)), cache, np.array([[0]]), np.array([0]), np.array([0, 2]),
                     np.array([[0], [2]], dtype=np.uint64), 1.0, out)
    np.testing.assert_array_equal(out, [[[0, 0]], [[2, 2]]])


def test_commit_moves_the_path_behind_the_prefix():
    k = np.arange(8.0).reshape(2, 1, 4, 1)
    cache = dict(k=k.copy(), v=-k, k_scale=None, v_scale=None)
    O.commit(cache, np.array([[1, 0]]), np.array([1]), np.array([[0, 2, 5]]), np.array([3]))
    # positions 0..7 held 4 5 6 7 0 1 2 3; nodes 0, 2, 5 are positions 1, 3, 6
    assert [cache["k"][p, 0, s, 0] for p, s in ((1, 0), (1, 1), (1, 2), (1, 3), (0, 0))] == [4, 5, 7, 2, 0]
