"""Pins of the oracle's tree and block functions (CPU)."""

import math

import numpy as np
import pytest

from oracle import mla_oracle as O


def test_tree_masks_and_depths_of_a_known_tree():
    parents = [-1, 0, 0, 1, -1, 3]
    assert O.tree_bits(parents) == [0b1, 0b11, 0b101, 0b1011, 0b10000, 0b101011]
    assert O.tree_depths(parents) == [0, 1, 1, 2, 0, 3]


@pytest.mark.parametrize("seed", range(3))
def test_a_chain_is_decoding_token_by_token(seed):
    rng = np.random.default_rng(seed)
    T, n, h, D, d_c = 5, 7, 3, 10, 6
    rows, q = rng.standard_normal((n + T, D)), rng.standard_normal((T, h, D))
    bits = O.tree_bits(range(-1, T - 1))
    out, lse = O.tree_attention(q, rows[:n], rows[n:], bits, d_c=d_c, scale=0.3)
    for t in range(T):
        want, z = O.latent_attention(q[t], rows[:n + t + 1], d_c=d_c, scale=0.3)
        assert np.allclose(out[t], want, rtol=1e-13) and np.allclose(lse[t], z, rtol=1e-13)


def test_each_branch_alone_gives_the_tree():
    """Token t's result is that of its own branch appended to the sequence."""
    rng = np.random.default_rng(1)
    n, h, D, d_c = 4, 2, 8, 5
    parents = [-1, 0, 0, 2, 1, -1]
    bits = O.tree_bits(parents)
    rows, q = rng.standard_normal((n + 6, D)), rng.standard_normal((6, h, D))
    out, lse = O.tree_attention(q, rows[:n], rows[n:], bits, d_c=d_c, scale=0.5)
    for t in range(6):
        branch, at = [], t
        while at >= 0:
            branch.insert(0, at)
            at = parents[at]
        kept = O.tree_accept(rows, n, branch)[:n + len(branch)]
        want, z = O.latent_attention(q[t], kept, d_c=d_c, scale=0.5)
        assert np.allclose(out[t], want) and np.allclose(lse[t], z)


def test_a_token_that_attends_nothing():
    out, lse = O.tree_attention(np.ones((1, 2, 4)), np.zeros((0, 4)), np.ones((1, 4)), [0], d_c=3, scale=1.0)
    assert (out == 0).all() and np.isneginf(lse).all()


def test_accepting_everything_or_nothing_changes_nothing():
    rows = np.arange(12.0).reshape(6, 2)
    assert np.array_equal(O.tree_accept(rows, 2, [0, 1, 2, 3]), rows)
    assert np.array_equal(O.tree_accept(rows, 2, []), rows)
    assert np.array_equal(O.tree_accept(rows, 2, [1, 3])[:, 0], [0, 2, 6, 10, 8, 10])


def test_block_means_of_ragged_length():
    rows = np.arange(70.0)[:, None] * np.ones((1, 3))
    assert np.allclose(O.block_means(rows), [[31.5] * 3, [66.5] * 3])
    assert O.block_means(np.zeros((0, 3))).shape == (0, 3)


def test_scores_are_exact_shares_where_blocks_are_constant():
    """With every token of a block equal to its mean the score is the
    attention the block draws, summed over heads."""
    rng = np.random.default_rng(0)
    n, h, D = 150, 4, 6
    means = rng.standard_normal((3, D))
    rows = means[np.arange(n) // 64]
    q = rng.standard_normal((h, D))
    got = O.block_scores(q, O.block_means(rows), n, scale=0.7)
    s = q @ rows.T * 0.7
    p = np.exp(s) / np.exp(s).sum(1, keepdims=True)
    want = [p[:, a:b].sum() for a, b in O.block_ranges(n)]
    assert np.allclose(got, want) and math.isclose(got.sum(), h)


def test_selection_order():
    nan = math.nan
    assert O.block_select([1.0, 3.0, 3.0, 2.0], 2, 0, 0) == [1, 2]
    assert O.block_select([3.0, 3.0, 3.0, 2.0], 2, 0, 0) == [0, 1]
    assert O.block_select([0.0, -0.0, 0.0], 1, 0, 0) == [0]
    assert O.block_select([1.0, 9.0, 9.0, 0.0], 3, 1, 1) == [0, 1, 3]
    assert O.block_select([nan, -math.inf, nan], 2, 0, 0) == [0, 1]
    assert O.block_select([math.inf, 1.0, 2.0], 1, 0, 1) == [2]
    assert O.block_select([nan, 9.0, 1.0], 1, 2, 0) == [0]
    assert O.block_select([5.0], 4, 0, 0) == [0]
    assert O.block_select([], 4, 1, 1) == []
