"""Pins of the oracle of drafted trees, sampling with limits and cache pages:
values by hand, and agreement with other definitions where they meet."""

import numpy as np
import pytest

from oracle import paged, tree

#       0
#     1   2
#    3 4   5
#    6
PARENTS = [-1, 0, 0, 1, 1, 2, 3]


def test_mask_by_hand():
    m = tree.mask(PARENTS)
    assert [np.nonzero(r)[0].tolist() for r in m] == \
        [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 4], [0, 2, 5], [0, 1, 3, 6]]
    assert tree.depths(PARENTS).tolist() == [0, 1, 1, 2, 2, 2, 3]
    assert tree.words(m, 1)[:, 0].tolist() == [1, 3, 5, 11, 19, 37, 75]
    big = np.zeros((1, 130), bool)
    big[0, [0, 63, 64, 129]] = True
    assert tree.words(big, 3).tolist() == [[1 - (1 << 63), 1, 2]]


def test_mask_is_the_transitive_closure():
    rng = np.random.default_rng(0)
    parents = [-1] + [int(rng.integers(0, i)) for i in range(1, 40)]
    a = np.eye(40)
    for i, p in enumerate(parents):
        if p >= 0:
            a[i, p] = 1
    assert np.array_equal(np.linalg.matrix_power(a, 40) > 0, tree.mask(parents))


def test_a_chain_is_causal_attention():
    rng = np.random.default_rng(1)
    q, k, v = rng.normal(size=(4, 2, 8)), rng.normal(size=(9, 1, 8)), rng.normal(size=(9, 1, 8))
    seen = np.concatenate([np.ones((4, 5), bool), tree.mask([-1, 0, 1, 2])], 1)
    for x, y in zip(tree.attention(q, k, v, 0.4, seen), paged.attention(q, k, v, 0.4, True)):
        assert np.allclose(x, y, atol=1e-14)


def test_accept_by_hand():
    tok = [9, 10, 11, 12, 13, 14, 15]
    assert tree.accept(PARENTS, tok, [10, 12, 0, 15, 0, 0, 77]) == ([0, 1, 3, 6], [10, 12, 15, 77])
    assert tree.accept(PARENTS, tok, [11, 0, 14, 0, 0, 5, 0]) == ([0, 2, 5], [11, 14, 5])
    assert tree.accept(PARENTS, tok, [12, 0, 0, 0, 0, 0, 0]) == ([0], [12])   # no child's token
    assert tree.accept(PARENTS, [9, 8, 8, 7, 7, 7, 7], [8, 7, 7, 1, 1, 1, 1]) == ([0, 1, 3], [8, 7, 1])
    assert tree.accept([-1, 0], [-1, -1], [-1, 0]) == ([0], [-1])
    assert tree.accept([], [], []) == ([], [])


def test_limits_by_hand():
    x = np.log([0.1, 0.4, 0.2, 0.2, 0.1])
    assert tree.kept(x, 1.0)[0].tolist() == [1, 2, 3, 0, 4]
    assert tree.kept(x, 1.0, top_k=2)[0].tolist() == [1, 2]           # a tie: the lower index
    assert tree.kept(x, 1.0, top_p=0.5)[0].tolist() == [1, 2]
    assert tree.kept(x, 1.0, top_p=0.0)[0].tolist() == [1]
    assert tree.kept(x, 1.0, top_p=0.79)[0].tolist() == [1, 2, 3]
    assert tree.kept(x, 1.0, min_p=0.45)[0].tolist() == [1, 2, 3]
    assert tree.kept(x, 1.0, min_p=3.0)[0].tolist() == [1]
    # top_p of what top_k left: 0.4 of 0.6 is two thirds
    assert tree.kept(x, 1.0, top_k=2, top_p=0.66)[0].tolist() == [1]
    assert tree.kept(x, 1.0, top_k=2, top_p=0.67)[0].tolist() == [1, 2]
    assert tree.kept(x, 0.5, min_p=0.3)[0].tolist() == [1]            # weights 1/16, 1, 1/4


def test_draws_follow_the_distribution_that_is_left():
    rng = np.random.default_rng(2)
    x = rng.normal(size=12)
    idx, w, _ = tree.kept(x, 0.7, top_k=8, top_p=0.9)
    draws = [tree.sample(x, rng.exponential(size=12), 0.7, 8, 0.9)[:2] for _ in range(4000)]
    share = np.bincount([t for t, _ in draws], minlength=12) / 4000
    p = np.zeros(12)
    p[idx] = w / w.sum()
    assert np.abs(share - p).max() < 5 * np.sqrt(0.25 / 4000)
    assert all(np.isclose(lp, np.log(p[t])) for t, lp in draws)


@pytest.mark.parametrize("row", [[np.nan, 1.0], [np.inf, 0.0], [-np.inf, -np.inf]])
def test_rows_without_probabilities(row):
    assert tree.sample(row, [1.0, 1.0], 1.0)[0] == -1 and tree.sample(row, [1.0, 1.0], 0.0)[0] == -1


def test_compact_by_hand():
    cache = np.arange(24.0).reshape(6, 4, 1)     # six pages of four rows
    tree.compact(cache, [5, 0, 2], 4, [0, 2, 5, 6], 3)
    # positions 3, 5, 8, 9 to 3, 4, 5, 6
    assert cache[5, 3, 0] == 23 and cache[0, :, 0].tolist() == [1, 8, 9, 3]


def test_pages_by_hand():
    refs = [1, 1, 0, 1, 0, 0]
    table = [[3, 0, 0], [1, 0, 0]]
    out = [[0] * 3 for _ in range(3)]
    assert tree.fork(table, [6, 4], [0, 0, 1], out, refs, 4) == [6, 6, 4]
    assert out == [[3, 0, 0], [3, 0, 0], [1, 0, 0]] and refs == [3, 2, 0, 3, 0, 0]
    # page 0 holds tokens 4 and 5 of its three owners: the two that write get their own
    assert tree.grow(out, [6, 6, 4], [7, 7, 4], refs, 4) == ([0, 0, -1], [2, 4, -1], 1)
    assert out[:2] == [[3, 2, 0], [3, 4, 0]] and refs == [1, 2, 1, 3, 1, 0]
    assert tree.grow(out, [7, 7, 4], [9, 9, 5], refs, 4) == ([-1] * 3, [-1] * 3, -2)
    tree.release(table, [6, 4], refs, 4)
    assert refs == [0, 1, 1, 2, 1, 0]
    tree.release(out, [7, 7, 4], refs, 4, [4, 0, 4])
    assert refs == [0, 1, 0, 1, 0, 0]


def test_the_last_owner_keeps_its_page():
    refs, table = [2, 0, 0], [[0], [0]]
    assert tree.grow(table, [1, 1], [2, 2], refs, 4) == ([0, -1], [1, -1], 1)
    assert table == [[1], [0]] and refs == [1, 1, 0]
