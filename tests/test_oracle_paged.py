"""Pins of the paged-cache oracle: hand-computed values, and agreement with the
dense attention oracle where the definitions meet."""

import numpy as np

import oracle
from oracle import paged


def test_slots_by_hand():
    pos, slot = paged.slots([0, 2, 2, 5], [18, 7, 2], [[4, 1], [0, 0], [9, 3]], 16, 7)
    assert pos.tolist() == [16, 17, 0, 0, 1, 0, 0]
    # the third sequence has three new tokens but two cached: its first has no place
    assert slot.tolist() == [16, 17, -1, 144, 145, -1, -1]


def test_rotation_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    cs = np.array([[0.0, 1.0, 1.0, 0.0]])        # pair 0: a quarter turn, pair 1: none
    assert paged.rotate(x, cs, False)[0, 0].tolist() == [-3.0, 2.0, 1.0, 4.0, 5.0]
    assert paged.rotate(x, cs, True)[0, 0].tolist() == [-2.0, 1.0, 3.0, 4.0, 5.0]


def test_head_norm_by_hand():
    y = paged.head_norm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.0)
    assert np.allclose(y, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]], atol=1e-15)


def test_attention_agrees_with_the_dense_oracle():
    rng = np.random.default_rng(0)
    n, kv, H, Hkv, d, page = 5, 21, 4, 2, 8, 8
    cache_k, cache_v = rng.normal(size=(2, 6, page, Hkv, d))
    row = [5, 0, 3]
    k, v = paged.gather(cache_k, row, page, kv), paged.gather(cache_v, row, page, kv)
    assert np.array_equal(k[17], cache_k[3, 1])
    q = rng.normal(size=(n, H, d))
    for causal in (False, True):
        o, lse, w, _ = paged.attention(q, k, v, 0.3, causal)
        o_ref, lse_ref = oracle.attention(q.transpose(1, 0, 2)[None], k.transpose(1, 0, 2)[None],
                                          v.transpose(1, 0, 2)[None], 0.3, causal)
        assert np.allclose(o, o_ref[0].transpose(1, 0, 2), atol=1e-13)
        assert np.allclose(lse, lse_ref[0].T, atol=1e-13)
        assert (w >= np.abs(o) - 1e-13).all()


def test_attention_rows_without_keys():
    o, lse, _, _ = paged.attention(np.ones((3, 1, 4)), np.ones((2, 1, 4)), np.ones((2, 1, 4)), 1.0,
                                   True)
    assert (o[0] == 0).all() and lse[0, 0] == -np.inf
    assert np.allclose(o[1:], 1.0)


def test_verify_by_hand():
    log = np.log
    target = np.array([log([0.5, 0.25, 0.25]), log([0.1, 0.8, 0.1]), log([0.2, 0.2, 0.6])])
    draft = np.array([log([0.25, 0.5, 0.25]), log([0.2, 0.2, 0.6])])
    one = np.ones(3)
    # position 0: token 0 has p > q: accepted whatever u; position 1: token 2 has
    # p / q = 1/6 < u: refused; the remainder is all on token 1
    out, n, _ = paged.verify(target, draft, [0, 2], [0.9, 0.5], one, 2, 1.0)
    assert out.tolist() == [0, 1, -1] and n == 1
    # both accepted (u below 1/6): one more token, the fastest of p / e
    out, n, _ = paged.verify(target, draft, [0, 2], [0.9, 0.1], np.array([0.1, 1.0, 1.0]), 2, 1.0)
    assert out.tolist() == [0, 2, 0] and n == 2
    # a draft with certainty: accepted with probability p(x); refused, x is out of the race
    out, n, _ = paged.verify(target, None, [0, 1], [0.6, 0.0], np.array([1e-9, 1.0, 0.5]), 2, 1.0)
    assert out.tolist() == [2, -1, -1] and n == 0
    # greedy
    out, n, _ = paged.verify(target, draft, [0, 1], [0.9, 0.9], one, 2, 0)
    assert out.tolist() == [0, 1, 2] and n == 2
    # no drafts at all
    out, n, _ = paged.verify(target, draft, [0, 2], [0.9, 0.5], one, 0, 1.0)
    assert out.tolist() == [0, -1, -1] and n == 0


def test_verify_emits_the_target_distribution():
    # one position: over many given random numbers, the emitted token (accepted
    # draft or redrawn one) follows p whatever q is
    rng = np.random.default_rng(3)
    p, q = np.array([0.6, 0.3, 0.1]), np.array([0.2, 0.3, 0.5])
    target, draft = np.log(np.stack([p, p])), np.log(q)[None]
    count = np.zeros(3)
    N = 4000
    for _ in range(N):
        x = rng.choice(3, p=q)
        out, _, _ = paged.verify(target, draft, [x], [rng.random()], rng.exponential(size=3), 1,
                                 1.0)
        count[out[0]] += 1
    # five standard deviations of a frequency over N draws
    assert (np.abs(count / N - p) < 5 * np.sqrt(p * (1 - p) / N)).all()
