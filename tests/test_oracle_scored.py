"""Pins of the float64 reference of capped and biased scores: closed forms, the
plain reference where the scores are plain, and gradients against differences."""
import numpy as np
import pytest

from oracle import scored as S
from oracle.packed import packed_attention


def _inputs(lens, Hq, Hk, d, seed=0):
    r = np.random.default_rng(seed)
    T = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    return [r.standard_normal((T, h, d)) for h in (Hq, Hk, Hk, Hq)] + [cu]


def test_plain_scores_are_the_plain_reference():
    q, k, v, do, cu = _inputs([5, 0, 9], 4, 2, 8)
    for causal in (True, False):
        a, _ = packed_attention(q, k, v, do, cu, 0.3, causal, 2.0 ** -8)
        b, _ = S.packed_attention(q, k, v, do, cu, 0.3, causal, 2.0 ** -8)
        for n in a:
            np.testing.assert_allclose(a[n], b[n], rtol=1e-12, atol=1e-12)


def test_a_prefix_of_everything_is_not_causal():
    q, k, v, do, cu = _inputs([7, 4], 2, 1, 8, 1)
    kw = dict(softcap=2.0, slopes=[0.3, 0.1])
    a, _ = S.packed_attention(q, k, v, do, cu, 0.5, True, 2.0 ** -8, prefixes=[7, 99], **kw)
    b, _ = S.packed_attention(q, k, v, do, cu, 0.5, False, 2.0 ** -8, **kw)
    c, _ = S.packed_attention(q, k, v, do, cu, 0.5, True, 2.0 ** -8, prefixes=[1, -3], **kw)
    e, _ = S.packed_attention(q, k, v, do, cu, 0.5, True, 2.0 ** -8, **kw)
    for n in a:
        np.testing.assert_array_equal(a[n], b[n])
        np.testing.assert_array_equal(c[n], e[n])      # (the first key is always seen)


def test_closed_forms():
    # keys of no score: weights 2^-(distance) with a slope of ln 2
    u, t, s = S.scores(np.zeros((4, 8)), np.zeros((4, 8)), 1.0, 5.0, np.log(2.0), np.arange(4), np.arange(4))
    P, LSE = S.softmax(u, S.visible(4, True, 0))
    np.testing.assert_allclose(P[3], np.array([1, 2, 4, 8]) / 15.0)
    np.testing.assert_allclose(LSE[3], np.log(15.0 / 8.0))
    # scores past all bounds: the cap
    u, t, s = S.scores(np.full((1, 8), 1e6), np.array([[1.0] * 8, [-1.0] * 8]), 1.0, 3.0, 0.0, np.arange(1), np.arange(2))
    np.testing.assert_allclose(u, [[3.0, -3.0]])


@pytest.mark.parametrize("softcap", [0.0, 0.7, 4.0])
@pytest.mark.parametrize("prefixes", [None, [3, 5]])
def test_gradients_against_differences(softcap, prefixes):
    q, k, v, do, cu = _inputs([6, 5], 2, 1, 4, 3)
    kw = dict(softcap=softcap, slopes=[0.5, 0.05], prefixes=prefixes)
    loss = lambda q, k, v: (S.packed_attention(q, k, v, do, cu, 0.6, True, 2.0 ** -8, **kw)[0]["O"] * do).sum()
    val, _ = S.packed_attention(q, k, v, do, cu, 0.6, True, 2.0 ** -8, **kw)
    h = 1e-5
    for name, x, at in (("dQ", q, 0), ("dK", k, 1), ("dV", v, 2)):
        for i in np.ndindex(x.shape):
            args = [[q, k, v], [q, k, v]]
            for sgn, a in zip((h, -h), args):
                a[at] = x.copy()
                a[at][i] += sgn
            # (third-order terms of a central difference of h = 1e-5, and roundings over 2 h)
            assert abs((loss(*args[0]) - loss(*args[1])) / (2 * h) - val[name][i]) < 1e-7, (name, i)
