"""The packed reference's gradients against differences of its own output."""
import numpy as np
import pytest

from oracle.packed import packed_attention


@pytest.mark.parametrize("causal", [False, True])
def test_gradients_against_differences(causal):
    rng = np.random.default_rng(3)
    cu, Hq, Hk, d, scale = [1, 6, 6, 10], 4, 2, 3, 0.6
    q, do = rng.standard_normal((2, 11, Hq, d))
    k, v = rng.standard_normal((2, 11, Hk, d))
    f = lambda q, k, v: np.nansum(packed_attention(q, k, v, do, cu, scale, causal, 0.0)[0]["O"] * do)
    val, _ = packed_attention(q, k, v, do, cu, scale, causal, 0.0)
    h = 1e-5
    for name, x in (("dQ", q), ("dK", k), ("dV", v)):
        for _ in range(12):
            i = tuple(rng.integers(n) for n in x.shape)
            old = x[i]
            x[i] = old + h
            up = f(q, k, v)
            x[i] = old - h
            down = f(q, k, v)
            x[i] = old
            want = (up - down) / (2 * h)
            got = val[name][i]
            if not cu[0] <= i[0] < cu[-1]:
                assert np.isnan(got) and want == 0.0
            else:
                assert abs(got - want) <= 1e-8, (name, i)


def test_sequences_do_not_see_each_other():
    rng = np.random.default_rng(4)
    q, do = rng.standard_normal((2, 9, 2, 4))
    k, v = rng.standard_normal((2, 9, 1, 4))
    both, _ = packed_attention(q, k, v, do, [0, 5, 9], 0.5, True, 0.0)
    one, _ = packed_attention(q[5:], k[5:], v[5:], do[5:], [0, 4], 0.5, True, 0.0)
    for name in ("O", "dQ", "dK", "dV"):
        assert np.allclose(both[name][5:], one[name], atol=1e-13)
    assert np.allclose(both["LSE"][:, 5:], one["LSE"], atol=1e-13)
