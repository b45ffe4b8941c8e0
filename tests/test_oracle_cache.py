"""The float64 reference of the paged cache against values worked by hand and
against the types' own conversions."""
import math

import numpy as np
import torch

from oracle import attention as A
from oracle import cache as C


def test_e4m3_rounding_matches_the_type_on_every_midpoint():
    vals = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()   # 0 .. 448
    assert vals[-1] == 448.0 and vals[1] == 2.0 ** -9
    mid = (vals[:-1] + vals[1:]) / 2
    x = np.concatenate([vals, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9)])
    x = np.concatenate([x, -x])
    got = C.e4m3_round(x)
    assert set(np.abs(got)) <= set(vals)
    lo = vals[np.searchsorted(vals, np.abs(x), side="right") - 1]
    hi = vals[np.minimum(np.searchsorted(vals, np.abs(x), side="left"), len(vals) - 1)]
    assert (np.abs(np.abs(got) - np.abs(x)) <= np.minimum(np.abs(x) - lo, hi - np.abs(x)) + 0).all()
    # halfway: the even code
    code = {v: i for i, v in enumerate(vals)}
    assert all(code[abs(v)] % 2 == 0 for v in C.e4m3_round(mid))


def test_scales_are_the_smallest_power_of_two():
    x = np.array([[448.0, 1.0], [449.0, 0.0], [0.0, 0.0], [7.0, -7.0], [np.inf, 3.0], [1e-30, 0.0]])
    y, s = C.e4m3_rows(x)
    assert list(s) == [1.0, 2.0, 2.0 ** -64, 2.0 ** -6, 2.0 ** -7, 2.0 ** -64]
    assert y[0, 0] == 448.0 and y[3, 0] == 448.0 and np.isnan(y[4, 0]) and y[4, 1] == 384.0 and y[5, 0] == 0.0


def test_cached_attention_is_the_last_rows_of_attention():
    rng = np.random.default_rng(0)
    n, d, page, Nq = 21, 8, 16, 3
    k, v, q = rng.standard_normal((3, n, d))
    kc, vc = np.full((4, 1, page, d), np.nan), np.full((4, 1, page, d), np.nan)
    table = np.array([[2, 0]])
    for j in range(n):
        kc[table[0, j // page], 0, j % page] = k[j]
        vc[table[0, j // page], 0, j % page] = v[j]
    o, lse, absv, _ = C.cached_attention(q[None, -Nq:, None], kc, vc, table, [n], 0.3)
    ref = A.head_forward(q, k, v, 0.3, np.tril(np.ones((n, n), bool)))
    assert np.allclose(o[0, :, 0], ref["O"][-Nq:], atol=1e-12)
    assert np.allclose(lse[0, 0], ref["LSE"][-Nq:], atol=1e-12)
    assert (absv >= np.abs(o) - 1e-15).all()
    o, lse, _, _ = C.cached_attention(q[None, -Nq:, None], kc, vc, table, [2], 0.3)
    assert (o[0, 0] == 0).all() and lse[0, 0, 0] == -math.inf     # two keys, three tokens
