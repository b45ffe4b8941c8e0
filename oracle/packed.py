"""Float64 reference of attention over packed sequences with grouped heads, its
gradients, and element-wise bounds of what 16-bit roundings may do to them."""
from __future__ import annotations

import numpy as np

from . import attention as A


def _mask(n, causal):
    return np.tril(np.ones((n, n), bool)) if causal else np.ones((n, n), bool)


def packed_attention(q, k, v, do, cu, scale, causal, u):
    """q, do [T, Hq, d]; k, v [T, Hk, d]; cu: bounds of the sequences. u: half
    a step of the 16-bit type relative to the value (2^-8 bf16, 2^-11 fp16).

    Returns (values, bounds), dicts of O, LSE, dQ, dK, dV; rows of no sequence
    are NaN in values (and have no bound). The bounds, per element:
      score    eS  = (d + 4) 2^-24 scale sum|q||k|        fp32 sums of d products
      weight   eP  = 2 (max_j eS + 2^-20) + 2^-21 (|LSE| + max|S|), relative
               (exponential, sums, LSE * log2 e), plus a = 2^-25 for fp16, the
               half step of its smallest numbers, or z = 2^-126, under which
               the exponential's results are flushed to zero
      O        (u + eP) sum P|V| + a n max|V| + u |O| + a     P and O rounded once
      dV       (u + eP) sum P|dO| + a sum|dO| + u |dV| + a
      D        sum_c |dO| bound(O)                        D is formed from rounded O
      dS       (u + eP) |dS| + P (bound(D) + 2^-24 d sum|dO||V|) + a + z |dP - D|
      dQ, dK   scale sum bound(dS) |K| (|Q|) + (u + 2^-20) of the sums' magnitudes + a
    The a of each output is its own rounding: fp16 numbers under 2^-14 are
    multiples of 2^-24, so rounding one is off by up to 2^-25 = a whatever its
    size, and u |x| alone (less than a there) does not cover it.
    """
    q, k, v, do = (np.asarray(x, dtype=np.float64) for x in (q, k, v, do))
    T, Hq, d = q.shape
    Hk = k.shape[1]
    G = Hq // Hk
    z = 2.0 ** -126
    a = 2.0 ** -25 if u < 2.0 ** -9 else z
    f32 = 2.0 ** -20
    nan = np.nan
    val = dict(O=np.full((T, Hq, d), nan), LSE=np.full((Hq, T), nan), dQ=np.full((T, Hq, d), nan),
               dK=np.full((T, Hk, d), nan), dV=np.full((T, Hk, d), nan))
    tol = {n: np.zeros(x.shape) for n, x in val.items()}
    for s, e in zip(cu[:-1], cu[1:]):
        n = e - s
        if n <= 0:
            continue
        allowed = _mask(n, causal)
        r = slice(s, e)
        for name in ("dK", "dV"):
            val[name][r] = 0.0
        for h in range(Hq):
            hk = h // G
            Q, K, V, dO = q[r, h], k[r, hk], v[r, hk], do[r, h]
            f = A.head_forward(Q, K, V, scale, allowed)
            P, O, LSE, S = f["P"], f["O"], f["LSE"], np.where(allowed, f["S"], 0.0)
            g = A.head_backward(Q, K, V, dO, scale, P, O)
            eS = (d + 4) * 2.0 ** -24 * scale * np.where(allowed, np.abs(Q) @ np.abs(K).T, 0.0).max(axis=1)
            eP = 2 * (eS + f32) + 2.0 ** -21 * (np.abs(LSE) + np.abs(S).max(axis=1))
            eP = eP[:, None]
            tO = ((u + eP) * (P @ np.abs(V)) + a * n * np.abs(V).max() + u * np.abs(O) + a)
            tD = (np.abs(dO) * tO).sum(axis=1, keepdims=True)
            dPm = 2.0 ** -24 * d * (np.abs(dO) @ np.abs(V).T)
            tS = np.where(allowed, (u + eP) * np.abs(g["dS"]) + P * (tD + dPm) + a + z * np.abs(g["dP"] - g["D"][:, None]), 0.0)
            val["O"][r, h], val["LSE"][h, r] = O, LSE
            tol["O"][r, h], tol["LSE"][h, r] = tO, eS + f32 + 2.0 ** -22 * np.abs(LSE)
            val["dQ"][r, h] = g["dQ"]
            tol["dQ"][r, h] = scale * ((tS + f32 * np.abs(g["dS"])) @ np.abs(K)) + u * np.abs(g["dQ"]) + a
            val["dK"][r, hk] += g["dK"]
            tol["dK"][r, hk] += scale * ((tS + f32 * np.abs(g["dS"])).T @ np.abs(Q))
            val["dV"][r, hk] += g["dV"]
            tol["dV"][r, hk] += ((u + eP + f32) * P).T @ np.abs(dO) + a * (allowed.T @ np.abs(dO))
        for name in ("dK", "dV"):
            tol[name][r] += u * np.abs(val[name][r]) + a
    return val, tol
