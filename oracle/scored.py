"""Float64 reference of attention whose scores are capped by a tanh, lowered
with distance or seen past the diagonal in a prefix (include/flash_attn_scored.h),
with element-wise bounds of what the roundings of 16-bit inputs and fp32
arithmetic may do to it."""
from __future__ import annotations

import numpy as np


def scores(q, k, scale, softcap, slope, rows, cols):
    """(u, t, s): scores of queries at places `rows` with keys at places `cols`."""
    s = scale * (q @ k.T)
    t = softcap * np.tanh(s / softcap) if softcap else s
    return t - slope * np.abs(rows[:, None] - cols[None, :]), t, s


def visible(n, causal, prefix):
    """Boolean [n, n] of a sequence's (query, key) pairs."""
    i, j = np.arange(n)[:, None], np.arange(n)[None, :]
    return (j <= i) | (j < prefix) if causal else np.ones((n, n), bool)


def softmax(u, seen):
    """(P, LSE) over the keys that are seen; a row that sees none has 0 and -inf."""
    u = np.where(seen, u, -np.inf)
    m = u.max(axis=1, initial=-np.inf)
    e = np.exp(u - np.where(np.isfinite(m), m, 0.0)[:, None])
    l = e.sum(axis=1)
    with np.errstate(divide="ignore"):
        return e / np.where(l > 0, l, 1.0)[:, None], np.where(l > 0, m + np.log(np.where(l > 0, l, 1.0)), -np.inf)


def score_error(q, k, scale, softcap, slope, rows, cols, u, t, LSE):
    """Bound of the error of u - LSE as fp32 forms it, per pair:
      (d + 4) 2^-24 scale sum|q||k|      sums of d products (the cap's slope is at most 1)
      2^-21 |t| + 2^-20 softcap          the cap's tanh
      2^-21 slope |i - j|                the slope's log2 e and the product with it
      2^-21 (|LSE| + |u|)                the arguments of the exponential"""
    d = q.shape[1]
    e = (d + 4) * 2.0 ** -24 * scale * (np.abs(q) @ np.abs(k).T)
    if softcap:
        e = np.minimum(e, 2 * softcap) + 2.0 ** -21 * np.abs(t) + 2.0 ** -20 * softcap
    e = e + 2.0 ** -21 * np.abs(slope) * np.abs(rows[:, None] - cols[None, :])
    return e + 2.0 ** -21 * (np.abs(np.where(np.isfinite(LSE), LSE, 0.0))[:, None] + np.abs(u))


def packed_attention(q, k, v, do, cu, scale, causal, u16, softcap=0.0, slopes=None, prefixes=None):
    """As oracle.packed.packed_attention (values and bounds of O, LSE, dQ, dK, dV;
    rows of no sequence are NaN), with these scores. u16: half a step of the
    16-bit type. A weight's relative error is that of its own score and the
    average of the others' (the sum it is divided by); dS has the cap's slope
    f = 1 - tanh^2, whose error is at most 0.77 of the score's over softcap plus
    2^-18 (two roundings of tanh, and of its square)."""
    q, k, v, do = (np.asarray(x, dtype=np.float64) for x in (q, k, v, do))
    T, Hq, d = q.shape
    Hk = k.shape[1]
    G = Hq // Hk
    z = 2.0 ** -126
    a = 2.0 ** -25 if u16 < 2.0 ** -9 else z
    f32 = 2.0 ** -20
    nan = np.nan
    val = dict(O=np.full((T, Hq, d), nan), LSE=np.full((Hq, T), nan), dQ=np.full((T, Hq, d), nan),
               dK=np.full((T, Hk, d), nan), dV=np.full((T, Hk, d), nan))
    tol = {n: np.zeros(x.shape) for n, x in val.items()}
    for b, (s, e) in enumerate(zip(cu[:-1], cu[1:])):
        n = e - s
        if n <= 0:
            continue
        seen = visible(n, causal, 0 if prefixes is None else min(max(int(prefixes[b]), 0), n))
        at = np.arange(n)
        r = slice(s, e)
        for name in ("dK", "dV"):
            val[name][r] = 0.0
        for h in range(Hq):
            hk = h // G
            slope = 0.0 if slopes is None else float(slopes[h])
            Q, K, V, dO = q[r, h], k[r, hk], v[r, hk], do[r, h]
            U, t, _ = scores(Q, K, scale, softcap, slope, at, at)
            P, LSE = softmax(U, seen)
            O = P @ V
            f = 1 - (t / softcap) ** 2 if softcap else np.ones_like(t)
            dP = dO @ V.T
            D = (dO * O).sum(axis=1, keepdims=True)
            dS = P * (dP - D) * f
            eU = np.where(seen, score_error(Q, K, scale, softcap, slope, at, at, U, t, LSE), 0.0)
            avg = (P * eU).sum(axis=1, keepdims=True)
            eP = np.expm1(eU + avg) + 2 * f32
            tO = P * (u16 + eP) @ np.abs(V) + a * n * np.abs(V).max() + u16 * np.abs(O) + a
            tD = (np.abs(dO) * tO).sum(axis=1, keepdims=True)
            dPm = 2.0 ** -24 * d * (np.abs(dO) @ np.abs(V).T)
            raw = (d + 4) * 2.0 ** -24 * scale * (np.abs(Q) @ np.abs(K).T)
            eF = 0.77 * raw / softcap + 2.0 ** -18 if softcap else 0.0
            tS = np.where(seen, (u16 + eP) * np.abs(dS) + P * f * (tD + dPm) + P * np.abs(dP - D) * eF + a
                          + z * np.abs(dP - D), 0.0)
            val["O"][r, h], val["LSE"][h, r] = O, LSE
            tol["O"][r, h], tol["LSE"][h, r] = tO, np.expm1(avg[:, 0]) + f32 + 2.0 ** -22 * np.abs(LSE)
            val["dQ"][r, h] = scale * (dS @ K)
            tol["dQ"][r, h] = scale * ((tS + f32 * np.abs(dS)) @ np.abs(K)) + u16 * np.abs(val["dQ"][r, h]) + a
            val["dK"][r, hk] += scale * (dS.T @ Q)
            tol["dK"][r, hk] += scale * ((tS + f32 * np.abs(dS)).T @ np.abs(Q))
            val["dV"][r, hk] += P.T @ dO
            tol["dV"][r, hk] += (P * (u16 + eP + f32)).T @ np.abs(dO) + a * (seen.T @ np.abs(dO))
        for name in ("dK", "dV"):
            tol[name][r] += u16 * np.abs(val[name][r]) + a
    return val, tol
