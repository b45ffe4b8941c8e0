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


def packed_attention(q, k, v, do, cu, scale, causal, u16, softcap=0.0, slopes=None, prefixes=None, relative_slope=False):
    """As oracle.packed.packed_attention (values and bounds of O, LSE, dQ, dK, dV;
    rows of no sequence are NaN), with these scores. u16: half a step of the
    16-bit type. A weight's relative error is that of its own score and the
    average of the others' (the sum it is divided by); dS has the cap's slope
    f = 1 - tanh^2, whose error is at most 0.77 of the score's over softcap plus
    2^-18 (two roundings of tanh, and of its square). relative_slope: at most f times
      expm1(2 raw / softcap)     |d ln f / ds| = 2 |tanh| / softcap, raw the score's error
      2^-21 |s| / softcap        f goes with exp(-2 |s| / softcap), whose argument has
                                 two roundings (of the factor and of the product)
      2^-18                      the exponential, the reciprocal, four products,
    which holds where the cap is saturated, too."""
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
            U, t, raw_s = scores(Q, K, scale, softcap, slope, at, at)
            P, LSE = softmax(U, seen)
            O = P @ V
            f = 1 / np.cosh(np.clip(raw_s / softcap, -350, 350)) ** 2 if softcap else np.ones_like(t)
            dP = dO @ V.T
            D = (dO * O).sum(axis=1, keepdims=True)
            dS = P * (dP - D) * f
            eU = np.where(seen, score_error(Q, K, scale, softcap, slope, at, at, U, t, LSE), 0.0)
            avg = (P * eU).sum(axis=1, keepdims=True)
            eP = np.expm1(eU + avg) + 2 * f32
            tO = P * (u16 + eP) @ np.abs(V) + a * n * np.abs(V).max() + u16 * np.abs(O) + a
            dPm = 2.0 ** -24 * d * (np.abs(dO) @ np.abs(V).T)
            tD = (P * (eP * np.abs(dP) + dPm)).sum(axis=1, keepdims=True)   # D = rowsum(P dP) in fp32
            raw = (d + 4) * 2.0 ** -24 * scale * (np.abs(Q) @ np.abs(K).T)
            eF = 0.77 * raw / softcap + 2.0 ** -18 if softcap else 0.0
            if softcap and relative_slope:
                eF = f * (np.expm1(2 * raw / softcap) + 2.0 ** -21 * np.abs(raw_s) / softcap + 2.0 ** -18)
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


def _tokens(cache, table_row, n, hk):
    """Rows (or weights) of a sequence's n tokens for head hk; zeros where a page
    lies outside the cache."""
    page = cache.shape[2]
    out = np.zeros((n,) + cache.shape[3:])
    for j in range(n):
        p = int(table_row[j // page])
        if 0 <= p < cache.shape[0]:
            out[j] = cache[p, hk, j % page]
    return out


def cached_attention(q, k_cache, v_cache, block_table, seq_lens, scale, softcap=0.0, slopes=None, lse=None):
    """The newest tokens against caches of dequantised values. Returns values O
    [B, Nq, Hq, d] and LSE [B, Hq, Nq], the bounds of the weights' relative errors
    averaged over each row (like LSE) and sum_j P_j |V_j| and sum_j P_j e_j |V_j|
    (like O), e_j the bound of a weight's relative error. With lse [B, Hq, Nq] also W,
    a list of [Hk, n] arrays for the sequences: what each token received by that
    LSE, and its bounds."""
    q = np.asarray(q, dtype=np.float64)
    B, Nq, Hq, d = q.shape
    pages, Hk, page, _ = k_cache.shape
    G = Hq // Hk
    r = dict(O=np.zeros(q.shape), LSE=np.full((B, Hq, Nq), -np.inf), avg=np.zeros((B, Hq, Nq)), absv=np.zeros(q.shape),
             errv=np.zeros(q.shape), W=[], tolW=[])
    for b in range(B):
        n = min(max(int(seq_lens[b]), 0), block_table.shape[1] * page)
        at = np.arange(n)
        rows = np.arange(n - Nq, n)
        seen = at[None, :] <= rows[:, None]
        W, tolW = np.zeros((Hk, n)), np.zeros((Hk, n))
        for h in range(Hq if n else 0):
            hk = h // G
            ks, vs = _tokens(k_cache, block_table[b], n, hk), _tokens(v_cache, block_table[b], n, hk)
            slope = 0.0 if slopes is None else float(slopes[h])
            u, t, _ = scores(q[b, :, h], ks, scale, softcap, slope, rows, at)
            P, L = softmax(u, seen)
            r["LSE"][b, h], r["O"][b, :, h] = L, P @ vs
            e = np.where(seen, score_error(q[b, :, h], ks, scale, softcap, slope, rows, at, u, t, L), 0.0)
            r["avg"][b, h] = (P * e).sum(axis=1)
            rel = np.expm1(e + r["avg"][b, h][:, None]) + 2.0 ** -19
            r["absv"][b, :, h], r["errv"][b, :, h] = P @ np.abs(vs), (P * rel) @ np.abs(vs)
            if lse is not None:
                given = lse[b, h].astype(np.float64)
                live = seen & np.isfinite(given)[:, None]
                g = np.where(np.isfinite(given), given, 0.0)[:, None]
                w = np.where(live, np.exp(np.where(live, u - g, 0.0)), 0.0)
                ew = score_error(q[b, :, h], ks, scale, softcap, slope, rows, at, u, t, given)
                W[hk] += w.sum(axis=0)
                tolW[hk] += (w * np.where(live, np.expm1(ew) + 2.0 ** -20, 0.0)).sum(axis=0)
        r["W"].append(W)
        r["tolW"].append(tolW + (Nq * G + 2) * 2.0 ** -24 * W)
    return r


def evict(weights, block_table, seq_lens, budget, recent, page):
    """Former places [B][Hk] of the tokens that stay, ascending. weights: [pages,
    Hk, page]; those of pages outside the cache, negative ones and NaN count as 0."""
    out = []
    for b in range(len(seq_lens)):
        n = min(max(int(seq_lens[b]), 0), block_table.shape[1] * page)
        heads = []
        for hk in range(weights.shape[1]):
            tokens = list(range(n))
            if n > budget:
                w = _tokens(weights, block_table[b], n, hk)
                w = np.where(w > 0, w, 0.0)
                older = sorted(range(n - recent), key=lambda j: (-w[j], j))[:budget - recent]
                tokens = sorted(older) + list(range(n - recent, n))
            heads.append(tokens)
        out.append(heads)
    return out
