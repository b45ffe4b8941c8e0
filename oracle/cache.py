"""Float64 reference of serving from a paged key/value cache: the quantisation
of the writer and attention of the newest tokens, written from the definitions
in include/flash_attn_cache.h with NumPy."""
from __future__ import annotations

import math

import numpy as np

E4M3_MAX = 448.0
MIN_EXP = -64


def e4m3_round(y):
    """Nearest e4m3 value (ties to even) of float64 y with |y| <= 448: three
    bits behind the leading one, steps of 2^-9 below 2^-6."""
    y = np.asarray(y, dtype=np.float64)
    _, e = np.frexp(np.maximum(np.abs(y), 2.0 ** -6))     # |y| in [2^(e-1), 2^e)
    step = np.ldexp(1.0, e - 4)
    return np.rint(y / step) * step                       # rint: half to even


def e4m3_rows(x):
    """(payload, scale) of rows x [..., d]: scale the smallest power of two
    >= 2^-64 with max |x| <= 448 scale over the finite elements; infinities and
    NaN become NaN."""
    x = np.asarray(x, dtype=np.float64)
    fin = np.isfinite(x)
    top = np.where(fin, np.abs(x), 0.0).max(axis=-1)
    scale = np.full(top.shape, np.nan)
    for e in range(130, MIN_EXP - 1, -1):                 # the last that holds is the smallest
        scale[top <= E4M3_MAX * 2.0 ** e] = 2.0 ** e
    y = e4m3_round(np.where(fin, x, 0.0) / scale[..., None])
    return np.where(fin, y, np.nan), scale


def cached_attention(q, k_cache, v_cache, block_table, seq_lens, scale):
    """O [B, Nq, Hq, d], LSE [B, Hq, Nq] in float64 from caches of dequantised
    values [pages, Hk, page, d], plus what error bounds need: sum_j P_j |V_j|
    (like O) and max_j scale sum_c |q_c k_jc| (like LSE). Pages outside the
    cache read as zeros."""
    q = np.asarray(q, dtype=np.float64)
    B, Nq, Hq, d = q.shape
    pages, Hk, page, _ = k_cache.shape
    G = Hq // Hk
    o, absv = np.zeros(q.shape), np.zeros(q.shape)
    lse, mag = np.full((B, Hq, Nq), -math.inf), np.zeros((B, Hq, Nq))
    for b in range(B):
        n = min(max(int(seq_lens[b]), 0), block_table.shape[1] * page)
        for hk in range(Hk):
            ks, vs = np.zeros((n, d)), np.zeros((n, d))
            for j in range(n):
                p = int(block_table[b, j // page])
                if 0 <= p < pages:
                    ks[j], vs[j] = k_cache[p, hk, j % page], v_cache[p, hk, j % page]
            for h in range(hk * G, (hk + 1) * G):
                for i in range(Nq):
                    m = max(0, n - (Nq - 1 - i))
                    if m == 0:
                        continue
                    s = scale * (ks[:m] @ q[b, i, h])
                    top = s.max()
                    w = np.exp(s - top)
                    lse[b, h, i] = top + math.log(w.sum())
                    w /= w.sum()
                    o[b, i, h] = w @ vs[:m]
                    absv[b, i, h] = w @ np.abs(vs[:m])
                    mag[b, h, i] = scale * (np.abs(ks[:m]) @ np.abs(q[b, i, h])).max()
    return o, lse, absv, mag
