"""Oracle of the 4-bit KV cache: what it keeps of a row, and the attention of
the newest tokens over it (TEST INFRASTRUCTURE ONLY, float64, like
:mod:`oracle.sambay_ref`).

A row of dh values is kept in blocks of 16:  x ~ 2^e * s * c  with
s = e4m3(min(448, max|x| 2^-e / 6)) and c = e2m1(|x| 2^-e / s) and x's sign,
both roundings to the nearest value and, half way, to the one whose code is
even.  A block that holds a NaN or an infinity is kept as NaN.
"""

from __future__ import annotations

import numpy as np

#: The values of the 4-bit code without its sign, and of the 8-bit scale's 127 finite codes (3 bits of mantissa, bias 7).
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)])[:127]


def nearest_code(x, values):
    """Index of the nearest of `values` (rising) to each x >= 0; half way, the even index; past the last, the last."""
    x = np.asarray(x, dtype=np.float64)
    mid = 0.5 * (values[1:] + values[:-1])
    code = np.searchsorted(mid, x, side="left")          # on a border: the lower code
    on = (code < len(mid)) & (mid[np.minimum(code, len(mid) - 1)] == x)
    return code + (on & (code % 2 == 1))


def kv4_kept(x, e=None):
    """x [..., Hkv, dh] as the cache keeps it, float64; e [Hkv] the heads' exponents (0)."""
    x = np.asarray(x, dtype=np.float64)
    two = np.ones(x.shape[-2]) if e is None else 2.0 ** np.asarray(e, dtype=np.float64)
    blocks = (x / two[:, None]).reshape(*x.shape[:-1], -1, 16)
    bad = ~np.isfinite(blocks).all(-1, keepdims=True)
    a = np.where(bad, 0.0, np.abs(blocks))
    s = E4M3[nearest_code(a.max(-1, keepdims=True) / 6.0, E4M3)]
    c = E2M1[nearest_code(a / np.where(s > 0, s, 1.0), E2M1)]
    kept = np.where(bad, np.nan, np.sign(np.where(bad, 0.0, blocks)) * c * s)
    return kept.reshape(x.shape) * two[:, None]


def kv4_attention_ref(q, K, V, lens, count=None, scale=None):
    """q [B, T, Hq, dh]; K, V [B, N, Hkv, dh] as kept.  Query t of the n =
    count[b] (T) newest tokens of sequence b sees the first lens[b] - (n - 1 - t)
    tokens; none: 0.  Rows from count[b] on: NaN (not computed).

    Returns (out, spread, logit): spread = sum_j p_j |v_j| (the size of the sum
    that out is, for error bounds) and logit = scale max_j sum_d |q_d k_jd| per row.
    """
    q, K, V = (np.asarray(a, dtype=np.float64) for a in (q, K, V))
    B, T, Hq, dh = q.shape
    G = Hq // K.shape[2]
    sc = 1.0 / np.sqrt(dh) if scale is None else float(scale)
    out, spread = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    logit = np.full((B, T, Hq), np.nan)
    for b in range(B):
        n = T if count is None else int(count[b])
        for t in range(n):
            see = max(0, int(lens[b]) - (n - 1 - t))
            for h in range(Hq):
                k, v = K[b, :see, h // G], V[b, :see, h // G]
                if see == 0:
                    out[b, t, h] = spread[b, t, h] = logit[b, t, h] = 0.0
                    continue
                w = k @ q[b, t, h] * sc
                p = np.exp(w - w.max())
                p /= p.sum()
                out[b, t, h], spread[b, t, h] = p @ v, p @ np.abs(v)
                logit[b, t, h] = (np.abs(k) @ np.abs(q[b, t, h])).max() * sc
    return out, spread, logit
