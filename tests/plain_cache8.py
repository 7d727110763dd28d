"""Plain 64-bit forms of the normed rotary write, of the 8-bit cache and of
attention through a window, written from their definitions (numpy, no code of
the library)."""
from __future__ import annotations

import numpy as np


def normed(x, weight, eps, offset=0.0):
    """x [T,N,D] float64 normed over each head (weight None: as it is)."""
    x = np.asarray(x, dtype=np.float64)
    if weight is None:
        return x
    mean = np.mean(x * x, axis=-1, keepdims=True)
    return x / np.sqrt(mean + eps) * (np.asarray(weight, np.float64) + offset)


def norm_error(head_dim):
    """Relative error of a normed value in fp32: the sum of squares of D terms
    (D half-ulps at worst, halved by the root), the root's own 2^-22, the mean,
    the sum with eps, the weight's sum and two products (6 half-ulps)."""
    return (head_dim / 2 + 6) * 2.0 ** -24 + 2.0 ** -22


def e4m3(x):
    """The nearest e4m3 value: 3 fraction bits down to 2^-6, below it multiples
    of 2^-9; ties to even; at most 448. NaN stays NaN."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        a = np.abs(np.where(np.isfinite(x), x, 1.0))
        step = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
        y = np.clip(np.where(np.isinf(x), x, np.rint(np.where(np.isinf(x), 0, x) / step) * step),
                    -448.0, 448.0)
    return np.where(np.isnan(x), np.nan, y)


def block_scale(top):
    """2^ceil(log2(top / 448)), at least 2^-100."""
    m, e = np.frexp(np.maximum(np.asarray(top, np.float64), 448.0 * 2.0 ** -100) / 448.0)
    return np.exp2(np.where(m == 0.5, e - 1, e).astype(np.float64))


def append(pool, scales, k, v, table, cu, lens):
    """pool [2,NB,BS,Hkv,D] (the e4m3 values), scales [2,NB,Hkv]; k, v [T,Hkv,D].
    Returns the pool and the scales after the write, and what each new row's
    values were before rounding (NaN where nothing is written)."""
    pool, scales = np.array(pool, np.float64), np.array(scales, np.float64)
    raw = np.full(pool.shape, np.nan)
    bs = pool.shape[2]
    new = np.stack([np.asarray(k, np.float64), np.asarray(v, np.float64)])
    for i in range(len(lens)):
        t0, n, L = int(cu[i]), int(cu[i + 1] - cu[i]), int(lens[i])
        for b in range((L - n) // bs, (L - 1) // bs + 1) if n else ():
            first, last = max(0, L - n - b * bs), min(bs, L - b * bs)
            x = new[:, t0 + b * bs + first - (L - n):t0 + b * bs + last - (L - n)]
            finite = np.where(np.isfinite(x), np.abs(x), 0)
            s = block_scale(finite.max((1, 3)))
            blk = table[i][b]
            if first:
                old = scales[:, blk]
                s = np.maximum(s, old)
                grown = (s != old)[:, None, :, None]
                again = e4m3(pool[:, blk, :first] * (old / s)[:, None, :, None])
                pool[:, blk, :first] = np.where(grown, again, pool[:, blk, :first])
            scales[:, blk] = s
            raw[:, blk, first:last] = x
            pool[:, blk, first:last] = e4m3(x / s[:, None, :, None])
    return pool, scales, raw


def attention(q, keys, values, lens, cu, scale, window=0, sink=0):
    """q [T,H,D]; keys(i), values(i) -> [L,Hkv,D] float64 of request i. Returns
    out [T,H,D], lse [T,H], and the weighted sum of |value| per output (the
    magnitude that rounding of the weights acts on). Rows of no request are NaN."""
    q = np.asarray(q, np.float64)
    out, mag = np.full(q.shape, np.nan), np.full(q.shape, np.nan)
    lse = np.full(q.shape[:2], np.nan)
    for i in range(len(lens)):
        t0, n, L = int(cu[i]), int(cu[i + 1] - cu[i]), int(lens[i])
        if n == 0:
            continue
        k, v = keys(i), values(i)
        g = q.shape[1] // k.shape[1]
        pos = (L - n + np.arange(n))[:, None]
        j = np.arange(L)[None, :]
        seen = j <= pos
        if window:
            seen &= (pos - j < window) | (j < sink)
        for h in range(q.shape[1]):
            vh = np.where(seen.any(0)[:, None], v[:, h // g], 0.0)
            kh = np.where(seen.any(0)[:, None], k[:, h // g], 0.0)
            s = np.where(seen, q[t0:t0 + n, h] @ kh.T * scale, -np.inf)
            m = s.max(1, keepdims=True)
            p = np.exp(s - m)
            total = p.sum(1, keepdims=True)
            out[t0:t0 + n, h] = p @ vh / total
            mag[t0:t0 + n, h] = p @ np.abs(vh) / total
            lse[t0:t0 + n, h] = (m + np.log(total))[:, 0]
    return out, lse, mag
