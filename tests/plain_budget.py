"""Plain 64-bit forms of the rotary cache write and the cache-budget calls,
written from their definitions (numpy, no code of the library)."""
from __future__ import annotations

import numpy as np


def rope(x, positions, inv_freq, factor, interleaved):
    """x [T,N,D] float64 rotated by positions [T]; also, per element, the sum
    of the magnitudes of the pair it came from (0 where it passes through)."""
    x = np.asarray(x, dtype=np.float64)
    r = 2 * len(inv_freq)
    t = np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq)[None, :]
    c, s = (factor * np.cos(t))[:, None, :], (factor * np.sin(t))[:, None, :]
    ia = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
    ib = ia + 1 if interleaved else ia + r // 2
    out, mag = x.copy(), np.zeros_like(x)
    a, b = x[..., ia], x[..., ib]
    out[..., ia], out[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = mag[..., ib] = factor * (np.abs(a) + np.abs(b))
    return out, mag


def key_weights(weights, q, k_rows, lse, cu, lens, rows, prior, decay, scale, out):
    """k_rows(i) -> [L,Hkv,D] float64 keys of request i. Returns (out, bound):
    bound is how far an fp32 computation may be off each entry."""
    out = np.array(out, dtype=np.float64)
    bound = np.zeros_like(out)
    hkv = out.shape[1]
    eps = 2.0 ** -24
    for i in range(len(lens)):
        n, L = int(cu[i + 1] - cu[i]), int(lens[i])
        if n == 0:
            continue
        k = k_rows(i)
        g = q.shape[1] // hkv
        old = prior[i] if prior is not None else L - n
        hidden = np.arange(L)[None, :] > (L - n + np.arange(n))[:, None]
        for h in range(hkv):
            total, err = np.zeros(L), np.zeros(L)
            for a in range(h * g, (h + 1) * g):
                qa, la = q[cu[i]:cu[i + 1], a].astype(np.float64), lse[cu[i]:cu[i + 1], a]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = qa @ k[:, h].T * scale
                    mag = np.abs(qa) @ np.abs(k[:, h]).T * scale
                    # a dot product of D terms (a tensor core may truncate: eps
                    # counts twice), the exponent's products and difference
                    # (three roundings of at most |s| + |lse|, the constant's
                    # among them), the exponential's own 2^-22
                    off = (q.shape[2] * 2 * eps * mag
                           + 3 * eps * (np.abs(s) + np.abs(la)[:, None]) + 2.0 ** -22)
                    w = np.exp(s - la[:, None])
                w = np.where(hidden | (la == -np.inf)[:, None], 0.0, w)
                total += w.sum(0)
                with np.errstate(invalid="ignore"):
                    err += np.where(w > 0, w * off, 0.0).sum(0)
            # summed one by one at worst
            err += total * eps * (n * g + 2)
            before = np.asarray(weights[rows[i], h, :L], np.float64)
            before = np.where(np.arange(L) < old, before, 0)
            if decay == 0:
                before = np.zeros(L)
            out[rows[i], h, :L] = decay * before + total
            bound[rows[i], h, :L] = err + eps * (2 * np.abs(decay * before) + total) + 1e-30
    return out, bound


def select(w, keep, sink, recent):
    """Indexes, ascending, that a row of L weights keeps."""
    L = len(w)
    r = min(recent, keep)
    s = min(sink, keep - r)
    middle = np.arange(s, L - r)
    v = np.asarray(w, dtype=np.float64)[middle]
    v = np.where(np.isnan(v), np.inf, v)
    nan = np.isnan(np.asarray(w, dtype=np.float64)[middle])
    order = np.lexsort((middle, -v, ~nan))  # NaN first, then by weight, then by index
    heavy = middle[order][:keep - s - r]
    return np.sort(np.concatenate([np.arange(s), heavy, np.arange(L - r, L)]))
