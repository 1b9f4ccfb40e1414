"""Plain numpy (fp64) forms of what stands beside and behind a projection, written
from their definitions: head norms with rotation, token log probabilities, low-rank
adapters.  Arrays in, arrays out; float inputs are taken as the values they hold.

A result comes with what an error of its fp32 arithmetic is relative to.
"""

import numpy as np


def angles(positions, rotated, base=10000.0, freq=None):
    """[positions, rotated / 2] angles: position * base^(-2 i / rotated)."""
    if freq is None:
        freq = np.float64(base) ** (-np.arange(0, rotated, 2) / np.float64(rotated))
    return np.arange(positions, dtype=np.float64)[:, None] * np.asarray(freq, np.float64)


def heads(x, w=None, eps=1e-5, w_offset=0.0, cos=None, sin=None, interleaved=False):
    """x [T, heads, D]; cos, sin [T, R / 2] or None.  Returns the heads and their
    magnitude: the sum of each element's absolute terms."""
    n = np.array(x, np.float64)
    if w is not None:
        n = n / np.sqrt((n * n).mean(2, keepdims=True) + eps) * (w_offset + np.asarray(w, np.float64))
    out, mag = n.copy(), np.abs(n)
    if cos is None:
        return out, mag
    for i in range(cos.shape[1]):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, cos.shape[1] + i)
        c, s = cos[:, i, None], sin[:, i, None]
        a, b = n[:, :, p], n[:, :, q]
        out[:, :, p], out[:, :, q] = a * c - b * s, b * c + a * s
        mag[:, :, p] = np.abs(a * c) + np.abs(b * s)
        mag[:, :, q] = np.abs(b * c) + np.abs(a * s)
    return out, mag


def logprobs(logits, scale=None):
    """log p [T, V], entropy [T], and the first two moments of scale * (max x - x)
    under p.  A row masked as a whole: -inf, 0.  One with a NaN, +inf or a scale that is
    not positive and finite: NaN."""
    x = np.asarray(logits, np.float64)
    T = x.shape[0]
    lp, H = np.empty(x.shape), np.empty(T)
    m1, m2 = np.zeros(T), np.zeros(T)
    for t in range(T):
        s = 1.0 if scale is None else float(scale[t])
        if np.isnan(x[t]).any() or (x[t] == np.inf).any() or not 0 < s < np.inf:
            lp[t], H[t] = np.nan, np.nan
            continue
        if (x[t] == -np.inf).all():
            lp[t], H[t] = -np.inf, 0.0
            continue
        z = s * (x[t] - x[t].max())
        e = np.exp(z)
        lp[t] = z - np.log(e.sum())
        p, live = e / e.sum(), e > 0
        H[t] = -(p[live] * lp[t][live]).sum()
        m1[t] = -(p[live] * z[live]).sum()
        m2[t] = (p[live] * z[live] ** 2).sum()
    return lp, H, m1, m2


def best(logits, top):
    """The ids of each row's `top` largest logits, equal ones by the lower id, -1 where
    only masked ones are left; a row with a NaN or +inf: -1."""
    x = np.asarray(logits, np.float64)
    out = np.full((x.shape[0], top), -1, np.int64)
    for t, row in enumerate(x):
        if np.isnan(row).any() or (row == np.inf).any():
            continue
        order = sorted(np.flatnonzero(row > -np.inf).tolist(), key=lambda v: (-row[v], v))[:top] \
            if len(row) < 4096 else _best_long(row, top)
        out[t, :len(order)] = order
    return out


def _best_long(row, top):
    """The same by the stable sort of numpy."""
    order = np.argsort(-row, kind="stable")[:top]
    return [v for v in order.tolist() if row[v] > -np.inf]


def add_adapters(x, ids, adapters, y):
    """adapters: a list of (A, B, scale) or None (an empty slot); ids outside the list:
    none.  Returns out, and for the error of its steps: sum_r |B| |h|, sum_r |B| sum_k |A x|
    and sum_r |B| max_r |h|, each with the scale."""
    x, out = np.asarray(x, np.float64), np.array(y, np.float64)
    mags = [np.zeros(out.shape) for _ in range(3)]
    for t, i in enumerate(np.asarray(ids).tolist()):
        if not 0 <= i < len(adapters) or adapters[i] is None:
            continue
        A, B, s = (np.asarray(v, np.float64) for v in adapters[i])
        h = s * (A @ x[t])
        out[t] += B @ h
        absB = np.abs(B)
        mags[0][t] = absB @ np.abs(h)
        mags[1][t] = absB @ (np.abs(s) * (np.abs(A) @ np.abs(x[t])))
        mags[2][t] = absB.sum(1) * np.abs(h).max()
    return (out, *mags)
