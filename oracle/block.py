"""Plain numpy (fp64) forms of the block norms and the 8-bit integer products,
written from their definitions.  Arrays in, arrays out; float inputs are taken
as the values they hold.

Each of the norm's results comes with a magnitude, the same sum over absolute
values: what a rounding error of its fp32 terms is relative to.
"""

import numpy as np


def rms_norm(v, w, eps, w_offset=0.0):
    v = np.asarray(v, np.float64)
    rstd = 1.0 / np.sqrt((v * v).mean(1, keepdims=True) + eps)
    return v * rstd * (w_offset + np.asarray(w, np.float64)), rstd


def gated_sum(y_perm, inv_perm, topk_w, y_shared=None, shared_gate=None):
    """sum_j topk_w[t, j] * y_perm[inv_perm[t*k + j]] + shared_gate * y_shared,
    and its magnitude."""
    T, k = topk_w.shape
    y = np.asarray(y_perm, np.float64)[np.asarray(inv_perm).reshape(T, k)]
    terms = y * np.asarray(topk_w, np.float64)[:, :, None]
    out, mag = terms.sum(1), np.abs(terms).sum(1)
    if y_shared is not None:
        s = np.asarray(y_shared, np.float64)
        if shared_gate is not None:
            s = s * np.asarray(shared_gate, np.float64)[:, None]
        out, mag = out + s, mag + np.abs(s)
    return out, mag


def block(r, y, pre_w=None, post_w=None, gate=None, y_scale=1.0, r_scale=1.0, eps=1e-5,
          w_offset=0.0, y_mag=None):
    """r' = r_scale r + y_scale gate (N(y; post_w) or y), n = N(r'; pre_w) or r'.
    r or y may be None.  Returns (r', its magnitude, n, its magnitude)."""
    out = mag = 0.0
    if y is not None:
        p = np.asarray(y, np.float64)
        m = np.abs(p) if y_mag is None else y_mag
        if post_w is not None:
            p, rstd = rms_norm(p, post_w, eps, w_offset)
            m = m * rstd * np.abs(w_offset + np.asarray(post_w, np.float64))
        g = 1.0 if gate is None else np.asarray(gate, np.float64)
        out, mag = y_scale * g * p, np.abs(y_scale * g) * m
    if r is not None:
        a = r_scale * np.asarray(r, np.float64)
        out, mag = out + a, mag + np.abs(a)
    if pre_w is None:
        return out, mag, out, mag
    n, rstd = rms_norm(out, pre_w, eps, w_offset)
    return out, mag, n, mag * rstd * np.abs(w_offset + np.asarray(pre_w, np.float64))


def quantize_i8(x):
    """Codes and scales of the rows of x: scale = a / 127 in fp32, code =
    rint(127 x / a), ties to even.  127 x is exact in fp64; a quotient of two
    fp32 numbers above 0.49 that is no tie lies at least 2^-33 off one, and the
    fp64 quotient within 2^-47 of it, so its rounding is the exact one's."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        a = np.abs(x).max(1)
        a = np.where(np.isnan(x).any(1), np.float32(np.nan), a).astype(np.float32)
        ok = np.isfinite(a) & (a >= np.float32(127) * np.float32(2.0 ** -126))
        scale = np.where(ok, a / np.float32(127), np.where(np.isfinite(a), 0, np.nan))
        v = np.where(ok[:, None], x.astype(np.float64) * 127 / np.where(ok, a, 1)[:, None], 0)
    return np.rint(v).astype(np.int8), scale.astype(np.float32)


def product_i8(q, W):
    """Exact integer sums of q [T, K] with the rows of W [N, K]."""
    # |sum| <= 127 * 128 * K < 2^53: fp64 holds every partial sum exactly
    return np.asarray(q, np.float64) @ np.asarray(W, np.float64).T


def expert_i8(q, scale, w13, s13, w2, s2, eps_h):
    """One expert on coded rows: y [rows, H] and how far another evaluation of h,
    off by at most eps_h of the row's largest |h|, can take it: codes that lie
    near the border between two integers (their number comes third) may come out
    as the other one."""
    I = w13.shape[0] // 2
    gu = product_i8(q, w13) * np.asarray(scale, np.float64)[:, None] * np.asarray(s13, np.float64)
    g, u = gu[:, :I], gu[:, I:]
    with np.errstate(over="ignore"):
        h = g / (1.0 + np.exp(-g)) * u
    a = np.abs(h).max(1, keepdims=True)
    live = a > 0
    v = np.where(live, h * 127.0 / np.where(live, a, 1.0), 0.0)
    step = a / 127.0 * np.asarray(s2, np.float64)
    near = np.abs(v - np.floor(v) - 0.5) <= 2 * 127 * eps_h
    aw = np.abs(np.asarray(w2, np.float64))
    y = step * product_i8(np.rint(v), w2)
    slack = step * (near.astype(np.float64) @ aw.T + 2 * eps_h * (np.abs(np.rint(v)) @ aw.T))
    return y, slack, int(near.sum())
