"""Adapters whose ranks differ strongly in size: what of A x reaches the result.

Tolerance, from the kernel's arithmetic, as in test_gpu_adapters.py but for the split of
h = s A x into two fp16 numbers.  The token's row of h goes to a largest of 2^14 to 2^15 by a
power of two.  The first number is off by half a step, 2^-11 of the value at most; the second by
2^-11 of that difference, or by half of fp16's smallest step, 2^-25.  So h is kept to 2^-22 of
itself or 2^-39 of the token's largest, whichever is more.
"""

import numpy as np
import pytest
import torch

import bit_quantized_moe_route_amd as moeq
from oracle import project as op
from tests.gpu_common import say
from tests.test_gpu_adapters import DEV, TINY, TYPES, f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("y", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("T,rank,K,N", [(1, 8, 64, 100), (37, 16, 200, 130), (50, 40, 1001, 64),
                                        (20, 200, 320, 72), (2800, 40, 64, 136), (1030, 100, 64, 70)])
def test_ranks_of_different_size(T, rank, K, N, y):
    """fp16: ranks down to 2^-18 of the largest, with columns of B that make up for it, and
    channels that see the small ones alone."""
    say("sizes", T, rank, K, N, y)
    rs = np.random.default_rng(T + rank)
    n = 2
    s = moeq.Adapters(n, rank, K, N, dtype=torch.float16)
    known = []
    for i in range(n):
        e = rs.integers(0, 19, rank)
        e[0], e[-1] = 0, 18
        a = 2.0 * rs.standard_normal((rank, K)) * K ** -0.5 * 2.0 ** -e[:, None]
        b = rs.standard_normal((N, rank)) * 2.0 ** (e - 6.0)
        b[::2, e < 9] = 0.0
        a, b = (torch.from_numpy(v).to(torch.float16).to(DEV) for v in (a, b))
        s.load(i, a, b, 0.75)
        known.append((f64(a), f64(b), np.float32(0.75)))
    ids = rs.integers(-1, n, T).astype(np.int32)
    ids[0] = 0
    x = torch.from_numpy(rs.standard_normal((T, K))).to(torch.float16).to(DEV)
    rows = torch.zeros((T, N), dtype=TYPES[y], device=DEV)
    got = moeq.add_adapters(s, x, moeq.adapter_plan(torch.from_numpy(ids).to(DEV), n), rows,
                            out=torch.empty_like(rows))
    ref, bh, bax, bmax = op.add_adapters(f64(x), ids, known, f64(rows))
    tol = 2.0 ** -23 * ((K / 16 + 152) * bax + (3 * rank + 8) * bh) + 2.0 ** -22 * bh + 2.0 ** -39 * bmax
    half = torch.finfo(rows.dtype).eps / 2
    tol = tol * (1 + half) + (half + 2.0 ** -24) * np.abs(ref) + TINY[rows.dtype]
    err = np.abs(f64(got) - ref)
    assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("w", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [5, 4200])
@pytest.mark.parametrize("e", [-118, -105, 100, 120])
def test_scales_far_from_one(e, T, w):
    """s A x near both ends of fp32's range, and results that return to its middle.  Numbers of
    fp32 below 2^-126 are off by 2^-150 a rounding (under 32 of them in h), those of bf16 by
    2^-134."""
    say("far scales", e, T, w)
    rs = np.random.default_rng(T)
    rank, K, N, n = 32, 96, 70, 2
    s, known = moeq.Adapters(n, rank, K, N, dtype=TYPES[w]), []
    back = -e if w == "bf16" else (12 if e < 0 else -12)
    for i in range(n):
        a = torch.from_numpy(rs.standard_normal((rank, K)) / 8).to(TYPES[w]).to(DEV)
        b = torch.from_numpy(rs.standard_normal((N, rank)) * 2.0 ** back).to(TYPES[w]).to(DEV)
        s.load(i, a, b, 2.0 ** e)
        known.append((f64(a), f64(b), np.float32(2.0 ** e)))
    ids = rs.integers(0, n, T).astype(np.int32)
    x = torch.from_numpy(rs.standard_normal((T, K))).to(TYPES[w]).to(DEV)
    y = torch.zeros((T, N), device=DEV)
    got = moeq.add_adapters(s, x, moeq.adapter_plan(torch.from_numpy(ids).to(DEV), n), y,
                            out=torch.empty_like(y))
    ref, bh, bax, bmax = op.add_adapters(f64(x), ids, known, f64(y))
    split = 2.0 ** -24 * bh if w == "bf16" else 2.0 ** -22 * bh + 2.0 ** -39 * bmax
    small = 2.0 ** -145 + (2.0 ** -134 if w == "bf16" else 0)
    absb = np.stack([np.abs(k[1]).sum(1) for k in known])[ids]
    tol = 2.0 ** -23 * ((K / 16 + 152) * bax + (3 * rank + 8) * bh) + split + small * absb
    tol = tol * (1 + 2.0 ** -24) + 2.0 ** -23 * np.abs(ref) + 2.0 ** -149
    err = np.abs(f64(got) - ref)
    assert np.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("w", ["bf16", "fp16"])
@pytest.mark.parametrize("T,rank", [(3, 1), (4200, 32)])
@pytest.mark.parametrize("y", ["fp32", "bf16"])
def test_the_largest_values(T, rank, y, w):
    """s A x between the largest number of bf16 and that of fp32 is a number like any other."""
    say("largest", T, rank, y, w)
    K, N = 40, 70
    s = moeq.Adapters(1, rank, K, N, dtype=TYPES[w])
    a, b = (torch.zeros(shape, dtype=TYPES[w], device=DEV) for shape in ((rank, K), (N, rank)))
    a[0, 3] = 1.0
    b[:, 0] = 2.0 ** -10 * (torch.arange(N, device=DEV) % 7 - 3)
    scale = float(np.float32(3.3975e38))
    s.load(0, a, b, scale)
    x = torch.zeros((T, K), dtype=TYPES[w], device=DEV)
    x[:, 3] = 1.0
    x[1::2, 3] = -1.0
    rows = torch.zeros((T, N), dtype=TYPES[y], device=DEV)
    got = moeq.add_adapters(s, x, moeq.adapter_plan(torch.zeros(T, dtype=torch.int32, device=DEV), 1),
                            rows, out=torch.empty_like(rows))
    ref = f64(x)[:, 3:4] * scale * f64(b)[:, 0]
    # one product: the split's 2^-24 (bf16, fp32 results), 2^-16 (bf16) or 2^-22 of h, two
    # roundings of fp32 and one of y
    split = 2.0 ** -22 if w == "fp16" else 2.0 ** -24 if y == "fp32" else 2.0 ** -16
    tol = (split + 2.0 ** -22 + torch.finfo(rows.dtype).eps / 2) * np.abs(ref)
    err = np.abs(f64(got) - ref)
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-300)).max())
