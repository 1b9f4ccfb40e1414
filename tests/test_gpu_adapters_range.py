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
