"""Token log probabilities where scale times logit leaves fp32's range: scales up to the
largest finite one, scaled logits that overflow, differences of logits that overflow.

Tolerances are test_gpu_logprobs.py's; a log probability below fp32's lowest value is -inf
there (the cases keep a factor of 1.05 from that border).
"""

import numpy as np
import pytest
import torch

import bit_quantized_moe_route_amd as moeq
from oracle import project as op
from tests.gpu_common import say
from tests.test_gpu_logprobs import DEV, STEP, TYPES

pytestmark = pytest.mark.gpu

LARGEST = float(np.finfo(np.float32).max)
V = 20000                                   # two slices


def check(x, scale, ids, top):
    T = x.shape[0]
    sc = torch.tensor(scale, dtype=torch.float32, device=DEV)
    at = torch.tensor(ids, dtype=torch.int32, device=DEV).repeat(T, 1)
    got = moeq.token_logprobs(x, at, top=top, scale=sc)
    x64 = x.to(torch.float64).cpu().numpy()
    lp, H, m1, m2 = op.logprobs(x64, sc.cpu().numpy())

    def close(a, b, tol, what):
        a = a.cpu().numpy().astype(np.float64)
        b = np.where(b < -LARGEST, -np.inf, b)
        assert np.array_equal(np.isnan(a), np.isnan(b)), what
        assert np.array_equal(np.isneginf(a), np.isneginf(b)), what
        live = np.isfinite(b)
        err = np.abs(np.where(live, a, 0) - np.where(live, b, 0))
        assert np.all(err <= tol), (what, float((err / tol).max()))

    def tol(want):
        return STEP * (np.where(want < -LARGEST, 0, -want) * 2 + m1[:, None] + 24)

    close(got[1], H, STEP * (m2 + m1 * m1 + 40 * m1 + 24), "entropy")
    want = lp[:, ids]
    close(got[0], want, tol(want), "log p")
    best = op.best(x64, top)
    assert np.array_equal(got[2].cpu().numpy(), best), "best tokens"
    want = np.take_along_axis(lp, best, 1)
    close(got[3], want, tol(want), "best log p")


@pytest.mark.parametrize("dt", sorted(TYPES))
def test_scales_up_to_the_largest(dt):
    """Scales that leave fp32's range once they are in units of log2 e are scales like any other:
    logits that lie a few parts of 2^-127 apart (fp16: the next one is 2^-24 off, and has
    no probability left)."""
    say("largest scales", dt)
    rs = np.random.default_rng(21)
    unit = 2.0 ** -24 if dt == "fp16" else 2.0 ** -127
    scales = (1.0e38, 1.7e38, 2.35e38, 2.4e38, 3.0e38, LARGEST)
    steps = rs.integers(0, 9, (len(scales), V))
    steps[1::2, :16384] += 1                # the largest in the second slice alone
    x = torch.from_numpy(-steps * unit).to(TYPES[dt]).to(DEV)
    check(x, scales, [0, 16383, 16384, V - 1], 12)


@pytest.mark.parametrize("dt,low,high,scale", [
    ("fp32", -6.0, 0.0, 1.2e38), ("bf16", -6.0, 0.0, 1.2e38), ("fp16", -6.0, 0.0, 1.2e38),
    ("fp32", -1e27, 0.0, 1e12), ("bf16", -1e27, 0.0, 1e12), ("fp16", -65504.0, 0.0, 1e35),
    ("fp32", -1e20, 0.0, 1e19), ("fp32", -1e20, 1e-15, 1e19), ("bf16", -1e20, -1e-15, 1e19),
    ("fp32", -6.0, 1e-34, 1.2e38), ("bf16", -1e30, 1.0, 1e9), ("fp32", -1e30, 700.0, 1e9)])
def test_scaled_logits_that_overflow(dt, low, high, scale):
    """Most logits times the scale are past fp32's range, two share the largest and one lies
    a part of the scale below: an entropy of those."""
    say("overflow", dt, low, high, scale)
    x = torch.full((4, V), low, dtype=TYPES[dt], device=DEV)
    x[0, 7] = x[0, 11] = high
    x[1, 7] = x[1, 17000] = high            # one in each slice
    x[2, 7] = x[2, 17000] = high
    x[2, 8] = high - 1 / scale
    x[3, 19999] = high                      # a slice of low ones, and one with the largest
    check(x, [scale] * 4, [0, 7, 8, 17000, 19999], 3)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_differences_that_overflow(dt):
    """Logits that lie further apart than fp32's largest value, at scales that bring them
    together again.  (3e-40 is held to 2^-150 as a factor of differences up to 2^129, so
    to 2^-21 of an exponent: under the tolerance's 24 parts of 2^-22.)"""
    say("differences", dt)
    rs = np.random.default_rng(22)
    x = torch.from_numpy(rs.integers(-3, 4, (10, V)) * 1e38).to(TYPES[dt]).to(DEV)
    x[5:, :16384] = -3e38                   # a slice apart from the largest
    x[5:, 19000] = 3e38
    scales = [2e-38, 3e-40, 1e-37, 1e-30, 1e-4] * 2
    check(x, scales, [0, 5, 16384, 18000, 19000], 8)
