"""The gate of the 8-bit feed-forward over its range: one middle channel, so that
y = silu(g) * u up to single roundings, with g and u exact by construction."""

import numpy as np
import pytest
import torch

import bit_quantized_moe_route_amd as moeq
from tests.gpu_common import say

pytestmark = pytest.mark.gpu

DEV = "cuda"
H = 72


def layer():
    """g = 2^-7 (127 q1 + q2), u = 127 / 128 of a row with q0 = 127 and scale 1."""
    w13 = torch.zeros((1, 2, H), dtype=torch.int8, device=DEV)
    w13[0, 0, 1], w13[0, 0, 2], w13[0, 1, 0] = 127, 1, 1
    return moeq.I8Layer(w13, torch.full((1, 2), 2.0 ** -7, device=DEV),
                        torch.ones((1, H, 1), dtype=torch.int8, device=DEV),
                        torch.ones((1, H), device=DEV))


def run(L, x, routed):
    T = x.shape[0]
    if not routed:
        return moeq.shared_ffn_i8(L, x)
    _, off, perm, _ = moeq.permute(torch.zeros((T, 1), dtype=torch.int32, device=DEV), 1)
    return moeq.expert_ffn_i8(L, x, perm, off, 1)


# coded inside the product, streaming, GEMM
@pytest.mark.parametrize("T", [1, 4, 12, 700])
@pytest.mark.parametrize("routed", [False, True])
def test_gate(T, routed):
    say("silu", T, routed)
    L = layer()
    rs = np.random.default_rng(T)
    for _ in range(40 if T < 100 else 4):
        q1, q2 = rs.integers(-80, 128, T), rs.integers(-127, 128, T)
        x = np.zeros((T, H), np.float32)
        x[:, 0], x[:, 1], x[:, 2] = 127, q1, q2
        g = (127.0 * q1 + q2) / 128
        ref = g / (1 + np.exp(-g)) * (127 / 128)
        y = run(L, torch.from_numpy(x).to(DEV), routed).double().cpu().numpy()
        # in units of 2^-24: exp 2, g exp, 1 + exp, the quotient, times u, the
        # scale h / 127, times the code 127: 8, and one for their products
        err = np.abs(y - ref[:, None])
        tol = 9 * 2.0 ** -24 * np.abs(ref[:, None])
        at = np.argmax(err - tol, 0)[0]
        assert np.all(err <= tol), (g[at], ref[at], y[at, 0])


@pytest.mark.parametrize("T", [1, 12, 300])
def test_far_gates(T):
    """Gates past the exponential's range: nothing but zeros, u and NaNs of NaNs."""
    L = layer()
    x = torch.zeros((T, H), device=DEV)
    x[:, 0], x[:, 1] = 127, -126.0                  # g near -125: h below the smallest row
    assert torch.all(run(L, x, False) == 0)
    x[:, 1] = 126.0                                 # silu(g) = g
    g = 126 * 127 / 128
    assert torch.all((run(L, x, False).double() - g * 127 / 128).abs() <= 9 * 2.0 ** -24 * g)
    x[0, 3] = float("nan")
    assert torch.isnan(run(L, x, False)[0]).all()
    # a gate that overflows: -inf gives 0, inf an infinite row, whose y is NaN
    big = moeq.I8Layer(torch.ones((1, 2, H), dtype=torch.int8, device=DEV),
                       torch.tensor([[2.0 ** 120, 1.0]], device=DEV),
                       torch.ones((1, H, 1), dtype=torch.int8, device=DEV),
                       torch.ones((1, H), device=DEV))
    x = torch.full((T, H), 2.0 ** 20, device=DEV)
    assert torch.all(run(big, -x, False) == 0)
    assert torch.isnan(run(big, x, False)).all()
