"""8-bit products whose row and channel scales have a product outside fp32's
normal range while the result lies inside: each kernel against fp64."""

import numpy as np
import pytest
import torch

import bit_quantized_moe_route_amd as moeq
from oracle import block as ob
from tests.gpu_common import say

pytestmark = pytest.mark.gpu

DEV = "cuda"


def f64(t):
    return t.double().cpu().numpy()


# coded inside the product, streaming, GEMM
@pytest.mark.parametrize("T", [1, 3, 12, 300])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("xs,ws", [(-90, -50), (-110, -36), (60, 40)])
def test_linear(T, xs, ws, bias):
    say("scales", T, xs, ws, bias)
    K, N = 712, 528
    rs = np.random.default_rng(T)
    W = rs.integers(-128, 128, (N, K)).astype(np.int8)
    W[5] = 0                                     # a sum of 0 stays 0
    S = (rs.uniform(1, 2, N) * 2.0 ** ws).astype(np.float32)
    x = (rs.standard_normal((T, K)) * 2.0 ** xs).astype(np.float32)
    b = (rs.standard_normal(N) * 2.0 ** (xs + ws + 8)).astype(np.float32) if bias else None
    lin = moeq.I8Linear(*(torch.from_numpy(t).to(DEV) for t in (W, S)),
                        None if b is None else torch.from_numpy(b).to(DEV))
    q, s = ob.quantize_i8(x)
    out = f64(moeq.linear_i8(lin, torch.from_numpy(x).to(DEV)))
    ref = ob.product_i8(q, W) * s[:, None].astype(np.float64) * S.astype(np.float64)
    mag = np.abs(ref)
    if bias:
        ref = ref + b.astype(np.float64)
        mag = mag + np.abs(ref)
    # four roundings and the bias' sum; results may be subnormal themselves
    err = np.abs(out - ref)
    assert np.all(err <= 5 * 2.0 ** -24 * mag + 2.0 ** -149), float((err / (mag + 1e-300)).max())


@pytest.mark.parametrize("T", [1, 3, 12, 300])
def test_linear_zero_sums_under_large_scales(T):
    """Scales whose product is past fp32: a sum of 0 is 0 (and not a NaN)."""
    K, N = 72, 40
    lin = moeq.I8Linear(torch.zeros((N, K), dtype=torch.int8, device=DEV),
                        torch.full((N,), 2.0 ** 100, device=DEV))
    x = torch.full((T, K), 2.0 ** 100, device=DEV)
    assert torch.all(moeq.linear_i8(lin, x) == 0)


@pytest.mark.parametrize("T", [1, 3, 12, 300])
@pytest.mark.parametrize("routed", [False, True])
def test_gate_and_up(T, routed):
    """g near 2^-125 from scales whose product is near 2^-145; h = g u / 2."""
    H, I = 712, 80
    rs = np.random.default_rng(T + 1)
    w13 = rs.integers(-128, 128, (1, 2 * I, H)).astype(np.int8)
    w2 = rs.integers(-128, 128, (1, H, I)).astype(np.int8)
    s13 = rs.uniform(1, 2, (1, 2 * I))
    s13[:, :I] *= 2.0 ** -45
    s13[:, I:] *= 2.0 ** 112
    s13, s2 = s13.astype(np.float32), (rs.uniform(1, 2, (1, H)) * 2.0 ** 80).astype(np.float32)
    layer = moeq.I8Layer(*(torch.from_numpy(t).to(DEV) for t in (w13, s13, w2, s2)))
    x = (rs.standard_normal((T, H)) * 2.0 ** -95).astype(np.float32)
    xd = torch.from_numpy(x).to(DEV)
    if routed:
        _, off, perm, _ = moeq.permute(torch.zeros((T, 1), dtype=torch.int32, device=DEV), 1)
        y = moeq.expert_ffn_i8(layer, xd, perm, off, 1)
    else:
        y = moeq.shared_ffn_i8(layer, xd)
    q, s = ob.quantize_i8(x)
    # g and u: 4 roundings each (8 * 2^-24), and silu's (2^-20): codes of h within
    # that of a tie may be either
    ref, slack, _ = ob.expert_i8(q, s, w13[0], s13[0], w2[0], s2[0], 2.0 ** -20 + 2.0 ** -21)
    err = np.abs(f64(y) - ref)
    tol = (2.0 ** -24 + 2.0 ** -20) * np.abs(ref) + 1.01 * slack
    assert np.all(err <= tol), float((err / tol).max())
