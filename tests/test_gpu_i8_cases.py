"""Every kernel of the 8-bit products against the oracle, and layers of up to 1024
experts: empty blocks of experts, the last one in use, one that takes all."""

import numpy as np
import pytest
import torch

import bit_quantized_moe_route_amd as moeq
from tests.gpu_common import say
from tests.i8_cases import EXPERTS, LINEAR, ROUTED, SHARED, ffn, one_pass, taken
from tests.test_gpu_i8 import (DEV, check_linear, check_rows, codes, f64, make_layer, rnd,
                               run_experts, same_codes, scales)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,K,N", LINEAR)
def test_linear(T, K, N):
    say("linear", T, K, N, one_pass(T, 1, 1, False, N, K, False))
    rs = np.random.default_rng(T + K + N)
    W, S, bias = codes(rs, (N, K)), scales(rs, N), rnd(rs, (N,), torch.float32)
    lin = moeq.I8Linear(W, S, bias)
    x = rnd(rs, (T, K), torch.bfloat16, 2.0)
    out = moeq.linear_i8(lin, x, out_dtype=torch.float32)
    q, s = moeq.quantize_i8(x)
    rq, rscale = same_codes(x, q, s, "x")
    check_linear(lin, W.cpu().numpy(), f64(S), f64(bias), rq, rscale, out, (T, K, N))
    assert torch.equal(moeq.linear_i8(lin, q, s, out_dtype=torch.float32), out)


@pytest.mark.parametrize("T,H,I", SHARED)
def test_shared(T, H, I):
    say("shared", T, H, I, ffn(T, 1, 1, False, H, I))
    rs = np.random.default_rng(T + H + I)
    layer, mats = make_layer(rs, 1, H, I)
    x = rnd(rs, (T, H), torch.bfloat16)
    y = moeq.shared_ffn_i8(layer, x, y_dtype=torch.float32)
    q, s = moeq.quantize_i8(x)
    rq, rscale = same_codes(x, q, s, "x")
    check_rows(layer, mats, 0, rq, rscale, y, (T, H, I))
    assert torch.equal(moeq.shared_ffn_i8(layer, q, s, y_dtype=torch.float32), y)


@pytest.mark.parametrize("T,E,k,H,I", ROUTED)
def test_routed(T, E, k, H, I):
    say("routed", T, E, k, H, I, ffn(T, k, E, True, H, I))
    run_experts(T, E, k, H, I, "bf16", "fp32", T + E + H)


@pytest.mark.parametrize("T,E,k,H,I,which", EXPERTS)
def test_many_experts(T, E, k, H, I, which):
    say("experts", T, E, k, H, I, which, ffn(T, k, E, True, H, I))
    rs = np.random.default_rng(T + E)
    choice = np.array(taken(E, which))
    ids = choice[np.argsort(rs.random((T, len(choice))), 1)[:, :k]]
    assert ids.shape == (T, k)
    run_experts(T, E, k, H, I, "bf16", "fp32", T + E, ids)
