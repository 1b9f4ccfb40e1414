"""CPU tests of the head norms with rotation, the token log probabilities and the
low-rank adapters: the oracle's pins, sizes, and the refusals of the C calls and the
binding (nothing is launched)."""

import ctypes
import math

import numpy as np
import pytest
import torch

import bit_quantized_moe_route_amd as moeq
from bit_quantized_moe_route_amd import adapters as ma
from bit_quantized_moe_route_amd import heads as mh
from oracle import project as op

P = 1 << 20        # an aligned address no refused call ever reads
BAD, UNSUPPORTED, WORKSPACE = moeq.MOE_EINVAL, moeq.MOE_EUNSUPPORTED, moeq.MOE_EWORKSPACE


# ------------------------------------------------------------------ oracle

def test_heads_closed_forms():
    x = np.array([[[3.0, -4.0, 1.0]]])
    out, _ = op.heads(x, np.ones(3), 0.0)
    assert np.allclose(out, x / math.sqrt(26 / 3), rtol=1e-15)
    # a quarter turn takes (a, b) to (-b, a)
    c, s = np.zeros((1, 1)), np.ones((1, 1))
    assert np.array_equal(op.heads(x, cos=c, sin=s)[0], [[[4.0, 3.0, 1.0]]])
    x4 = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    c, s = np.zeros((1, 2)), np.ones((1, 2))
    assert np.array_equal(op.heads(x4, cos=c, sin=s)[0], [[[-3.0, -4.0, 1.0, 2.0]]])
    assert np.array_equal(op.heads(x4, cos=c, sin=s, interleaved=True)[0],
                          [[[-2.0, 1.0, -4.0, 3.0]]])
    # a query's product with a key depends on how far apart they are
    rs = np.random.default_rng(0)
    q, k = rs.standard_normal((2, 1, 1, 16))
    ang = op.angles(40, 16)
    turn = lambda v, p: op.heads(v, cos=np.cos(ang[p:p + 1]), sin=np.sin(ang[p:p + 1]))[0]  # noqa: E731
    assert np.isclose((turn(q, 5) * turn(k, 2)).sum(), (turn(q, 33) * turn(k, 30)).sum(), rtol=1e-12)


def test_logprobs_closed_forms():
    ninf = -np.inf
    lp, H, m1, m2 = op.logprobs(np.array([[0.0, 0.0, ninf, 0.0], [ninf] * 4, [1.0, np.nan, 0, 0],
                                          [1.0, np.inf, 0, 0], [2.0, 0.0, ninf, ninf]]),
                                scale=[1.0, 1.0, 1.0, 1.0, 0.5])
    assert np.allclose(lp[0, [0, 1, 3]], -math.log(3)) and lp[0, 2] == ninf
    assert np.isclose(H[0], math.log(3)) and H[1] == 0 and np.all(lp[1] == ninf)
    assert np.isnan(lp[2]).all() and np.isnan(H[2]) and np.isnan(lp[3]).all()
    p = 1 / (1 + math.exp(-1.0))
    assert np.isclose(lp[4, 0], math.log(p)) and np.isclose(m1[4], 1 - p) and np.isclose(m2[4], 1 - p)
    x = np.array([[1.0, 3.0, 3.0, ninf, 2.0], [ninf] * 5, [-0.0, 0.0, 0.0, 1.0, ninf]])
    assert op.best(x, 4).tolist() == [[1, 2, 4, 0], [-1] * 4, [3, 0, 1, 2]]
    rs = np.random.default_rng(1)
    x = rs.integers(0, 9, (2, 5000)).astype(float)
    assert op.best(x, 20).tolist() == [
        sorted(range(5000), key=lambda v: (-r[v], v))[:20] for r in x]


def test_adapters_definition():
    rs = np.random.default_rng(2)
    x, y = rs.standard_normal((3, 5)), rs.standard_normal((3, 4))
    A, B = rs.standard_normal((2, 5)), rs.standard_normal((4, 2))
    out = op.add_adapters(x, [0, -1, 1], [(A, B, 0.5), None], y)[0]
    assert np.allclose(out[0], y[0] + 0.5 * (B @ A) @ x[0], rtol=1e-13)
    assert np.array_equal(out[1:], y[1:])


# ------------------------------------------------------------------ tables and sizes

def test_rope_table():
    t = moeq.rope_table(131072, 64, device="cpu")
    assert t.shape == (131072, 64) and t.dtype == torch.float32
    ang = op.angles(131072, 64)
    assert np.abs(t[:, :32].numpy() - np.cos(ang)).max() <= 2.0 ** -25 + 1e-10
    assert np.abs(t[:, 32:].numpy() - np.sin(ang)).max() <= 2.0 ** -25 + 1e-10
    f = moeq.rope_table(10, 4, freq=[1.0, 0.25], scale=2.0, device="cpu").numpy()
    assert np.allclose(f[3], [2 * math.cos(3), 2 * math.cos(0.75), 2 * math.sin(3),
                              2 * math.sin(0.75)], rtol=1e-7)
    for args in ((0, 4), (4, 0), (4, 3)):
        with pytest.raises(ValueError):
            moeq.rope_table(*args, device="cpu")
    with pytest.raises(ValueError, match="freq"):
        moeq.rope_table(4, 4, freq=[1.0], device="cpu")


def test_sizes():
    L = moeq.lib()
    assert L.moe_token_logprobs_workspace_bytes(3, 16384, 5) == 3 * 56
    assert L.moe_token_logprobs_workspace_bytes(3, 16385, 0) == 3 * 2 * 16
    for bad in ((-1, 8, 0), (1, 0, 0), (1, 1048577, 0), (1, 8, 33), (1, 8, -1)):
        assert L.moe_token_logprobs_workspace_bytes(*bad) == 0
    assert L.moe_adapter_bytes(0, 17, 129, 5) == 2 * 8 * 1024
    assert L.moe_adapter_bytes(1, 17, 129, 65) == 2 * 2 * 2048
    for bad in ((2, 1, 1, 1), (0, 0, 1, 1), (0, 257, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0)):
        assert L.moe_adapter_bytes(*bad) == 0
    assert L.moe_adapter_plan_bytes(0, 1) > 0 and L.moe_adapter_plan_bytes(5, 1023) > 0
    for bad in ((-1, 1), (1, 0), (1, 1024), (1 << 31, 1)):
        assert L.moe_adapter_plan_bytes(*bad) == 0


# ------------------------------------------------------------------ refusals

def refused(name, *args, status=BAD, says=None):
    L = moeq.lib()
    got = getattr(L, name)(*args)
    detail = L.moe_last_error().decode()
    assert got == status, (name, got, detail)
    assert name in detail and (says is None or says in detail), detail


def head_set(**kw):
    d = dict(x=P, ld_t=256, ld_h=64, out=P + (1 << 20), ld_out_t=256, ld_out_h=64, w=P, heads=4)
    d.update(kw)
    return mh.HeadSetC(**d)


def heads(k=None, q=None, **kw):
    d = dict(pos=P, table=P, table_rows=8, D=64, R=64, pos_bits=32, dtype=2, w_dtype=2, eps=1e-5)
    d.update(kw)
    return ctypes.byref(mh.HeadsC(q=head_set(**(q or {})), k=head_set(**(k or {})), **d))


@pytest.mark.parametrize("kw,T,status,says", [
    ({}, -1, BAD, "T"),
    ({}, 1 << 31, BAD, "T"),
    (dict(D=0), 1, BAD, "D"),
    (dict(D=1025, k=dict(heads=0)), 1, UNSUPPORTED, "1024"),
    (dict(dtype=4), 1, UNSUPPORTED, "type"),
    (dict(w_dtype=0), 1, UNSUPPORTED, "weights"),
    (dict(eps=-1.0), 1, BAD, "eps"),
    (dict(eps=math.nan), 1, BAD, "eps"),
    (dict(w_offset=math.inf), 1, BAD, "w_offset"),
    (dict(q=dict(heads=-1)), 1, BAD, "q must have"),
    (dict(k=dict(heads=4097)), 1, BAD, "k must have"),
    (dict(q=dict(x=None)), 1, BAD, "null"),
    (dict(k=dict(out=None)), 1, BAD, "null"),
    (dict(q=dict(x=P + 1)), 1, BAD, "aligned"),
    (dict(k=dict(w=P + 1)), 1, BAD, "aligned"),
    (dict(q=dict(ld_t=-1)), 1, BAD, "strides"),
    (dict(q=dict(ld_out_h=63)), 1, BAD, "overlap"),
    (dict(q=dict(ld_out_t=255)), 2, BAD, "overlap"),
    (dict(q=dict(ld_out_t=64, ld_out_h=127)), 2, BAD, "overlap"),
    (dict(q=dict(out=P, ld_t=512)), 1, BAD, "in place"),
    (dict(pos_bits=16), 1, BAD, "pos_bits"),
    (dict(pos=P + 2), 1, BAD, "pos is"),
    (dict(pos=P + 4, pos_bits=64), 1, BAD, "pos is"),
    (dict(R=66), 1, BAD, "R must"),
    (dict(R=0), 1, BAD, "R must"),
    (dict(R=31), 1, BAD, "R must"),
    (dict(table=None), 1, BAD, "table"),
    (dict(table_rows=0), 1, BAD, "table"),
    (dict(table=P + 2), 1, BAD, "table"),
    (dict(pos=None, q=dict(w=None), k=dict(w=None)), 1, BAD, "neither"),
])
def test_head_refusals(kw, T, status, says):
    refused("moe_head_norm_rope", heads(**kw), T, None, status=status, says=says)


def logargs(**kw):
    d = dict(logits=P, ld=100, ids=P, logprob=P, entropy=P, top_ids=P, top_logprob=P, V=100, m=1,
             top=5, dtype=2, id_bits=32)
    d.update(kw)
    return ctypes.byref(mh.LogprobsC(**d))


@pytest.mark.parametrize("kw,T,ws,status,says", [
    ({}, -1, 1 << 20, BAD, "T"),
    (dict(V=0), 1, 1 << 20, BAD, "V"),
    (dict(V=1048577, ld=1048577), 1, 1 << 20, UNSUPPORTED, "1048576"),
    (dict(top=33), 1, 1 << 20, BAD, "32"),
    (dict(top=-1), 1, 1 << 20, BAD, "top"),
    (dict(m=1025), 1, 1 << 20, BAD, "m must"),
    (dict(m=-1), 1, 1 << 20, BAD, "m must"),
    (dict(logits=None), 1, 1 << 20, BAD, "logits"),
    (dict(logits=P + 1), 1, 1 << 20, BAD, "aligned"),
    (dict(ld=99), 1, 1 << 20, BAD, "stride"),
    (dict(dtype=4), 1, 1 << 20, UNSUPPORTED, "type"),
    (dict(ids=None), 1, 1 << 20, BAD, "go together"),
    (dict(m=0), 1, 1 << 20, BAD, "go together"),
    (dict(logprob=None), 1, 1 << 20, BAD, "go together"),
    (dict(id_bits=8), 1, 1 << 20, BAD, "id_bits"),
    (dict(ids=P + 4, id_bits=64), 1, 1 << 20, BAD, "ids is"),
    (dict(top=0), 1, 1 << 20, BAD, "top_ids"),
    (dict(top_ids=None), 1, 1 << 20, BAD, "top_ids"),
    (dict(ids=None, m=0, logprob=None, entropy=None, top=0, top_ids=None, top_logprob=None), 1,
     1 << 20, BAD, "no output"),
    ({}, 2, 111, WORKSPACE, "112"),
])
def test_logprob_refusals(kw, T, ws, status, says):
    refused("moe_token_logprobs", logargs(**kw), T, P, ws, None, status=status, says=says)


def test_logprob_workspace_refusals():
    refused("moe_token_logprobs", logargs(), 1, None, 1 << 20, None, status=WORKSPACE)
    refused("moe_token_logprobs", logargs(), 1, P + 16, 1 << 20, None, says="256")


def adapters(**kw):
    d = dict(n=4, rank=16, K=64, N=32, w_dtype=2, a=P, b=P, ranks=P, scales=P)
    d.update(kw)
    return ctypes.byref(ma.AdaptersC(**d))


@pytest.mark.parametrize("kw,status", [
    (dict(n=0), BAD), (dict(n=1024), BAD), (dict(rank=0), BAD), (dict(rank=257), BAD),
    (dict(K=0), BAD), (dict(N=0), BAD), (dict(w_dtype=1), UNSUPPORTED),
    (dict(w_dtype=4), UNSUPPORTED), (dict(a=None), BAD), (dict(b=P + 8), BAD),
    (dict(ranks=None), BAD), (dict(scales=None), BAD)])
def test_adapter_set_refusals(kw, status):
    refused("moe_pack_adapter", adapters(**kw), 0, P, 64, P, 16, 16, 1.0, None, status=status)
    refused("moe_add_adapters", adapters(**kw), P, 2, 64, None, P, 1, P, 32, P, 32, 2, P, 1 << 20,
            None, status=status)


@pytest.mark.parametrize("args,says", [
    ((-1, P, 64, P, 16, 16, 1.0), "slot"),
    ((4, P, 64, P, 16, 16, 1.0), "slot"),
    ((0, P, 64, P, 16, 17, 1.0), "rank"),
    ((0, P, 64, P, 16, -1, 1.0), "rank"),
    ((0, P, 64, P, 16, 16, math.inf), "scale"),
    ((0, None, 64, P, 16, 16, 1.0), "null"),
    ((0, P, 63, P, 16, 16, 1.0), "stride"),
    ((0, P, 64, P, 15, 16, 1.0), "stride"),
    ((0, P + 1, 64, P, 16, 16, 1.0), "aligned")])
def test_pack_adapter_refusals(args, says):
    refused("moe_pack_adapter", adapters(), *args, None, says=says)


@pytest.mark.parametrize("args,status,says", [
    ((P, 2, 64, None, P, -1, P, 32, P, 32, 2, P, 1 << 20), BAD, "T"),
    ((None, 2, 64, None, P, 1, P, 32, P, 32, 2, P, 1 << 20), BAD, "null"),
    ((P, 2, 64, None, None, 1, P, 32, P, 32, 2, P, 1 << 20), BAD, "null"),
    ((P, 2, 64, None, P, 1, None, 32, P, 32, 2, P, 1 << 20), BAD, "null"),
    ((P, 2, 64, None, P, 1, P, 32, None, 32, 2, P, 1 << 20), BAD, "null"),
    ((P, 3, 64, None, P, 1, P, 32, P, 32, 2, P, 1 << 20), UNSUPPORTED, "type"),
    ((P, 1, 64, None, P, 1, P, 32, P, 32, 2, P, 1 << 20), UNSUPPORTED, "type"),
    ((P, 2, 63, None, P, 1, P, 32, P, 32, 2, P, 1 << 20), BAD, "stride of x"),
    ((P, 2, 64, P, P, 1, P, 32, P, 32, 2, P, 1 << 20), BAD, "x_scale"),
    ((P, 4, 64, None, P, 1, P, 32, P, 32, 2, P, 1 << 20), BAD, "x_scale"),
    ((P, 4, 60, P, P, 1, P, 32, P, 32, 2, P, 1 << 20), BAD, "64 codes"),
    ((P, 2, 64, None, P, 1, P, 31, P, 32, 2, P, 1 << 20), BAD, "stride of y"),
    ((P, 2, 64, None, P, 1, P, 32, P + 64, 31, 2, P, 1 << 20), BAD, "stride of out"),
    ((P, 2, 64, None, P, 1, P, 32, P, 40, 2, P, 1 << 20), BAD, "in place"),
    ((P, 2, 64, None, P, 1, P, 32, P, 32, 4, P, 1 << 20), UNSUPPORTED, "type"),
    ((P, 2, 64, None, P + 4, 1, P, 32, P, 32, 2, P, 1 << 20), BAD, "plan"),
    ((P, 2, 64, None, P, 1, P, 32, P, 32, 2, None, 1 << 20), WORKSPACE, "256"),
    ((P, 2, 64, None, P, 5, P, 32, P, 32, 2, P, 511), WORKSPACE, "512"),
    ((P, 2, 64, None, P, 1, P, 32, P, 32, 2, P + 16, 1 << 20), BAD, "256"),
])
def test_add_adapters_refusals(args, status, says):
    refused("moe_add_adapters", adapters(), *args, None, status=status, says=says)


@pytest.mark.parametrize("n", [1, 8, 33, 1023])
@pytest.mark.parametrize("rank,K", [(16, 100), (32, 4096), (64, 6144), (256, 512)])
def test_bytes_never_fall_with_the_tokens(n, rank, K):
    s = ma.AdaptersC(n=n, rank=rank, K=K, N=64)
    Ts = list(range(1, 1100)) + list(range(1100, 9000, 61)) + [n * 32 - 1, n * 32, 40000]
    Ts.sort()
    L = moeq.lib()
    plans = [L.moe_adapter_plan_bytes(T, n) for T in Ts]
    spaces = [L.moe_add_adapters_workspace_bytes(ctypes.byref(s), T) for T in Ts]
    assert plans == sorted(plans) and spaces == sorted(spaces)


@pytest.mark.parametrize("n", [1, 8, 64, 300, 1023])
def test_bytes_never_fall_where_the_sort_changes(n):
    """Around the token counts at which the sort of a large plan, its tiles or the dispatch of
    the products change: multiples of 65536 and of 32 slots, and sizes spread up to 2^31."""
    s = ma.AdaptersC(n=n, rank=64, K=6144, N=64)
    Ts = {(1 << 31) - 4097}
    for base in [*range(0, 20 << 16, 1 << 16), 1024, 4096, 32 * n, *(1 << i for i in range(21, 31))]:
        Ts.update(range(max(1, base - 3), base + 4))
    T = 1
    while T < (1 << 31) - 4096:
        Ts.add(T)
        T += T // 97 + 1
    Ts = sorted(Ts)
    L = moeq.lib()
    plans = [L.moe_adapter_plan_bytes(T, n) for T in Ts]
    spaces = [L.moe_add_adapters_workspace_bytes(ctypes.byref(s), T) for T in Ts]
    assert plans[0] and plans == sorted(plans) and spaces == sorted(spaces)


def test_plan_refusals():
    for T, n in ((-1, 1), (1, 0), (1, 1024), (1 << 31, 1)):
        refused("moe_adapter_plan", P, T, n, P, 1 << 20, None)
    refused("moe_adapter_plan", None, 1, 1, P, 1 << 20, None, says="null")
    refused("moe_adapter_plan", P, 1, 1, None, 1 << 20, None, says="null")
    refused("moe_adapter_plan", P + 2, 1, 1, P, 1 << 20, None, says="ids")
    refused("moe_adapter_plan", P, 1, 1, P + 8, 1 << 20, None, says="16")
    refused("moe_adapter_plan", P, 1, 1, P, 8, None, status=WORKSPACE)


def test_nothing_to_do():
    L = moeq.lib()
    assert L.moe_head_norm_rope(heads(), 0, None) == 0
    assert L.moe_head_norm_rope(heads(q=dict(heads=0), k=dict(heads=0)), 3, None) == 0
    assert L.moe_token_logprobs(logargs(), 0, None, 0, None) == 0
    assert L.moe_adapter_plan(None, 0, 1, None, 0, None) == 0
    assert L.moe_add_adapters(adapters(), None, 2, 64, None, None, 0, None, 32, None, 32, 2, None, 0,
                              None) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros((2, 3, 64))
    for call in (lambda: moeq.head_norm_rope(x, q_w=torch.ones(64)),
                 lambda: moeq.token_logprobs(x[0]),
                 lambda: moeq.adapter_plan(torch.zeros(2, dtype=torch.int32), 1)):
        with pytest.raises(ValueError, match="device"):
            call()
    with pytest.raises(ValueError, match="bf16 or fp16"):
        moeq.Adapters(1, 8, 64, 64, dtype=torch.float32, device="cpu")
    for kw in (dict(n=0), dict(n=1024), dict(rank=257), dict(K=0)):
        with pytest.raises(ValueError):
            moeq.Adapters(**{**dict(n=1, rank=8, K=64, N=64), **kw}, device="cpu")
    s = moeq.Adapters(2, 8, 64, 64, device="cpu")
    with pytest.raises(ValueError, match="device"):
        s.load(0, torch.zeros((8, 64), dtype=torch.bfloat16), torch.zeros((64, 8)))
    with pytest.raises(ValueError, match="device"):
        moeq.add_adapters(s, x[0], None, x[0])


def test_head_set_checks():
    x = torch.zeros((2, 3, 8))
    check = lambda x, w, o: mh._head_set(x, "q", w, o, 2, 8, -1, torch.float32, torch.float32)  # noqa: E731
    ok, out = check(x[:, 1:], None, None)
    assert ok[1:3] == (24, 8) and out.shape == (2, 2, 8)
    for bad, w, o, says in ((x[0], None, None, "must be"), (x.transpose(1, 2), None, None, "must be"),
                            (torch.zeros(2, 8, 3).transpose(1, 2), None, None, "side by side"),
                            (x, torch.zeros(7), None, "q_w"), (x, torch.zeros(8).half(), None, "q_w"),
                            (x, None, torch.zeros(2, 3, 9), "q_out"),
                            (x, None, torch.zeros(2, 3, 8).half(), "q_out")):
        with pytest.raises(ValueError, match=says):
            check(bad, w, o)
    with pytest.raises(ValueError, match="pos"):
        mh._whole(torch.zeros(3), "pos", (3,), -1)
    assert mh._whole(torch.zeros(3, dtype=torch.int64), "pos", (3,), -1)[1] == 64
    assert ma._pitch(x[0][:, 2:6], "y", 3, 4) == 8 and ma._pitch(x[0][:1, :4], "y", 1, 4) == 8
    with pytest.raises(ValueError, match="side by side"):
        ma._pitch(x[0].t(), "y", 8, 3)
