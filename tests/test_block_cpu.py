"""CPU tests of the block norms and the 8-bit products: the oracle's pins and
the refusals of the C calls and the binding (nothing is launched)."""

import ctypes

import numpy as np
import pytest
import torch

import bit_quantized_moe_route_amd as moeq
from bit_quantized_moe_route_amd import block as mb
from oracle import block as ob

P = 1 << 20        # an aligned address no refused call ever reads


# ------------------------------------------------------------------ oracle

def test_rms_norm_closed_forms():
    v = np.array([[3.0, -4.0], [0.0, 0.0], [1.0, 1.0]])
    n, _ = ob.rms_norm(v, [2.0, 1.0], 0.5)
    assert np.allclose(n[0], np.array([6.0, -4.0]) / np.sqrt(13.0), rtol=1e-15)
    assert np.all(n[1] == 0) and np.allclose(n[2], np.array([2.0, 1.0]) / np.sqrt(1.5), rtol=1e-15)
    # a norm takes no notice of its input's scale, and w_offset is added to w
    rs = np.random.default_rng(0)
    x, w = rs.standard_normal((4, 33)), rs.standard_normal(33)
    assert np.allclose(ob.rms_norm(x, w, 0)[0], ob.rms_norm(x * 1e3, w, 0)[0], rtol=1e-12)
    assert np.allclose(ob.rms_norm(x, w, 0, 1.0)[0], ob.rms_norm(x, w + 1, 0)[0], rtol=1e-12)
    t = torch.nn.functional.rms_norm(torch.from_numpy(x), (33,), torch.from_numpy(w), 1e-5)
    assert np.allclose(ob.rms_norm(x, w, 1e-5)[0], t.numpy(), rtol=1e-12)


def test_block_steps():
    rs = np.random.default_rng(1)
    T, H, k = 3, 8, 2
    yp = rs.standard_normal((T * k, H))
    inv = rs.permutation(T * k).astype(np.int32)
    w = rs.random((T, k))
    b, mag = ob.gated_sum(yp, inv, w)
    for t in range(T):
        want = sum(w[t, j] * yp[inv[t * k + j]] for j in range(k))
        assert np.allclose(b[t], want, rtol=1e-14)
    assert np.all(mag >= np.abs(b) - 1e-15)
    r, g = rs.standard_normal((T, H)), rs.random((T, 1))
    r1, _, n, _ = ob.block(r, b, np.ones(H), None, g, 0.5, 2.0)
    assert np.allclose(r1, 2 * r + 0.5 * g * b, rtol=1e-14)
    assert np.allclose(n, ob.rms_norm(r1, np.ones(H), 1e-5)[0], rtol=1e-14)
    assert np.array_equal(ob.block(r, None)[0], r)


def test_quantize_properties():
    rs = np.random.default_rng(2)
    x = (rs.standard_normal((50, 40)) * 10.0 ** rs.integers(-30, 30, (50, 1))).astype(np.float32)
    x[7] = 0
    q, s = ob.quantize_i8(x)
    a = np.abs(x.astype(np.float64)).max(1)
    live = a > 127 * 2.0 ** -126
    assert np.all(np.abs(q).max(1)[live] == 127) and not q[~live].any() and not s[~live].any()
    err = np.abs(q * s[:, None].astype(np.float64) - x)
    assert np.all(err[live] <= 0.5 * s[live, None] * (1 + 2.0 ** -16))
    q2, s2 = ob.quantize_i8(np.array([[1, np.nan], [np.inf, 1], [-np.inf, 0]], np.float32))
    assert not q2.any() and np.isnan(s2).all()


def test_expert_against_dense_form():
    rs = np.random.default_rng(3)
    H, I, R = 24, 16, 5
    w13, w2 = rs.integers(-128, 128, (2 * I, H)), rs.integers(-128, 128, (H, I))
    s13, s2 = rs.random(2 * I) * 0.01, rs.random(H) * 0.01
    x = rs.standard_normal((R, H)).astype(np.float32)
    q, s = ob.quantize_i8(x)
    y, slack, near = ob.expert_i8(q, s, w13, s13, w2, s2, 0.0)
    for i in range(R):
        h = np.empty(I)
        for c in range(I):
            g = s[i] * s13[c] * sum(int(a) * int(b) for a, b in zip(q[i], w13[c]))
            u = s[i] * s13[I + c] * sum(int(a) * int(b) for a, b in zip(q[i], w13[I + c]))
            h[c] = g / (1 + np.exp(-g)) * u
        step = np.abs(h).max() / 127
        want = [step * s2[n] * sum(np.rint(h[c] / step) * w2[n, c] for c in range(I))
                for n in range(H)]
        assert np.allclose(y[i], want, rtol=1e-9, atol=1e-12)
    assert slack.max() == 0 and near == 0


# ------------------------------------------------------------------ refusals

def refused(name, *args, status=moeq.MOE_EINVAL, says=None):
    L = moeq.lib()
    got = getattr(L, name)(*args)
    detail = L.moe_last_error().decode()
    assert got == status, (name, got, detail)
    assert name in detail and (says is None or says in detail), detail


def good_block(**kw):
    d = dict(r=P, ld_r=64, r_dtype=2, pre_w=P, w_dtype=2, n_out=P, ld_n=64, n_dtype=2, y_scale=1.0,
             r_scale=1.0, eps=1e-5)
    d.update(kw)
    return mb.BlockC(**d)


@pytest.mark.parametrize("kw,T,H,status,says", [
    ({}, -1, 64, moeq.MOE_EINVAL, "T"),
    ({}, 1 << 31, 64, moeq.MOE_EINVAL, "T"),
    ({}, 1, 0, moeq.MOE_EINVAL, "H"),
    ({}, 1, 32769, moeq.MOE_EUNSUPPORTED, "32768"),
    (dict(r=None), 1, 64, moeq.MOE_EINVAL, "neither"),
    (dict(n_out=None), 1, 64, moeq.MOE_EINVAL, "output"),
    (dict(post_w=P), 1, 64, moeq.MOE_EINVAL, "need y"),
    (dict(gate=P, gate_dtype=2, gate_ld_h=1), 1, 64, moeq.MOE_EINVAL, "need y"),
    (dict(y=P, ld_y=64, y_dtype=2, gate=P, gate_dtype=2, gate_ld_h=2), 1, 64, moeq.MOE_EINVAL,
     "gate_ld_h"),
    (dict(y=P, ld_y=64, y_dtype=2, gate=P, gate_dtype=2, gate_ld_t=-1), 1, 64, moeq.MOE_EINVAL,
     "gate_ld_t"),
    (dict(y=P, ld_y=64, y_dtype=2, gate=P, gate_dtype=2, gate_ld_t=32, gate_ld_h=1), 1, 64,
     moeq.MOE_EINVAL, "gate"),
    (dict(y=P, ld_y=64, y_dtype=2, gate=P, gate_dtype=9), 1, 64, moeq.MOE_EUNSUPPORTED, "gate"),
    (dict(y=P, ld_y=64, y_dtype=2, k=17), 1, 64, moeq.MOE_EINVAL, "k"),
    (dict(y=P, ld_y=64, y_dtype=2, k=2), 1, 64, moeq.MOE_EINVAL, "inv_perm"),
    (dict(y=P, ld_y=64, y_dtype=2, inv_perm=P), 1, 64, moeq.MOE_EINVAL, "inv_perm"),
    (dict(y=P, ld_y=64, y_dtype=2, y_shared=P, ld_y_shared=64, y_shared_dtype=2), 1, 64,
     moeq.MOE_EINVAL, "y_shared"),
    (dict(y=P, ld_y=64, y_dtype=2, shared_gate=P), 1, 64, moeq.MOE_EINVAL, "shared_gate"),
    (dict(y=P, ld_y=64, y_dtype=2, k=16, inv_perm=P, topk_w=P), 1 << 28, 64, moeq.MOE_EINVAL,
     "T*k"),
    (dict(y=P, ld_y=64, y_dtype=4), 1, 64, moeq.MOE_EUNSUPPORTED, "y"),
    (dict(r_dtype=0), 1, 64, moeq.MOE_EUNSUPPORTED, "r "),
    (dict(ld_r=63), 1, 64, moeq.MOE_EINVAL, "stride of r"),
    (dict(ld_n=63), 1, 64, moeq.MOE_EINVAL, "stride of n_out"),
    (dict(r=P + 1), 1, 64, moeq.MOE_EINVAL, "aligned"),
    (dict(pre_w=P + 2, w_dtype=1), 1, 64, moeq.MOE_EINVAL, "aligned"),
    (dict(q_out=P), 1, 64, moeq.MOE_EINVAL, "together"),
    (dict(q_scale=P), 1, 64, moeq.MOE_EINVAL, "together"),
    (dict(q_out=P, q_scale=P, ld_q=48), 1, 48, moeq.MOE_EINVAL, "q_out"),
    (dict(q_out=P, q_scale=P, ld_q=72), 1, 64, moeq.MOE_EINVAL, "q_out"),
    (dict(q_out=P + 8, q_scale=P, ld_q=64), 1, 64, moeq.MOE_EINVAL, "q_out"),
    (dict(eps=-1.0), 1, 64, moeq.MOE_EINVAL, "eps"),
    (dict(eps=float("nan")), 1, 64, moeq.MOE_EINVAL, "eps"),
    (dict(r_scale=float("inf")), 1, 64, moeq.MOE_EINVAL, "finite"),
])
def test_block_norm_refusals(kw, T, H, status, says):
    refused("moe_block_norm", ctypes.byref(good_block(**kw)), T, H, None, status=status, says=says)


def test_null_descriptors():
    refused("moe_block_norm", None, 1, 64, None)
    refused("moe_linear_i8", None, P, 2, 64, None, 1, P, 2, 16, P, 1 << 20, None)
    refused("moe_expert_ffn_i8", None, P, 2, 64, None, P, P, 1, 1, P, 2, P, 1 << 20, None)
    refused("moe_shared_ffn_i8", None, P, 2, 64, None, 1, P, 2, P, 1 << 20, None)


@pytest.mark.parametrize("args,status", [
    ((P, 2, 64, -1, 64, P, 64, P), moeq.MOE_EINVAL),
    ((P, 2, 64, 1, 0, P, 64, P), moeq.MOE_EINVAL),
    ((None, 2, 64, 1, 64, P, 64, P), moeq.MOE_EINVAL),
    ((P, 2, 64, 1, 64, None, 64, P), moeq.MOE_EINVAL),
    ((P, 2, 64, 1, 64, P, 64, None), moeq.MOE_EINVAL),
    ((P, 4, 64, 1, 64, P, 64, P), moeq.MOE_EUNSUPPORTED),
    ((P, 2, 63, 1, 64, P, 64, P), moeq.MOE_EINVAL),
    ((P + 1, 2, 64, 1, 64, P, 64, P), moeq.MOE_EINVAL),
    ((P, 2, 65, 1, 65, P, 64, P), moeq.MOE_EINVAL),
    ((P, 2, 64, 1, 64, P, 72, P), moeq.MOE_EINVAL),
    ((P, 2, 64, 1, 64, P + 4, 64, P), moeq.MOE_EINVAL),
])
def test_quantize_refusals(args, status):
    refused("moe_quantize_i8", *args, None, status=status)


def test_matrix_sizes_and_pack_refusals():
    L = moeq.lib()
    assert L.moe_i8_matrix_bytes(16, 64) == 2048 and L.moe_i8_matrix_bytes(17, 129) == 8192
    assert L.moe_i8_record_bytes(0, 65, 17) == 2 * 4096 and L.moe_i8_record_bytes(1, 17, 129) == 8192
    for n, k in ((0, 64), (16, 0), (16, 131072), ((1 << 24) + 1, 64)):
        assert L.moe_i8_matrix_bytes(n, k) == 0
    assert L.moe_i8_record_bytes(2, 64, 64) == 0 and L.moe_i8_record_bytes(0, 64, 131072) == 0
    refused("moe_pack_i8", P, 64, 0, 64, P, None)
    refused("moe_pack_i8", P, 63, 16, 64, P, None)
    refused("moe_pack_i8", None, 64, 16, 64, P, None)
    refused("moe_pack_i8", P, 64, 16, 64, P + 8, None)
    refused("moe_pack_i8_expert", P, P, P, 0, 16, P, P, None)
    refused("moe_pack_i8_expert", P, P, None, 16, 16, P, P, None)
    refused("moe_pack_i8_expert", P, P, P, 16, 16, P + 8, P, None)


def test_calls_past_one_launch_are_refused():
    """Products of 2^32 threads and more, and a matrix of 64 GiB."""
    refused("moe_pack_i8", P, 1 << 12, 1 << 24, 1 << 12, P, None, status=moeq.MOE_EUNSUPPORTED)
    refused("moe_linear_i8", lin(N=1 << 16), P, 4, 64, P, 1 << 24, P, 2, 1 << 16, None, 0, None,
            status=moeq.MOE_EUNSUPPORTED, says="too many")
    refused("moe_expert_ffn_i8", lay(H=1 << 16, I=64, w13_stride=1 << 24, w2_stride=1 << 24), P, 2,
            1 << 16, None, P, P, 1 << 23, 4, P, 2, P, 1 << 20, None, status=moeq.MOE_EUNSUPPORTED,
            says="too many")


def lin(**kw):
    d = dict(N=32, K=64, w=P, w_scale=P)
    d.update(kw)
    return ctypes.byref(mb.I8LinearC(**d))


@pytest.mark.parametrize("desc,args,status", [
    (dict(N=0), (P, 2, 64, None, 1, P, 2, 32, P, 1 << 20), moeq.MOE_EINVAL),
    (dict(K=131072), (P, 2, 131072, None, 1, P, 2, 32, P, 1 << 20), moeq.MOE_EUNSUPPORTED),
    (dict(w=None), (P, 2, 64, None, 1, P, 2, 32, P, 1 << 20), moeq.MOE_EINVAL),
    (dict(w=P + 8), (P, 2, 64, None, 1, P, 2, 32, P, 1 << 20), moeq.MOE_EINVAL),
    (dict(w_scale=None), (P, 2, 64, None, 1, P, 2, 32, P, 1 << 20), moeq.MOE_EINVAL),
    ({}, (P, 2, 64, None, -1, P, 2, 32, P, 1 << 20), moeq.MOE_EINVAL),
    ({}, (None, 2, 64, None, 1, P, 2, 32, P, 1 << 20), moeq.MOE_EINVAL),
    ({}, (P, 2, 64, None, 1, None, 2, 32, P, 1 << 20), moeq.MOE_EINVAL),
    ({}, (P, 2, 64, None, 1, P, 4, 32, P, 1 << 20), moeq.MOE_EUNSUPPORTED),
    ({}, (P, 2, 64, None, 1, P, 2, 31, P, 1 << 20), moeq.MOE_EINVAL),
    ({}, (P, 2, 64, None, 1, P + 1, 2, 32, P, 1 << 20), moeq.MOE_EINVAL),
    ({}, (P, 2, 63, None, 1, P, 2, 32, P, 1 << 20), moeq.MOE_EINVAL),
    ({}, (P, 7, 64, None, 1, P, 2, 32, P, 1 << 20), moeq.MOE_EUNSUPPORTED),
    ({}, (P, 2, 64, P, 1, P, 2, 32, P, 1 << 20), moeq.MOE_EINVAL),
    ({}, (P, 4, 64, None, 1, P, 2, 32, None, 0), moeq.MOE_EINVAL),
    ({}, (P, 4, 48, P, 1, P, 2, 32, None, 0), moeq.MOE_EINVAL),
    ({}, (P + 4, 4, 64, P, 1, P, 2, 32, None, 0), moeq.MOE_EINVAL),
    ({}, (P, 2, 64, None, 1, P, 2, 32, None, 0), moeq.MOE_EWORKSPACE),
    ({}, (P, 2, 64, None, 1, P, 2, 32, P, 64), moeq.MOE_EWORKSPACE),
    ({}, (P, 2, 64, None, 1, P, 2, 32, P + 16, 1 << 20), moeq.MOE_EINVAL),
    (dict(N=1 << 24), (P, 4, 64, P, 1 << 24, P, 2, 1 << 24, None, 0), moeq.MOE_EUNSUPPORTED),
])
def test_linear_refusals(desc, args, status):
    refused("moe_linear_i8", lin(**desc), *args, None, status=status)


def lay(**kw):
    d = dict(E=4, H=64, I=32, w13=P, w13_stride=8192, w2=P, w2_stride=8192, w13_scale=P,
             w2_scale=P)
    d.update(kw)
    return ctypes.byref(mb.I8LayerC(**d))


@pytest.mark.parametrize("desc", [dict(E=0), dict(E=1025), dict(H=0), dict(I=0), dict(w13=None),
                                  dict(w2_scale=None), dict(w13=P + 4), dict(w2_stride=4104),
                                  dict(w13_stride=4096), dict(w2_stride=4096)])
def test_layer_refusals(desc):
    refused("moe_expert_ffn_i8", lay(**desc), P, 2, 64, None, P, P, 1, 1, P, 2, P, 1 << 20, None)
    if "E" not in desc:
        refused("moe_shared_ffn_i8", lay(**dict(desc, E=1)), P, 2, 64, None, 1, P, 2, P, 1 << 20,
                None)


@pytest.mark.parametrize("args,status", [
    ((P, 2, 64, None, P, P, -1, 1, P, 2, P, 1 << 20), moeq.MOE_EINVAL),
    ((P, 2, 64, None, P, P, 1, 0, P, 2, P, 1 << 20), moeq.MOE_EINVAL),
    ((P, 2, 64, None, P, P, 1, 5, P, 2, P, 1 << 20), moeq.MOE_EINVAL),
    ((P, 2, 64, None, P, P, 1 << 30, 2, P, 2, P, 1 << 20), moeq.MOE_EINVAL),
    ((P, 2, 64, None, None, P, 1, 1, P, 2, P, 1 << 20), moeq.MOE_EINVAL),
    ((P, 2, 64, None, P, None, 1, 1, P, 2, P, 1 << 20), moeq.MOE_EINVAL),
    ((P, 2, 64, None, P, P, 1, 1, None, 2, P, 1 << 20), moeq.MOE_EINVAL),
    ((P, 2, 64, None, P, P, 1, 1, P, 0, P, 1 << 20), moeq.MOE_EUNSUPPORTED),
    ((P, 2, 64, None, P, P, 1, 1, P + 1, 2, P, 1 << 20), moeq.MOE_EINVAL),
    ((P, 2, 63, None, P, P, 1, 1, P, 2, P, 1 << 20), moeq.MOE_EINVAL),
    ((P, 4, 64, None, P, P, 1, 1, P, 2, P, 1 << 20), moeq.MOE_EINVAL),
    ((P, 2, 64, None, P, P, 1, 1, P, 2, None, 1 << 20), moeq.MOE_EWORKSPACE),
    ((P, 2, 64, None, P, P, 1, 1, P, 2, P, 256), moeq.MOE_EWORKSPACE),
    ((P, 2, 64, None, P, P, 1, 1, P, 2, P + 16, 1 << 20), moeq.MOE_EINVAL),
])
def test_expert_ffn_refusals(args, status):
    refused("moe_expert_ffn_i8", lay(), *args, None, status=status)


def test_shared_ffn_needs_one_expert():
    refused("moe_shared_ffn_i8", lay(), P, 2, 64, None, 1, P, 2, P, 1 << 20, None, says="E == 1")


def test_nothing_to_do():
    """T = 0 is valid and launches nothing."""
    L = moeq.lib()
    assert L.moe_block_norm(ctypes.byref(good_block()), 0, 64, None) == 0
    assert L.moe_quantize_i8(None, 2, 64, 0, 64, None, 64, None, None) == 0
    assert L.moe_linear_i8(lin(), None, 2, 64, None, 0, None, 2, 32, None, 0, None) == 0
    assert L.moe_expert_ffn_i8(lay(), None, 2, 64, None, None, None, 0, 1, None, 2, None, 0,
                               None) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device"):
        moeq.block_norm(x, torch.ones(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="device"):
        moeq.quantize_i8(x)
    with pytest.raises(ValueError, match="device"):
        moeq.I8Linear(torch.zeros((16, 64), dtype=torch.int8), torch.ones(16))
    with pytest.raises(ValueError, match="device"):
        moeq.I8Layer(torch.zeros((1, 32, 64), dtype=torch.int8), torch.ones(1, 32),
                     torch.zeros((1, 64, 16), dtype=torch.int8), torch.ones(1, 64))


def test_row_checks():
    t = torch.zeros((4, 10))
    dev = t.device
    assert mb._rows(t, "t", 4, 10, dev) == 10
    assert mb._rows(t[:, 2:8], "t", 4, 6, dev) == 10
    assert mb._rows(t[::2], "t", 2, 10, dev) == 20
    assert mb._rows(t[:1, :3], "t", 1, 3, dev) == 3
    for bad in (t.t(), t[:, ::2], t[0]):
        with pytest.raises(ValueError):
            mb._rows(bad, "t", bad.shape[0], bad.shape[-1], dev)
    with pytest.raises(ValueError):
        mb._rows(t, "t", 4, 9, dev)
    with pytest.raises(ValueError):
        mb._rows(t, "t", 4, 10, dev, torch.bfloat16)
    with pytest.raises(ValueError, match="fp32, bf16 or fp16"):
        mb._dt(torch.float64)
    assert [mb.codes_width(k) for k in (1, 64, 65, 6144)] == [64, 64, 128, 6144]


def test_function_table_is_replaced_whole():
    """A thread that looked the table up keeps a whole one while another binds."""
    first = mb._bind(moeq.lib())
    names = set(first)
    second = mb._bind(moeq.lib())
    assert second is not first and set(first) == names == set(second)
    assert mb._fns is second and first["lib"] is moeq.lib()


def test_code_outputs_need_codes():
    r, w = torch.zeros((2, 64)), torch.ones(64)
    for kw in (dict(q=torch.zeros((2, 64), dtype=torch.int8)), dict(scale=torch.zeros(2))):
        with pytest.raises(ValueError, match="codes=True"):
            mb._block(r.device, 2, 64, r, None, w, 0, None, None, None, None, None, None, 1.0, 1.0,
                      1e-5, 0.0, None, None, None, False, kw.get("q"), kw.get("scale"))
