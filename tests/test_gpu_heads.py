"""GPU parity of the head norms with rotation (moe_head_norm_rope) against the fp64
oracle.

Tolerance, from the kernel's arithmetic: a sum of squares adds at most 16 values of
a thread and 6 lane stages, each rounding 2^-24, and enters as a square root (half);
the norm's other steps are 6 roundings, a rotation's 3, the table's entries half a
step each.  2^-19 of the sum of the terms' magnitudes covers them; half a step of the
type comes on top.
"""

import numpy as np
import pytest
import torch

import bit_quantized_moe_route_amd as moeq
from oracle import project as op
from tests.gpu_common import say

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
REL32 = 2.0 ** -19


def rnd(rs, shape, dtype, scale=1.0):
    return torch.from_numpy((rs.standard_normal(shape) * scale).astype(np.float32)).to(dtype).to(DEV)


def f64(t):
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def close(got, ref, mag, what):
    half = torch.finfo(got.dtype).eps / 2
    tol = half * np.abs(ref) + (1 + half) * REL32 * mag + TINY[got.dtype]
    err = np.abs(f64(got) - ref)
    assert np.all(err <= tol), (what, float(np.nanmax(err / tol)))


def cos_sin(pos, R, P):
    a = op.angles(P, R)[pos]
    return np.cos(a), np.sin(a)


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,R", [
    (1, 64, 8, 128, 128), (3, 5, 1, 64, 32), (2, 3, 2, 80, 32), (5, 4, 4, 192, 64),
    (2, 2, 1, 1024, 1024), (2, 3, 1, 1024, 16), (4, 7, 3, 36, 20), (2, 2, 2, 260, 260),
    (2, 1, 1, 516, 4), (1, 1, 1, 2, 2), (2, 3, 1, 1, 0), (3, 5, 2, 33, 30), (2, 2, 1, 131, 130),
    (2, 2, 1, 258, 6), (1, 2, 1, 1023, 1022), (2, 9, 2, 16, 16), (700, 16, 4, 64, 64),
    (900, 9, 5, 66, 26), (1500, 3, 1, 512, 500)])
def test_heads(T, Hq, Hk, D, R, inter, dt):
    say("heads", T, Hq, Hk, D, R, inter, dt)
    rs = np.random.default_rng(T * 7 + D)
    dtype, P = TYPES[dt], 5000
    q, k = rnd(rs, (T, Hq, D), dtype, 3.0), rnd(rs, (T, Hk, D), dtype)
    qw, kw = rnd(rs, (D,), dtype), rnd(rs, (D,), dtype)
    pos = rs.integers(0, P, T)
    rope = {}
    c = s = None
    if R:
        rope = dict(pos=torch.from_numpy(pos).to(DEV), table=moeq.rope_table(P, R),
                    interleaved=inter)
        c, s = cos_sin(pos, R, P)
    qo, ko = moeq.head_norm_rope(q, k, qw, kw, eps=1e-5, w_offset=0.5, **rope)
    for x, w, o in ((q, qw, qo), (k, kw, ko)):
        close(o, *op.heads(f64(x), f64(w), 1e-5, 0.5, c, s, inter), "norm and rotation")
    if not R:
        return
    # one of the two only, 32-bit positions, queries alone, in place: the same bits
    rope["pos"] = rope["pos"].int()
    again = q.clone()
    got, none = moeq.head_norm_rope(again, None, qw, w_offset=0.5, q_out=again, **rope)
    assert got is again and none is None and torch.equal(again, qo)
    plain = moeq.head_norm_rope(q, k, None, None, **rope)
    for x, o in ((q, plain[0]), (k, plain[1])):
        close(o, *op.heads(f64(x), None, cos=c, sin=s, interleaved=inter), "rotation")
    half = moeq.head_norm_rope(q, k, qw, None, eps=1e-5, w_offset=0.5, **rope)
    assert torch.equal(half[0], qo) and torch.equal(half[1], plain[1])
    normed = moeq.head_norm_rope(q, k, qw, kw)
    for x, w, o in ((q, qw, normed[0]), (k, kw, normed[1])):
        close(o, *op.heads(f64(x), f64(w)), "norm")


def test_far_positions():
    """Angles of positions far out, and of a table with its own frequencies."""
    rs = np.random.default_rng(0)
    P, D = 1 << 20, 128
    q = rnd(rs, (4, 2, D), torch.float32)
    pos = np.array([P - 1, 0, P // 2 + 1, 777777])
    table = moeq.rope_table(P, D, 500000.0)
    a = op.angles(P, D, 500000.0)[pos]
    got, _ = moeq.head_norm_rope(q, pos=torch.from_numpy(pos).to(DEV), table=table)
    # cosines and sines of angles up to 2^20: an fp64 product is off by 2^-33
    close(got, *op.heads(f64(q), cos=np.cos(a), sin=np.sin(a)), "far")


@pytest.mark.parametrize("D,R", [(64, 64), (66, 20), (36, 12)])
@pytest.mark.parametrize("bits", [torch.int32, torch.int64])
def test_positions_outside_the_table(D, R, bits):
    rs = np.random.default_rng(1)
    q, w = rnd(rs, (5, 3, D), torch.bfloat16), rnd(rs, (D,), torch.bfloat16)
    table = moeq.rope_table(16, R)
    big = 1 << 40 if bits == torch.int64 else 1 << 30
    pos = torch.tensor([3, -1, 16, 15, big], dtype=bits, device=DEV)
    ok = torch.tensor([3, 0, 0, 15, 0], dtype=bits, device=DEV)
    got, _ = moeq.head_norm_rope(q, None, w, pos=pos, table=table)
    ref, _ = moeq.head_norm_rope(q, None, w, pos=ok, table=table)
    for t in (0, 3):
        assert torch.equal(got[t], ref[t])
    for t in (1, 2, 4):
        assert torch.isnan(got[t, :, :R]).all() and torch.equal(got[t, :, R:], ref[t, :, R:])


@pytest.mark.parametrize("D,R", [(128, 64), (66, 66), (36, 8)])
@pytest.mark.parametrize("dt", sorted(TYPES))
def test_strides(D, R, dt):
    """Heads inside wider tensors, at odd places, by head first: the same bits, and
    nothing else is written."""
    rs = np.random.default_rng(D)
    T, Hq, Hk, dtype = 6, 4, 2, TYPES[dt]
    q, k = rnd(rs, (T, Hq, D), dtype), rnd(rs, (T, Hk, D), dtype)
    qw, kw = rnd(rs, (D,), dtype), rnd(rs, (D,), dtype)
    kwargs = dict(pos=torch.arange(T, device=DEV) + 9, table=moeq.rope_table(32, R))
    ref = moeq.head_norm_rope(q, k, qw, kw, **kwargs)
    for off in (0, 1, 8, 13):
        say("strides", D, R, dt, off)
        wide = torch.full((T, (Hq + Hk) * D + 2 * off + 3), 7.0, dtype=dtype, device=DEV)
        vq = wide[:, off:off + Hq * D].unflatten(1, (Hq, D))
        vk = wide[:, off + Hq * D:off + (Hq + Hk) * D].unflatten(1, (Hk, D))
        vq.copy_(q)
        vk.copy_(k)
        out = torch.full((Hq + Hk, T + 1, D + off), 5.0, dtype=dtype, device=DEV)
        oq, ok = (out[a:b, :T, off:].transpose(0, 1) for a, b in ((0, Hq), (Hq, Hq + Hk)))
        moeq.head_norm_rope(vq, vk, qw, kw, q_out=oq, k_out=ok, **kwargs)
        assert torch.equal(oq, ref[0]) and torch.equal(ok, ref[1])
        assert (out[:, T] == 5).all() and (out[:, :, :off] == 5).all()
        moeq.head_norm_rope(vq, vk, qw, kw, q_out=vq, k_out=vk, **kwargs)
        assert torch.equal(vq, ref[0]) and torch.equal(vk, ref[1])
        assert (wide[:, :off] == 7).all() and (wide[:, off + (Hq + Hk) * D:] == 7).all()
    # a broadcast input
    one = q[:1].expand(T, Hq, D)
    got, _ = moeq.head_norm_rope(one, None, qw, **kwargs)
    assert torch.equal(got, moeq.head_norm_rope(one.contiguous(), None, qw, **kwargs)[0])


def test_bits_do_not_follow_the_batch():
    rs = np.random.default_rng(3)
    for D, R in ((128, 128), (66, 18), (36, 36)):
        T, Hq = 2000, 40
        q, w = rnd(rs, (T, Hq, D), torch.float32), rnd(rs, (D,), torch.float32)
        table = moeq.rope_table(T, R)
        pos = torch.arange(T, device=DEV)
        whole, _ = moeq.head_norm_rope(q, None, w, pos=pos, table=table)
        for t, h in ((0, 0), (1999, 39), (1000, 7)):
            one, _ = moeq.head_norm_rope(q[t:t + 1, h:h + 1], None, w, pos=pos[t:t + 1], table=table)
            assert torch.equal(one[0, 0], whole[t, h])


def test_range_of_the_norm():
    """Heads whose squares leave fp32's range; zeros; an infinity or a NaN stays in
    its head."""
    rs = np.random.default_rng(4)
    for D in (64, 66, 36):
        x = rs.standard_normal((6, 2, D)).astype(np.float32)
        for t, s in enumerate((1e30, 1e-30, 3e37, 2e-38, 1.0, 0.0)):
            x[t] *= s
        q, w = torch.from_numpy(x).to(DEV), rnd(rs, (D,), torch.float32)
        got, _ = moeq.head_norm_rope(q, None, w, eps=0.0)
        ref, mag = op.heads(f64(q)[:5], f64(w), 0.0)
        close(got[:5], ref, mag, "range")
        assert torch.isnan(got[5]).all()
        assert (moeq.head_norm_rope(q[5:], None, w, eps=1e-6)[0] == 0).all()
        q[4, 0, 3], q[3, 1, 0] = float("inf"), float("nan")
        bad, _ = moeq.head_norm_rope(q, None, w, eps=0.0)
        keep = torch.ones(6, 2, dtype=torch.bool)
        keep[4, 0] = keep[3, 1] = keep[5, 0] = keep[5, 1] = False
        assert torch.equal(bad[keep], got[keep])
        assert torch.isnan(bad[3, 1]).all() and torch.isnan(bad[4, 0, 3])


def test_nothing_to_do_and_refusals():
    q, w = torch.zeros((0, 4, 64), device=DEV), torch.ones(64, device=DEV)
    assert moeq.head_norm_rope(q, None, w)[0].shape == (0, 4, 64)
    q = torch.zeros((2, 4, 64), device=DEV)
    assert moeq.head_norm_rope(q[:, :0], q, w, w)[1].shape == q.shape
    table = moeq.rope_table(4, 64)
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    for kw, says in ((dict(pos=pos), "needs a table"), (dict(table=table), "needs pos"),
                     (dict(pos=pos[:1], table=table), "pos must"),
                     (dict(pos=pos.float(), table=table), "pos must"),
                     (dict(pos=pos, table=table.half()), "table must"),
                     (dict(pos=pos, table=table.t()), "table must"),
                     (dict(pos=pos, table=table.cpu()), "table must"),
                     (dict(k_w=w), "need k"), (dict(k=q.half(), q_w=w), "k must"),
                     (dict(k=q.cpu(), q_w=w), "k must"), (dict(k=q[:1], q_w=w), "k must")):
        with pytest.raises(ValueError, match=says):
            moeq.head_norm_rope(q, **kw)
    with pytest.raises(moeq.MoeError, match="neither"):
        moeq.head_norm_rope(q)
    with pytest.raises(moeq.MoeError, match="overlap"):
        moeq.head_norm_rope(q, None, w, q_out=q[:1].expand(2, 4, 64))
    with pytest.raises(moeq.MoeError, match="R must"):
        moeq.head_norm_rope(q, pos=pos, table=moeq.rope_table(4, 66))


def test_stream_and_graph():
    """On a stream of the caller's, and captured: replays follow the inputs."""
    rs = np.random.default_rng(5)
    q, k = rnd(rs, (3, 8, 128), torch.bfloat16), rnd(rs, (3, 2, 128), torch.bfloat16)
    w, table = rnd(rs, (128,), torch.bfloat16), moeq.rope_table(64, 128)
    pos = torch.tensor([1, 2, 3], device=DEV)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    run = lambda: moeq.head_norm_rope(q, k, w, w, pos=pos, table=table, q_out=qo, k_out=ko)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for i in range(3):
        q.copy_(rnd(rs, q.shape, q.dtype))
        pos.add_(7)
        g.replay()
        torch.cuda.synchronize()
        want = moeq.head_norm_rope(q, k, w, w, pos=pos, table=table)
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1]), i


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,R", [(520, 28, 4, 128, 128), (700, 12, 4, 192, 64),
                                         (9000, 3, 0, 80, 16)])
def test_results_past_the_caches(T, Hq, Hk, D, R, inter, dt):
    """2^21 elements and more, whose results go past the caches."""
    say("large", T, Hq, Hk, D, R, inter, dt)
    assert T * (Hq + Hk) * D >= 2 ** 21 and D % 16 == 0 and R % 16 == 0
    rs = np.random.default_rng(T)
    q = rnd(rs, (T, Hq, D), TYPES[dt], 3.0)
    k = rnd(rs, (T, Hk, D), TYPES[dt]) if Hk else None
    qw, kw = rnd(rs, (D,), TYPES[dt]), rnd(rs, (D,), TYPES[dt]) if Hk else None
    pos = rs.integers(0, 3000, T)
    c, s = cos_sin(pos, R, 3000)
    outs = moeq.head_norm_rope(q, k, qw, kw, pos=torch.from_numpy(pos).to(DEV),
                               table=moeq.rope_table(3000, R), interleaved=inter)
    for x, w, o in ((q, qw, outs[0]), (k, kw, outs[1])):
        if x is not None:
            close(o, *op.heads(f64(x), f64(w), 1e-5, 0.0, c, s, inter), "norm and rotation")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("D,R", [(64, 32), (66, 2), (36, 36), (1003, 4)])
def test_small_elements_of_far_heads(D, R, dt):
    """Heads whose squares leave fp32's range hold elements far below the others: these keep
    their accuracy (their norms are over 2^-126)."""
    say("far heads", D, R, dt)
    rs = np.random.default_rng(D)
    T, Hq = 6, 3
    # an element of 2^66 among ones of 2^-55; of 2^-60 among ones of 2^-145; mixed in a wave
    big = np.array([2.0 ** 66, 1.0, 2.0 ** 100, 2.0 ** -60, 2.0 ** 66, 2.0 ** 40])[:, None, None]
    rest = np.array([2.0 ** -55, 2.0 ** -100, 2.0 ** -20, 2.0 ** -120, 2.0 ** -50, 2.0 ** -70])[:, None, None]
    x = rest * (1 + rs.random((T, Hq, D))) * rs.choice([-1, 1], (T, Hq, D))
    x[:, :, D // 2:D // 2 + 2] = big * (1 + rs.random((T, Hq, 2)))
    q = torch.from_numpy(x).to(TYPES[dt]).to(DEV)
    w = (rnd(rs, (D,), torch.float32).abs() + 0.5).to(TYPES[dt])
    pos = torch.arange(T, device=DEV) + 3
    c, s = cos_sin(pos.cpu().numpy(), R, 16)
    got, _ = moeq.head_norm_rope(q, None, w, pos=pos, table=moeq.rope_table(16, R), eps=0.0)
    close(got, *op.heads(f64(q), f64(w), 0.0, 0.0, c, s), "far heads")
