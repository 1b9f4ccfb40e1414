"""GPU parity of the block norms (moe_block_norm) against the fp64 oracle.

Tolerance, from the kernel's arithmetic: everything is fp32 until one rounding
to the output's type.  A sum of H squares adds at most 40 values in one chain
(8 of a thread, 6 lane stages, then 16 parts in order or, where there are more,
8 a lane and 6 lane stages), each rounding 2^-24, and
enters as a square root (half); the other steps of an element are under 30
roundings (k <= 16 products and sums among them).  64 * 2^-24 = 2^-18 of the
sum of the terms' magnitudes covers them; half a step of the output type comes
on top.
"""

import numpy as np
import pytest
import torch

import bit_quantized_moe_route_amd as moeq
from oracle import block as ob
from tests.gpu_common import say

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
REL32 = 2.0 ** -18


def rnd(rs, shape, dtype, scale=1.0):
    return torch.from_numpy((rs.standard_normal(shape) * scale).astype(np.float32)).to(dtype).to(DEV)


def f64(t):
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def close(got, ref, mag, what):
    half = torch.finfo(got.dtype).eps / 2
    tol = half * np.abs(ref) + (1 + half) * REL32 * mag + TINY[got.dtype]
    err = np.abs(f64(got) - ref)
    assert np.all(err <= tol), (what, float((err / tol).max()), np.argmax(err / tol))


def close_codes(q, scale, n, mag, H, what):
    """|q * scale - n| is half a step, and the error of n and of the scale."""
    q, scale = q.cpu().numpy().astype(np.float64), f64(scale)[:, None]
    assert np.all(q[:, H:moeq.codes_width(H)] == 0), what
    q = q[:, :H]
    a = np.abs(n).max(1, keepdims=True)
    slack = REL32 * mag.max(1, keepdims=True)
    assert np.all(np.abs(scale * 127 - a) <= slack + 2.0 ** -22 * a), what
    tol = 0.5 * scale * (1 + 2.0 ** -16) + 2 * slack + 2.0 ** -22 * a
    err = np.abs(q * scale - n)
    assert np.all(err <= tol), (what, float((err / tol).max()))


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("T,H", [(1, 1), (1, 6144), (3, 7), (5, 64), (2, 1003), (7, 8192),
                                 (2, 8200), (2, 16392), (2, 32768), (3, 8193), (2, 32767),
                                 (260, 136), (300, 8192), (2200, 1000)])
def test_norm(T, H, dt):
    say("block_norm", T, H, dt)
    rs = np.random.default_rng(H * 7 + T)
    r, w = rnd(rs, (T, H), TYPES[dt], 3.0), rnd(rs, (H,), TYPES[dt])
    n, q, s = moeq.block_norm(r, w, eps=1e-5, codes=True)
    _, mag, ref, nmag = ob.block(f64(r), None, f64(w), eps=1e-5)
    close(n, ref, nmag, "n")
    close_codes(q, s, ref, nmag, H, "codes")
    only = moeq.block_norm(r, w, eps=1e-5)
    assert torch.equal(only, n)
    none, q2, s2 = moeq.block_norm(r, w, eps=1e-5, codes=True, out=False)
    assert none is None and torch.equal(q2, q) and torch.equal(s2, s)


@pytest.mark.parametrize("r_t,y_t,w_t,n_t", [("bf16", "bf16", "bf16", "bf16"),
                                             ("fp32", "bf16", "fp32", "bf16"),
                                             ("fp16", "fp32", "fp16", "fp32"),
                                             ("fp32", "fp16", "bf16", "fp16")])
@pytest.mark.parametrize("gate", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("T,H", [(1, 24), (5, 1000), (4, 333)])
def test_residual(T, H, post, gate, r_t, y_t, w_t, n_t):
    rs = np.random.default_rng(H + T)
    r, y = rnd(rs, (T, H), TYPES[r_t]), rnd(rs, (T, H), TYPES[y_t], 2.0)
    w = rnd(rs, (H,), TYPES[w_t], 0.3)
    pw = rnd(rs, (H,), TYPES[w_t], 0.3) if post else None
    shape = {"none": None, "token": (T, 1), "channel": (1, H), "full": (T, H)}[gate]
    g = rnd(rs, shape, TYPES[y_t]) if shape else None
    kw = dict(y_scale=0.7, r_scale=1.3, eps=1e-6, w_offset=1.0)
    r2, n, q, s = moeq.block_residual(r, y, w, post_w=pw, gate=g, out_dtype=TYPES[n_t], codes=True,
                                      **kw)
    assert r2.dtype == r.dtype and n.dtype == TYPES[n_t]
    ref_r, rmag, ref_n, nmag = ob.block(f64(r), f64(y), f64(w), f64(pw), f64(g), **kw)
    close(r2, ref_r, rmag, "r'")
    close(n, ref_n, nmag, "n")
    close_codes(q, s, ref_n, nmag, H, "codes")
    # the residual stream updated in place, and without a norm after it
    r3 = r.clone()
    got, none = moeq.block_residual(r3, y, None, post_w=pw, gate=g, r_out=r3, **kw)
    assert got is r3 and none is None and torch.equal(r3, r2)


@pytest.mark.parametrize("y_t,r_t", [("fp32", "bf16"), ("bf16", "bf16"), ("fp16", "fp32")])
@pytest.mark.parametrize("T,k,H,E", [(1, 8, 6144, 256), (3, 1, 40, 4), (9, 3, 333, 5),
                                     (2, 16, 128, 16), (65, 8, 264, 32), (520, 3, 4104, 8)])
@pytest.mark.parametrize("shared", [0, 1, 2])
def test_combine(T, k, H, E, shared, y_t, r_t):
    rs = np.random.default_rng(T + k + H)
    logits = torch.from_numpy(rs.standard_normal((T, E)).astype(np.float32)).to(DEV)
    ids, tw, _, _, _, inv = moeq.route_permute(logits, k)
    y, r = rnd(rs, (T * k, H), TYPES[y_t]), rnd(rs, (T, H), TYPES[r_t])
    ys = rnd(rs, (T, H), TYPES[y_t]) if shared else None
    sg = rnd(rs, (T,), torch.float32) if shared == 2 else None
    w, pw = rnd(rs, (H,), TYPES[r_t]), rnd(rs, (H,), TYPES[r_t])
    b, bmag = ob.gated_sum(f64(y), inv.cpu().numpy(), f64(tw), f64(ys), f64(sg))
    for post in (None, pw):
        r2, n, q, s = moeq.combine_residual(r, y, inv, tw, w, y_shared=ys, shared_gate=sg,
                                            post_w=post, y_scale=0.5, codes=True)
        ref_r, rmag, ref_n, nmag = ob.block(f64(r), b, f64(w), f64(post), y_scale=0.5, y_mag=bmag)
        close(r2, ref_r, rmag, "r'")
        close(n, ref_n, nmag, "n")
        close_codes(q, s, ref_n, nmag, H, "codes")
    # no residual stream: the gated sum alone
    out, none = moeq.combine_residual(None, y, inv, tw, y_shared=ys, shared_gate=sg)
    assert none is None and out.dtype == torch.float32
    close(out, b, bmag, "sum")


def test_strides_and_offsets():
    """Rows of wider tensors, starting on and off 16 bytes: the same bits, and
    nothing outside the rows is written."""
    T, H = 5, 256
    rs = np.random.default_rng(5)
    for dt in TYPES.values():
        r, y = rnd(rs, (T, H), dt), rnd(rs, (T, H), dt)
        w, pw, g = rnd(rs, (H,), dt), rnd(rs, (H,), dt), rnd(rs, (1, H), dt)
        ref = moeq.block_residual(r, y, w, post_w=pw, gate=g, codes=True)
        for off, extra in ((0, 64), (8, 24), (1, 7), (3, 0)):
            say("strides", dt, off, extra)
            wide = [torch.full((T, H + off + extra), 7.0, dtype=dt, device=DEV) for _ in range(4)]
            views = [t[:, off:off + H] for t in wide]
            views[0].copy_(r)
            views[1].copy_(y)
            qw = torch.full((T, 512), 9, dtype=torch.int8, device=DEV)
            got = moeq.block_residual(views[0], views[1], w, post_w=pw, gate=g, r_out=views[2],
                                      out=views[3], codes=True, q=qw[:, 16:16 + 256])
            if off % 8 == 0 and extra % 8 == 0:
                for a, b in zip(got, ref):
                    assert torch.equal(a, b)
            ref_r, rmag, ref_n, nmag = ob.block(f64(r), f64(y), f64(w), f64(pw), f64(g))
            close(got[0], ref_r, rmag, "r'")
            close(got[1], ref_n, nmag, "n")
            close_codes(got[2], got[3], ref_n, nmag, H, "codes")
            for t in wide:
                assert torch.all(t[:, :off] == 7) and torch.all(t[:, off + H:] == 7)
            assert torch.all(qw[:, :16] == 9) and torch.all(qw[:, 272:] == 9)


def test_rows_do_not_depend_on_the_batch():
    """A row's bits are the same alone and among others, and run to run."""
    T, H, k, E = 2100, 1024, 4, 16
    rs = np.random.default_rng(8)
    logits = torch.from_numpy(rs.standard_normal((T, E)).astype(np.float32)).to(DEV)
    _, tw, _, _, _, inv = moeq.route_permute(logits, k)
    y, r = rnd(rs, (T * k, H), torch.bfloat16), rnd(rs, (T, H), torch.bfloat16)
    w = rnd(rs, (H,), torch.bfloat16)
    full = moeq.combine_residual(r, y, inv, tw, w, codes=True)
    again = moeq.combine_residual(r, y, inv, tw, w, codes=True)
    for a, b in zip(full, again):
        assert torch.equal(a, b)
    for t in (0, 517, T - 1):
        yt = y[inv[t * k:(t + 1) * k].long()]
        one = moeq.combine_residual(r[t:t + 1], yt, torch.arange(k, dtype=torch.int32, device=DEV),
                                    tw[t:t + 1].contiguous(), w, codes=True)
        for a, b in zip(one, full):
            assert torch.equal(a[0], b[t])


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("T,H,off", [(3, 8, 1), (5, 256, 3), (2100, 1024, 1), (2, 9000, 5)])
def test_bits_do_not_follow_the_alignment(T, H, off, dt):
    """Rows at an element's alignment give the bits of the same rows on 16 bytes,
    also where the results go over the operands."""
    rs = np.random.default_rng(H + off)
    k = 2
    r, y = rnd(rs, (T, H), TYPES[dt]), rnd(rs, (T * k, H), TYPES[dt])
    w, tw = rnd(rs, (H,), TYPES[dt]), rnd(rs, (T, k), torch.float32)
    inv = torch.arange(T * k, dtype=torch.int32, device=DEV).flip(0).contiguous()
    wide = torch.full((T, H + off + 2), 7.0, dtype=TYPES[dt], device=DEV)
    at = wide[:, off:off + H]
    ref = moeq.block_residual(r, y[:T], w, post_w=w, codes=True)
    at.copy_(r)
    got = moeq.block_residual(at, y[:T], w, post_w=w, r_out=at, codes=True)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    ref = moeq.combine_residual(r, y, inv, tw, w, codes=True)
    at.copy_(r)
    got = moeq.combine_residual(at, y, inv, tw, w, r_out=at, codes=True)
    for a, b in zip(got, ref):
        assert torch.equal(a, b)
    at.copy_(r)
    for a, b in zip(moeq.quantize_i8(at), moeq.quantize_i8(r)):
        assert torch.equal(a, b)
    assert torch.all(wide[:, :off] == 7) and torch.all(wide[:, off + H:] == 7)


@pytest.mark.parametrize("H", [7, 8, 9, 15, 511, 513, 1003, 8191, 8193, 16391, 32767])
def test_odd_rows_in_place(H):
    """The last chunk of a row shares elements with the one before: results over
    the operands are those beside them."""
    rs = np.random.default_rng(H)
    for T in (3, 700):
        r, y, w = rnd(rs, (T, H), torch.bfloat16), rnd(rs, (T, H), torch.bfloat16), \
            rnd(rs, (H,), torch.bfloat16)
        ref_r, ref_n = moeq.block_residual(r, y, w, post_w=w, gate=y)
        r2 = r.clone()
        _, n2 = moeq.block_residual(r2, y, w, post_w=w, gate=y, r_out=r2)
        assert torch.equal(r2, ref_r) and torch.equal(n2, ref_n)
        want = ob.block(f64(r), f64(y), f64(w), f64(w), f64(y))
        close(ref_r, want[0], want[1], "r'")
        close(ref_n, want[2], want[3], "n")


def test_more_rows_than_one_launch_holds():
    """A launch ends at 2^32 threads, 2^26 rows of one wave each: the rows behind
    it, and those beside the border, are done all the same."""
    T, n = (1 << 26) + 37, 1 << 26
    x = torch.ones((T, 1), dtype=torch.bfloat16, device=DEV)
    x[-50:, 0] = torch.arange(1, 51, device=DEV)
    w = torch.full((1,), 2.0, dtype=torch.bfloat16, device=DEV)
    # rows of one element: n = w * r / sqrt(r^2), r' = r + 3
    r2, out = moeq.block_residual(x, torch.full_like(x, 3.0), w, eps=0.0)
    assert torch.all(out == 2.0)
    assert torch.equal(r2[-50:, 0], torch.arange(4, 54, device=DEV).to(torch.bfloat16))
    assert torch.all(r2[:-50] == 4.0)
    del r2, out
    # codes 127 of rows of one element
    q, s = moeq.quantize_i8(x)
    assert torch.all(q[:, 0] == 127) and torch.all(q[n - 64:, 1:] == 0)
    a = x[-50:, 0].to(torch.float64)
    assert torch.all((s[-50:].to(torch.float64) * 127 - a).abs() <= 2.0 ** -24 * a)
    assert torch.all(s[:-50] == s[0])


def test_non_finite_rows_stay_apart():
    T, H = 6, 72
    rs = np.random.default_rng(9)
    r, w = rnd(rs, (T, H), torch.float32), rnd(rs, (H,), torch.float32)
    clean = moeq.block_norm(r, w, codes=True)
    r[1, 5], r[3, 71] = float("nan"), float("inf")
    r[4] = 0.0
    n, q, s = moeq.block_norm(r, w, codes=True)
    for t in (0, 2, 5):
        assert torch.equal(n[t], clean[0][t]) and torch.equal(q[t], clean[1][t])
        assert torch.equal(s[t], clean[2][t])
    assert torch.isnan(n[1]).all() and torch.isnan(s[1]) and torch.all(q[1] == 0)
    assert torch.isnan(s[3]) and torch.all(q[3] == 0)
    assert torch.all(n[4] == 0) and s[4] == 0 and torch.all(q[4] == 0)


def test_empty_batch():
    e = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    r2, n, q, s = moeq.block_residual(e, e, w, codes=True)
    assert r2.shape == n.shape == (0, 64) and q.shape == (0, 64) and s.shape == (0,)


def test_graph_and_side_stream():
    """Captured and replayed on new inputs, and run on another stream."""
    T, H = 9, 512
    rs = np.random.default_rng(10)
    r, y = rnd(rs, (T, H), torch.bfloat16), rnd(rs, (T, H), torch.bfloat16)
    w = rnd(rs, (H,), torch.bfloat16)
    ro, n = torch.empty_like(r), torch.empty_like(r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ref = moeq.block_residual(r, y, w)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    moeq.block_residual(r, y, w, r_out=ro, out=n)
    torch.cuda.synchronize()
    assert torch.equal(ro, ref[0]) and torch.equal(n, ref[1])
    with torch.cuda.graph(g):
        moeq.block_residual(r, y, w, r_out=ro, out=n)
    for i in range(4):
        y.copy_(rnd(rs, (T, H), torch.bfloat16))
        ref = moeq.block_residual(r, y, w)
        ro.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(ro, ref[0]) and torch.equal(n, ref[1]), i
