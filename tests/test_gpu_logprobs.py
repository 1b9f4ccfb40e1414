"""GPU parity of the token log probabilities (moe_token_logprobs) against the fp64
oracle.

Tolerances, from the kernel's arithmetic.  With z = scale (x - max), fp32 takes z to
2^-22 |z| (the difference, the scale in units of log2 e, their product) and its
exponential to one step, 2^-23, on top; a sum has at most 55 additions in a chain (32 of a
thread, 6 lane stages, 8 waves, a slice's factor, 6 lane stages again).  Under p, m1 = E|z|
and m2 = E z^2:
    log S is off by 2^-22 (m1 + 20),
    log p by that, 2^-22 |z| and a few roundings of its own, 2^-22 |log p| (|z| <= |log p|),
    the entropy by 2^-22 (m2 + m1^2 + 40 m1 + 24).
Best tokens are exact.
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
STEP = 2.0 ** -22


def check(x, top=0, ids=None, scale=None, **kw):
    T, V = x.shape
    got = moeq.token_logprobs(x, ids, top=top, scale=scale, **kw)
    x64 = x.to(torch.float64).cpu().numpy()
    sc = None if scale is None else scale.cpu().numpy()
    lp, H, m1, m2 = op.logprobs(x64, sc)

    def close(a, b, tol, what):
        a = a.cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isnan(a), np.isnan(b)), what
        assert np.array_equal(np.isneginf(a), np.isneginf(b)), what
        live = np.isfinite(b)
        err = np.abs(np.where(live, a, 0) - np.where(live, b, 0))
        assert np.all(err <= tol), (what, float((err / tol).max()))

    close(got[1], H, STEP * (m2 + m1 * m1 + 40 * m1 + 24), "entropy")
    if ids is not None:
        at = ids.reshape(T, -1).cpu().numpy().astype(np.int64)
        want = np.where((at >= 0) & (at < V), np.take_along_axis(lp, np.clip(at, 0, V - 1), 1), np.nan)
        tol = STEP * (np.abs(np.nan_to_num(want, nan=0, neginf=0)) * 2 + m1[:, None] + 24)
        assert got[0].shape == ids.shape
        close(got[0].reshape(T, -1), want, tol, "log p")
    if top:
        bad = np.isnan(H)
        best = op.best(x64, top)
        best[bad] = -1
        assert np.array_equal(got[2].cpu().numpy(), best), "best tokens"
        want = np.where(best >= 0, np.take_along_axis(lp, np.maximum(best, 0), 1),
                        np.where(bad[:, None], np.nan, -np.inf))
        tol = STEP * (np.abs(np.nan_to_num(want, nan=0, neginf=0)) * 2 + m1[:, None] + 24)
        close(got[3], want, tol, "best log p")
    return got


def rows(rs, T, V, dtype, spread=3.0):
    return torch.from_numpy((rs.standard_normal((T, V)) * spread).astype(np.float32)).to(dtype).to(DEV)


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("T,V,top,m", [
    (1, 1, 1, 1), (2, 1, 3, 2), (1, 7, 7, 1), (3, 8, 5, 0), (5, 1003, 20, 3), (2, 4096, 32, 1),
    (4, 16383, 8, 1), (3, 16384, 0, 1), (2, 16385, 32, 4), (3, 16391, 5, 1), (1, 32768, 1, 70),
    (2, 50257, 20, 2), (1, 131072, 32, 1), (1, 262147, 20, 1), (600, 2000, 3, 1)])
def test_rows(T, V, top, m, dt):
    say("logprobs", T, V, top, m, dt)
    rs = np.random.default_rng(V + T)
    x = rows(rs, T, V, TYPES[dt])
    ids = torch.from_numpy(rs.integers(0, V, (T, m)).astype(np.int32)).to(DEV) if m else None
    scale = torch.from_numpy(rs.uniform(0.3, 2, T).astype(np.float32)).to(DEV)
    check(x, top, ids)
    got = check(x, top, None if ids is None else ids.long(), scale)
    again = moeq.token_logprobs(x, ids, top=top, scale=scale)
    for a, b in zip(got, again):
        assert a is None and b is None or torch.equal(a, b)


def test_largest_vocabulary():
    rs = np.random.default_rng(9)
    x = rows(rs, 1, 1 << 20, torch.bfloat16)
    check(x, 32, torch.tensor([5], device=DEV))


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("V", [60, 5000, 40000])
def test_masks(V, dt):
    """Masked tokens, rows that are masked but for a few or as a whole, the lowest finite
    value as a mask, slices with nothing left."""
    say("masks", V, dt)
    rs = np.random.default_rng(V)
    dtype = TYPES[dt]
    x = rows(rs, 8, V, dtype)
    ninf, low = -float("inf"), torch.finfo(dtype).min
    x[0, ::3] = ninf
    x[1] = ninf
    x[2, : V - 2] = ninf
    x[3] = ninf
    x[3, V // 2] = -5.0
    x[4, ::2] = low
    x[5] = low
    x[6, 16:] = ninf
    x[7, : V - 1] = low
    ids = torch.tensor([[0, 1], [0, V - 1], [V - 1, 0], [V // 2, 0], [0, 1], [3, V - 1], [2, 20],
                        [V - 1, 0]], dtype=torch.int32, device=DEV)
    got = check(x, 20, ids)
    assert got[1][1] == 0 and (got[2][1] == -1).all()
    assert got[2][3].tolist() == [V // 2] + [-1] * 19 and got[3][3, 0] == 0
    assert got[2][5].tolist() == list(range(20))
    check(x, 5, ids, torch.full((8,), 0.25, device=DEV))


@pytest.mark.parametrize("dt", sorted(TYPES))
def test_rows_without_a_distribution(dt):
    """NaN, +inf and scales that are none: NaN and -1 in that row, the others as they are."""
    rs = np.random.default_rng(6)
    x = rows(rs, 9, 20000, TYPES[dt])
    ref = check(x, 4, torch.zeros(9, dtype=torch.int32, device=DEV))
    y = x.clone()
    y[1, 19999] = float("nan")
    y[2, 3] = float("inf")
    y[3] = float("nan")
    y[4] = -float("inf")
    y[4, 17000] = float("nan")
    scale = torch.ones(9, device=DEV)
    scale[5], scale[6], scale[7] = 0.0, -1.0, float("inf")
    got = check(y, 4, torch.zeros(9, dtype=torch.int32, device=DEV), scale)
    for t in (0, 8):
        assert all(torch.equal(a[t], b[t]) for a, b in zip(got, ref))


@pytest.mark.parametrize("dt", sorted(TYPES))
def test_large_magnitudes(dt):
    """Logits far from zero on either side, up to the type's largest: only differences count."""
    rs = np.random.default_rng(11)
    big = float(torch.finfo(TYPES[dt]).max)
    x = torch.empty((12, 20000), dtype=TYPES[dt], device=DEV)
    for t, base in enumerate((1e4, 6e5, 9e5, 3e6, 1e10, 1e20, 1e28, 1e30, 1e38)):
        base = min(base, big / 2)
        step = base * torch.finfo(TYPES[dt]).eps
        x[t] = (1 if t % 2 else -1) * base + torch.from_numpy(rs.integers(0, 9, 20000) * step).to(DEV)
    x[9], x[10], x[11] = big, -big, 0.0
    x[11, 7], x[11, 9] = -big, big
    ids = torch.tensor([3, 9], dtype=torch.int32, device=DEV).repeat(12, 1)
    check(x, 9, ids)
    check(x, 9, ids, torch.full((12,), 1e-4, device=DEV))


def test_ids_outside():
    x = rows(np.random.default_rng(1), 2, 100, torch.float32)
    ids = torch.tensor([[-1, 100, 5], [99, -2 ** 31, 2 ** 31 - 1]], dtype=torch.int32, device=DEV)
    got, _ = check(x, 0, ids)
    assert torch.isnan(got).tolist() == [[True, True, False], [False, True, True]]
    check(x, 0, torch.tensor([1 << 40, -(1 << 40)], device=DEV))


@pytest.mark.parametrize("dt", sorted(TYPES))
def test_orders_and_ties(dt):
    """The best tokens where they lie all together, in rising and falling rows, among many equal
    logits, and with both zeros."""
    rs = np.random.default_rng(7)
    V = 40000
    dtype = TYPES[dt]
    x = torch.empty((8, V), dtype=dtype, device=DEV)
    ramp = torch.arange(V, device=DEV).float() / V * 30
    x[0], x[1] = ramp, ramp.flip(0)
    x[2] = 1.0
    x[3] = torch.from_numpy(rs.integers(0, 2, V)).to(DEV)
    x[4] = torch.from_numpy(rs.integers(0, 40, V)).to(DEV)
    x[5] = 0.0
    x[5, ::2] = -0.0
    x[6] = rows(rs, 1, V, torch.float32)[0]
    x[6, 20000:20064] = 50 + torch.arange(64, device=DEV) % 7       # neighbours, in 8 lots of 8
    x[7] = -1.0
    x[7, 8::4096] = 2.0                                              # one thread's logits
    x[7, 39990:] = 2.0
    for top in (1, 5, 20, 32):
        check(x, top)


def test_strides():
    rs = np.random.default_rng(8)
    x = rows(rs, 5, 999, torch.bfloat16)
    ids = torch.arange(5, dtype=torch.int32, device=DEV)
    ref = moeq.token_logprobs(x, ids, top=6)
    for off, extra in ((0, 25), (1, 0), (8, 8), (3, 7)):
        wide = torch.full((5, 999 + off + extra), 1e4, dtype=x.dtype, device=DEV)
        wide[:, off:off + 999] = x
        for a, b in zip(moeq.token_logprobs(wide[:, off:off + 999], ids, top=6), ref):
            assert torch.equal(a, b)
    got = moeq.token_logprobs(x[::2], ids[::2].contiguous(), top=6)
    for a, b in zip(got, ref):
        assert torch.equal(a, b[::2])


def test_bits_do_not_follow_the_batch():
    rs = np.random.default_rng(10)
    x = rows(rs, 700, 30011, torch.float16)
    ids = torch.from_numpy(rs.integers(0, 30011, 700).astype(np.int32)).to(DEV)
    whole = moeq.token_logprobs(x, ids, top=9)
    for t in (0, 333, 699):
        for a, b in zip(moeq.token_logprobs(x[t:t + 1], ids[t:t + 1], top=9), whole):
            assert torch.equal(a[0], b[t])


def test_outputs_and_refusals():
    x = rows(np.random.default_rng(2), 3, 50, torch.float32)
    ids = torch.zeros(3, dtype=torch.int32, device=DEV)
    lp, en = torch.empty(3, device=DEV), torch.empty(3, device=DEV)
    ti, tl = torch.empty((3, 2), dtype=torch.int32, device=DEV), torch.empty((3, 2), device=DEV)
    ws = moeq.token_logprobs_workspace(x, 2)
    got = moeq.token_logprobs(x, ids, top=2, logprob=lp, entropy=en, top_ids=ti, top_logprob=tl, ws=ws)
    assert all(a is b for a, b in zip(got, (lp, en, ti, tl)))
    assert moeq.token_logprobs(x)[0] is None
    assert moeq.token_logprobs(x, ids[:, None][:, :0])[0].shape == (3, 0)
    empty = moeq.token_logprobs(x[:0], ids[:0], top=2)
    assert [tuple(t.shape) for t in empty] == [(0,), (0,), (0, 2), (0, 2)]
    for kw, says in ((dict(top=33), "top"), (dict(top=-1), "top"), (dict(ids=ids[:2]), "ids"),
                     (dict(ids=ids.float()), "ids"), (dict(ids=ids.cpu()), "ids"),
                     (dict(logprob=lp), "needs ids"), (dict(top_ids=ti), "top > 0"),
                     (dict(ids=ids, logprob=lp[:2]), "logprob"), (dict(entropy=en.half()), "entropy"),
                     (dict(scale=en[:2]), "scale"), (dict(top=2, top_ids=ti.long()), "top_ids"),
                     (dict(ws=ws.float()), "workspace")):
        with pytest.raises(ValueError, match=says):
            moeq.token_logprobs(x, **kw)
    with pytest.raises(moeq.MoeError, match="workspace"):
        moeq.token_logprobs(x, top=30, ws=ws[:256])
    for bad in (x.t(), x[0], x.double()):
        with pytest.raises(ValueError):
            moeq.token_logprobs(bad)


def test_stream_and_graph():
    rs = np.random.default_rng(3)
    x = rows(rs, 4, 33000, torch.bfloat16)
    ids = torch.tensor([1, 2, 3, 4], dtype=torch.int32, device=DEV)
    out = dict(logprob=torch.empty(4, device=DEV), entropy=torch.empty(4, device=DEV),
               top_ids=torch.empty((4, 7), dtype=torch.int32, device=DEV),
               top_logprob=torch.empty((4, 7), device=DEV), ws=moeq.token_logprobs_workspace(x, 7))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moeq.token_logprobs(x, ids, top=7, **out)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moeq.token_logprobs(x, ids, top=7, **out)
    for i in range(3):
        x.copy_(rows(rs, 4, 33000, torch.bfloat16))
        ids.add_(11)
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(moeq.token_logprobs(x, ids, top=7), list(out.values())):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("top", [0, 8])
def test_more_logits_than_the_caches_hold(top, dt):
    """2^28 bytes of logits and more, which are read past the caches: rows among them against the
    oracle, and all of them bit for bit as in batches that are not."""
    say("large", top, dt)
    V = 50257
    T = 2 ** 28 // (V * (4 if dt == "fp32" else 2)) + 2
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn((T, V), generator=g, device=DEV).mul_(3).to(TYPES[dt])
    x[T // 2, ::5] = -float("inf")
    ids = torch.randint(0, V, (T, 2), generator=g, device=DEV, dtype=torch.int32)
    whole = moeq.token_logprobs(x, ids, top=top)
    half = T // 2 + 1
    for a, b in ((0, half), (half, T)):
        for u, v in zip(moeq.token_logprobs(x[a:b], ids[a:b], top=top), whole):
            assert torch.equal(u, v[a:b])
    some = [0, T // 2, T - 1]
    got = check(x[some], top, ids[some])
    for u, v in zip(got, whole):
        assert torch.equal(u, v[some])
