"""GPU parity of the low-rank adapters (moe_pack_adapter, moe_adapter_plan,
moe_add_adapters) against the fp64 oracle.

Tolerance, from the kernel's arithmetic.  A matrix instruction's fp32 sums are taken at
2^-23 a step.  h = s A x: a chain of at most K / 16 + 128 inputs, 16 parts, two scales,
so 2^-23 (K / 16 + 152) of s sum |A x|.  h enters B h as the sum of 16-bit numbers: bf16 to
2^-16 of itself, or 2^-24 where y is fp32, fp16 to 2^-21 of the token's largest.  B h: 2^-23
(3 r + 8) of sum |B h|.  One addition of y in fp32 and half a step of y's type on top.
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


def rnd(rs, shape, dtype, scale=1.0):
    return torch.from_numpy((rs.standard_normal(shape) * scale).astype(np.float32)).to(dtype).to(DEV)


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def make(rs, n, rank, K, N, dtype, ranks=None, empty=()):
    """A set with adapters in its slots but `empty`, and what the oracle takes."""
    s = moeq.Adapters(n, rank, K, N, dtype=dtype)
    known = []
    for i in range(n):
        r = rank if ranks is None else ranks[i % len(ranks)]
        if i in empty:
            known.append(None)
            continue
        a, b, scale = rnd(rs, (r, K), dtype, K ** -0.5), rnd(rs, (N, r), dtype, 0.5), 0.5 + i / 8
        s.load(i, a, b, scale)
        known.append((f64(a), f64(b), np.float32(scale)))
    return s, known


def close(got, x, ids, known, y, w_dtype, what):
    K = x.shape[1]
    rank = max([k[0].shape[0] for k in known if k is not None] or [0])
    ref, bh, bax, bmax = op.add_adapters(x, ids, known, f64(y))
    split = 2.0 ** -21 * bmax if w_dtype == torch.float16 else \
        (2.0 ** -24 if y.dtype == torch.float32 else 2.0 ** -16) * bh
    tol = 2.0 ** -23 * ((K / 16 + 152) * bax + (3 * rank + 8) * bh) + split
    half = torch.finfo(y.dtype).eps / 2
    tol = tol * (1 + half) + (half + 2.0 ** -24) * np.abs(ref) + TINY[y.dtype]
    err = np.abs(f64(got) - ref)
    assert np.all(err <= tol), (what, float((err / tol).max()))


@pytest.mark.parametrize("w,x,y", [("bf16", "bf16", "bf16"), ("bf16", "codes", "fp32"),
                                   ("fp16", "fp16", "fp16"), ("fp16", "codes", "fp32"),
                                   ("bf16", "bf16", "fp16"), ("fp16", "fp16", "bf16"),
                                   ("bf16", "codes", "bf16"), ("bf16", "bf16", "fp32")])
@pytest.mark.parametrize("T,n,rank,K,N", [
    (1, 1, 16, 256, 128), (1, 3, 1, 1, 1), (2, 2, 8, 7, 9), (5, 4, 17, 129, 65), (16, 1, 32, 2048, 64),
    (17, 1, 64, 130, 200), (40, 8, 48, 1001, 250), (64, 64, 16, 512, 1000), (33, 3, 100, 300, 72),
    (20, 2, 256, 640, 333), (70, 1023, 4, 64, 40), (1030, 5, 40, 333, 130), (1100, 3, 130, 200, 88), (600, 2, 16, 2100, 70),
    (1030, 2, 128, 333, 130), (2050, 20, 64, 2100, 70), (2800, 3, 40, 130, 100), (4100, 3, 32, 70, 72)])
def test_products(T, n, rank, K, N, w, x, y):
    say("adapters", T, n, rank, K, N, w, x, y)
    rs = np.random.default_rng(T + K + N)
    dtype = TYPES[w]
    s, known = make(rs, n, rank, K, N, dtype, ranks=[rank, max(1, rank // 3), max(1, rank - 1)],
                    empty=(1,) if n > 2 else ())
    ids = rs.integers(-1, n, T).astype(np.int32)
    ids[0] = 0
    plan = moeq.adapter_plan(torch.from_numpy(ids).to(DEV), n)
    xt, scale = rnd(rs, (T, K), dtype), None
    x64 = f64(xt)
    if x == "codes":
        xt, scale = moeq.quantize_i8(xt)
        x64 = f64(xt)[:, :K] * f64(scale)[:, None]
    yt = rnd(rs, (T, N), TYPES[y])
    before = yt.clone()
    out = torch.empty_like(yt)
    got = moeq.add_adapters(s, xt, plan, yt, scale=scale, out=out)
    assert got is out and torch.equal(yt, before)
    close(got, x64, ids, known, yt, dtype, "sum")
    again = moeq.add_adapters(s, xt, plan, yt, scale=scale)
    assert again is yt and torch.equal(yt, got)


@pytest.mark.parametrize("T,n", [(1, 1), (1, 1023), (15, 3), (1023, 3), (1024, 32), (1024, 33), (4096, 7), (4097, 7), (4097, 1023),
                                 (9000, 1), (20000, 300)])
def test_plans(T, n):
    """Every token once, by its adapter, in tiles of one adapter."""
    say("plan", T, n)
    rs = np.random.default_rng(T)
    ids = rs.integers(-2, n + 2, T).astype(np.int32)
    ids[0], ids[-1] = 2 ** 31 - 1, -2 ** 31
    plan = moeq.adapter_plan(torch.from_numpy(ids).to(DEV), n)
    p = plan.data.view(torch.int32).cpu().numpy()
    bins = np.where((ids >= 0) & (ids < n), ids, n)
    tile = 64 if T >= 1024 and T >= 32 * n else 16
    tiles = T // tile + min(T, n + 1)
    recs = p[:tiles * (4 + tile)].reshape(tiles, 4 + tile)
    order = p[recs.size:recs.size + T]
    assert np.array_equal(order, np.argsort(bins, kind="stable"))
    used = sum(-(-c // tile) for c in np.bincount(bins))
    at = 0
    for rec in recs[:used]:
        a, first, count, zero = rec[:4].tolist()
        assert first == at and 1 <= count <= tile and zero == 0
        mine = order[first:first + count]
        assert np.all(bins[mine] == a) and np.array_equal(rec[4:4 + count], mine)
        assert np.all(rec[4 + count:] == mine[-1])
        at += count
    assert at == T and np.all(recs[used:, 0] == n) and not recs[used:, 1:4].any()
    again = moeq.adapter_plan(torch.from_numpy(ids).to(DEV), n, plan)
    assert again is plan and np.array_equal(plan.data.view(torch.int32).cpu().numpy()[:recs.size + T],
                                            p[:recs.size + T])


def test_many_tokens():
    """A plan of more tokens than one workgroup sorts, and tiles of every kind."""
    rs = np.random.default_rng(11)
    T, n, K, N = 5000, 6, 96, 80
    s, known = make(rs, n, 20, K, N, torch.bfloat16, ranks=[20, 3, 16, 17], empty=(4,))
    ids = rs.choice([-1, 0, 0, 0, 1, 2, 3, 4, 5], T).astype(np.int32)
    x, y = rnd(rs, (T, K), torch.bfloat16), rnd(rs, (T, N), torch.float32)
    got = moeq.add_adapters(s, x, moeq.adapter_plan(torch.from_numpy(ids).to(DEV), n), y,
                            out=torch.empty_like(y))
    close(got, f64(x), ids, known, y, torch.bfloat16, "many")


def test_bits_do_not_follow_the_batch():
    """A token alone, among others, at both sizes of the dispatch: the same bits; tokens
    without an adapter are copies."""
    rs = np.random.default_rng(12)
    for w, y in ((torch.bfloat16, torch.float32), (torch.float16, torch.float16)):
        T, n, K, N = 2100, 4, 3000, 200
        s, _ = make(rs, n, 60, K, N, w, ranks=[60, 20, 16, 7])
        ids = torch.from_numpy(rs.integers(-1, n, T).astype(np.int32)).to(DEV)
        xt, yt = rnd(rs, (T, K), w), rnd(rs, (T, N), y)
        whole = moeq.add_adapters(s, xt, moeq.adapter_plan(ids, n), yt, out=torch.empty_like(yt))
        for t in (0, 3, 700, 2099):
            one = moeq.add_adapters(s, xt[t:t + 1], moeq.adapter_plan(ids[t:t + 1].clone(), n),
                                    yt[t:t + 1], out=torch.empty_like(yt[:1]))
            assert torch.equal(one[0], whole[t])
        part = moeq.add_adapters(s, xt[:90], moeq.adapter_plan(ids[:90].clone(), n), yt[:90],
                                 out=torch.empty_like(yt[:90]))
        assert torch.equal(part, whole[:90])
        none = ids < 0
        assert none.any() and torch.equal(whole[none], yt[none])


def test_strides():
    """Rows of wider tensors on and off 16 bytes, matrices inside wider ones: the same
    bits, and nothing else is written."""
    rs = np.random.default_rng(13)
    T, n, K, N, r = 21, 2, 200, 136, 24
    a, b = rnd(rs, (r, K + 5), torch.bfloat16)[:, 3:K + 3], rnd(rs, (N, r + 3), torch.bfloat16)[:, 1:r + 1]
    s, t = (moeq.Adapters(n, r, K, N) for _ in range(2))
    s.load(1, a, b, 2.0)
    t.load(1, a.contiguous(), b.contiguous(), 2.0)
    ids = torch.ones(T, dtype=torch.int32, device=DEV)
    ids[::5] = 0
    plan = moeq.adapter_plan(ids, n)
    x = rnd(rs, (T, K), torch.bfloat16)
    for dt in TYPES.values():
        y = rnd(rs, (T, N), dt)
        ref = moeq.add_adapters(t, x, plan, y, out=torch.empty_like(y))
        for off, extra in ((0, 0), (8, 8), (1, 0), (3, 2)):
            say("strides", dt, off, extra)
            wx = torch.full((T, K + off + extra), float("nan"), dtype=x.dtype, device=DEV)
            wx[:, off:off + K] = x
            wy, wo = (torch.full((T, N + off + extra), 7.0, dtype=dt, device=DEV) for _ in range(2))
            wy[:, off:off + N] = y
            moeq.add_adapters(s, wx[:, off:off + K], plan, wy[:, off:off + N], out=wo[:, off:off + N])
            assert torch.equal(wo[:, off:off + N], ref)
            assert (wo[:, :off] == 7).all() and (wo[:, off + N:] == 7).all()
            moeq.add_adapters(s, wx[:, off:off + K], plan, wy[:, off:off + N])
            assert torch.equal(wy[:, off:off + N], ref) and (wy[:, off + N:] == 7).all()


def test_slots_change():
    """Slots loaded again with a smaller rank, emptied, filled; the set's other slots stay."""
    rs = np.random.default_rng(14)
    K, N = 70, 50
    s, known = make(rs, 3, 40, K, N, torch.float16)
    ids = np.array([0, 1, 2, 1], np.int32)
    plan = moeq.adapter_plan(torch.from_numpy(ids).to(DEV), 3)
    x, y = rnd(rs, (4, K), torch.float16), rnd(rs, (4, N), torch.float32)
    for step in range(3):
        if step == 1:
            a, b = rnd(rs, (5, K), torch.float16), rnd(rs, (N, 5), torch.float16)
            s.load(1, a, b, -1.5)
            known[1] = (f64(a), f64(b), -1.5)
        if step == 2:
            s.unload(0)
            known[0] = None
        got = moeq.add_adapters(s, x, plan, y, out=torch.empty_like(y))
        close(got, f64(x), ids, known, y, torch.float16, step)
    assert torch.equal(got[0], y[0])


@pytest.mark.parametrize("w", [torch.bfloat16, torch.float16])
def test_values_that_are_not_finite(w):
    """An infinity or a NaN of a row, or a row of codes with scale NaN, stays in its row; small and
    large rows keep their accuracy."""
    rs = np.random.default_rng(15)
    T, K, N = 20, 300, 70
    s, known = make(rs, 1, 33, K, N, w)
    ids = np.zeros(T, np.int32)
    plan = moeq.adapter_plan(torch.zeros(T, dtype=torch.int32, device=DEV), 1)
    x = rnd(rs, (T, K), w)
    # fp16's smallest rows stay normal numbers
    for t, e in ((0, 6), (1, -6), (2, 12), (3, -10)):
        x[t] *= 2.0 ** e
    y = torch.zeros((T, N), device=DEV)
    got = moeq.add_adapters(s, x, plan, y, out=torch.empty_like(y))
    close(got, f64(x), ids, known, y, w, "scaled rows")
    z = x.clone()
    z[5, 7], z[6, K - 1] = float("inf"), float("nan")
    bad = moeq.add_adapters(s, z, plan, y, out=torch.empty_like(y))
    keep = torch.ones(T, dtype=torch.bool)
    keep[5] = keep[6] = False
    assert torch.equal(bad[keep], got[keep]) and not torch.isfinite(bad[5:7]).any()
    q, scale = moeq.quantize_i8(z)
    codes = moeq.add_adapters(s, q, plan, y, scale=scale, out=torch.empty_like(y))
    assert torch.isnan(codes[5:7]).all() and torch.isfinite(codes[keep]).all()


def test_empty_and_refusals():
    s = moeq.Adapters(2, 8, 64, 32)
    x, y = torch.zeros((3, 64), dtype=torch.bfloat16, device=DEV), torch.ones((3, 32), device=DEV)
    ids = torch.zeros(3, dtype=torch.int32, device=DEV)
    plan = moeq.adapter_plan(ids, 2)
    assert (moeq.add_adapters(s, x, plan, y, out=torch.empty_like(y)) == 1).all()   # nothing loaded
    none = moeq.adapter_plan(ids[:0], 2)
    assert moeq.add_adapters(s, x[:0], none, y[:0]).shape == (0, 32)
    for call, says in (
            (lambda: moeq.add_adapters(s, x[:2], plan, y[:2]), "plan is of 3"),
            (lambda: moeq.add_adapters(s, x, moeq.adapter_plan(ids, 3), y), "and 2"),
            (lambda: moeq.add_adapters(s, x.half(), plan, y), "x must be"),
            (lambda: moeq.add_adapters(s, x.float(), plan, y), "x must be"),
            (lambda: moeq.add_adapters(s, x.to(torch.int8), plan, y), "scales"),
            (lambda: moeq.add_adapters(s, x, plan, y, scale=y[:, 0]), "codes only"),
            (lambda: moeq.add_adapters(s, x, plan, y[:, :31]), "y must"),
            (lambda: moeq.add_adapters(s, x, plan, y.double()), "fp32"),
            (lambda: moeq.add_adapters(s, x, plan, y, out=y.half()), "out must"),
            (lambda: moeq.adapter_plan(ids.long(), 2), "ids must"),
            (lambda: moeq.adapter_plan(ids, 0), "unsupported"),
            (lambda: moeq.adapter_plan(ids, 2, none), "0 tokens"),
            (lambda: s.load(2, x[:1], y[:, :1]), "slot"),
            (lambda: s.load(0, torch.zeros((9, 64), dtype=x.dtype, device=DEV), y), "1 to 8"),
            (lambda: s.load(0, x, y), "b must"),
            (lambda: s.load(0, x.half(), y), "a must"),
            (lambda: s.load(0, x[:, :63], y), "a must")):
        with pytest.raises(ValueError, match=says):
            call()
    with pytest.raises(moeq.MoeError, match="workspace"):
        moeq.add_adapters(s, x, plan, y, ws=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(moeq.MoeError, match="slot"):
        s.unload(2)


def test_stream_and_graph():
    """Plan and products on a stream of the caller's and captured: replays follow ids, rows
    and slots."""
    rs = np.random.default_rng(16)
    K, N, n, T = 256, 192, 5, 24
    s, _ = make(rs, n, 16, K, N, torch.bfloat16)
    ids = torch.zeros(T, dtype=torch.int32, device=DEV)
    x, y = rnd(rs, (T, K), torch.bfloat16), rnd(rs, (T, N), torch.bfloat16)
    out, ws = torch.empty_like(y), moeq.add_adapters_workspace(s, T)
    plan = moeq.adapter_plan(ids, n)

    def run():
        moeq.adapter_plan(ids, n, plan)
        moeq.add_adapters(s, x, plan, y, out=out, ws=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for i in range(3):
        ids.copy_(torch.from_numpy(rs.integers(-1, n, T).astype(np.int32)))
        x.copy_(rnd(rs, x.shape, x.dtype))
        s.load(i, rnd(rs, (9, K), torch.bfloat16), rnd(rs, (N, 9), torch.bfloat16), 1.0)
        g.replay()
        torch.cuda.synchronize()
        want = moeq.add_adapters(s, x, moeq.adapter_plan(ids, n), y, out=torch.empty_like(y))
        assert torch.equal(out, want), i


@pytest.mark.parametrize("T,K,N", [(1, 256, 128), (40, 200, 100), (700, 264, 192)])
def test_beside_an_8_bit_product(T, K, N):
    """linear_i8 with adapters is the product and then add_adapters, for rows and codes."""
    rs = np.random.default_rng(17)
    lin = moeq.I8Linear.quantized(rnd(rs, (N, K), torch.float32))
    s, _ = make(rs, 3, 16, K, N, torch.bfloat16)
    ids = rs.integers(-1, 3, T).astype(np.int32)
    plan = moeq.adapter_plan(torch.from_numpy(ids).to(DEV), 3)
    x = rnd(rs, (T, K), torch.bfloat16)
    q, scale = moeq.quantize_i8(x)
    for rows, sc in ((x, None), (q, scale)):
        y = moeq.linear_i8(lin, rows, sc, out_dtype=torch.float32)
        want = moeq.add_adapters(s, rows, plan, y.clone(), scale=sc)
        got = moeq.linear_i8(lin, rows, sc, out_dtype=torch.float32, adapters=s, plan=plan)
        assert torch.equal(got, want) and torch.equal(got, y) == (ids < 0).all()
    other = moeq.Adapters(3, 16, K, N + 1)
    for kw in (dict(adapters=s), dict(plan=plan), dict(adapters=other, plan=plan),
               dict(adapters=s, plan=moeq.adapter_plan(torch.zeros(T, dtype=torch.int32, device=DEV), 2))):
        with pytest.raises(ValueError, match="adapters"):
            moeq.linear_i8(lin, x, **kw)
    with pytest.raises(ValueError, match="adapters"):
        moeq.linear_i8(lin, x.half(), adapters=s, plan=plan)


@pytest.mark.parametrize("w", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("T,rank,K", [(4100, 32, 1300), (2100, 60, 3000), (2800, 48, 130), (1030, 128, 700),
                                      (1700, 80, 2100), (1100, 130, 520), (2050, 16, 400)])
def test_bits_in_every_kernel(T, rank, K, codes, w):
    """The same bits for a token alone, in a few and among many, at every set of kernels that the
    dispatch takes for the batch: rows and codes, ranks to 32, 64 and 128, more, and 16."""
    say("bits", T, rank, K, codes, w)
    rs = np.random.default_rng(T + rank)
    n, N = 4, 136
    s, _ = make(rs, n, rank, K, N, w, ranks=[rank, rank // 3, rank - 1, 5])
    ids = torch.from_numpy(rs.integers(-1, n, T).astype(np.int32)).to(DEV)
    x, scale = rnd(rs, (T, K), w), None
    if codes:
        x, scale = moeq.quantize_i8(x)
    for yt in (torch.float32, w):
        y = rnd(rs, (T, N), yt)

        def run(a, b):
            return moeq.add_adapters(s, x[a:b], moeq.adapter_plan(ids[a:b].clone(), n), y[a:b],
                                     scale=None if scale is None else scale[a:b].clone(),
                                     out=torch.empty_like(y[a:b]))

        whole = run(0, T)
        for a, b in ((0, 1), (77, 78), (T - 1, T), (500, 590), (0, 1000)):
            assert torch.equal(run(a, b), whole[a:b]), (a, b)
