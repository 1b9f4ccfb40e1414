"""The operators of a decoder step in the order in which they are used: block norm and its
codes, the 8-bit product to queries, keys and values with its requests' adapters, the heads'
norms and rotation in place, and behind a second norm the product to logits and their log
probabilities.  Each against the fp64 form of its own inputs, and the whole captured.

Tolerances: each operator's own (test_gpu_adapters.py, test_gpu_heads.py,
test_gpu_logprobs.py); a product in 8 bits is compared with its codes' exact sums, rounded to
bf16 (half a step, 2^-8) after a few roundings of fp32.
"""

import numpy as np
import pytest
import torch

import bit_quantized_moe_route_amd as moeq
from oracle import block as ob
from oracle import project as op
from tests import test_gpu_adapters as ta
from tests import test_gpu_heads as th
from tests import test_gpu_logprobs as tl

pytestmark = pytest.mark.gpu

DEV = "cuda"


class Step:
    """One layer's end and the model's, for T tokens of up to n requests' adapters."""

    def __init__(self, T, H=320, Hq=6, Hk=2, D=64, V=1500, n=4, seed=0):
        rs = np.random.default_rng(seed)
        rnd = lambda *s: th.rnd(rs, s, torch.bfloat16)  # noqa: E731
        self.T, self.Hq, self.Hk, self.D, self.rs = T, Hq, Hk, D, rs
        N = (Hq + 2 * Hk) * D
        self.r, self.y, self.w = rnd(T, H), rnd(T, H), rnd(H)
        w8 = rs.integers(-127, 128, (N, H)).astype(np.int8), rs.integers(-127, 128, (V, H)).astype(np.int8)
        self.codes = [torch.from_numpy(w).to(DEV) for w in w8]
        self.scales = [torch.full((w.shape[0],), 0.02 / 127, device=DEV) for w in w8]
        self.qkv, self.head = (moeq.I8Linear(c, s) for c, s in zip(self.codes, self.scales))
        self.set, self.known = ta.make(rs, n, 16, H, N, torch.bfloat16, ranks=[16, 5], empty=(2,))
        self.ids = torch.from_numpy(rs.integers(-1, n, T).astype(np.int32)).to(DEV)
        self.plan = moeq.adapter_plan(self.ids, n)
        self.qw, self.kw = rnd(D), rnd(D)
        self.pos = torch.from_numpy(rs.integers(0, 4096, T)).to(DEV)
        self.table = moeq.rope_table(4096, D)
        self.tokens = torch.from_numpy(rs.integers(0, V, T).astype(np.int32)).to(DEV)
        self.rows = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)

    def heads(self, rows):
        a, b = self.Hq * self.D, (self.Hq + self.Hk) * self.D
        return (rows[:, :a].unflatten(1, (self.Hq, self.D)),
                rows[:, a:b].unflatten(1, (self.Hk, self.D)))

    def run(self):
        moeq.adapter_plan(self.ids, self.set.n, self.plan)
        r, n, q, s = moeq.block_residual(self.r, self.y, self.w, codes=True)
        moeq.linear_i8(self.qkv, q, s, out=self.rows, adapters=self.set, plan=self.plan)
        qh, kh = self.heads(self.rows)
        moeq.head_norm_rope(qh, kh, self.qw, self.kw, pos=self.pos, table=self.table, q_out=qh,
                            k_out=kh)
        _, n2, q2, s2 = moeq.block_residual(r, n, self.w, codes=True)
        logits = moeq.linear_i8(self.head, q2, s2, out_dtype=torch.bfloat16)
        return [q, s, self.rows, logits, *moeq.token_logprobs(logits, self.tokens, top=5)]


@pytest.mark.parametrize("T", [1, 7, 600])
def test_step(T):
    st = Step(T)
    q, s, rows, logits, lp, ent, ti, tl_ = st.run()
    H = st.r.shape[1]
    x64 = q.cpu().numpy().astype(np.float64)[:, :H] * s.cpu().numpy().astype(np.float64)[:, None]
    # the product, the adapters on its rounded result, and the heads of that
    base = moeq.linear_i8(st.qkv, q, s, out_dtype=torch.bfloat16)
    exact = ob.product_i8(q.cpu().numpy()[:, :H], st.codes[0].cpu().numpy()) \
        * s.cpu().numpy().astype(np.float64)[:, None] * st.scales[0].cpu().numpy().astype(np.float64)
    assert np.all(np.abs(th.f64(base) - exact) <= (2.0 ** -8 + 2.0 ** -20) * np.abs(exact) + 1e-30)
    full = moeq.linear_i8(st.qkv, q, s, out_dtype=torch.bfloat16, adapters=st.set, plan=st.plan)
    ta.close(full, x64, st.ids.cpu().numpy(), st.known, base, torch.bfloat16, "adapters")
    a = op.angles(4096, st.D)[st.pos.cpu().numpy()]
    for src, dst, w in zip(st.heads(full), st.heads(rows), (st.qw, st.kw)):
        th.close(dst, *op.heads(th.f64(src), th.f64(w), 1e-5, 0.0, np.cos(a), np.sin(a)), "heads")
    b = (st.Hq + st.Hk) * st.D
    assert torch.equal(rows[:, b:], full[:, b:])                 # the values stay
    got = tl.check(logits, 5, st.tokens)
    for x, y in zip(got, (lp, ent, ti, tl_)):
        assert torch.equal(x, y)


def test_step_captured():
    """Replays with other inputs, eager work between them, against eager runs; another graph of
    the same operators in flight on its own workspace."""
    st, other = Step(9), Step(5, seed=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        st.run()
        other.run()
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for s in (st, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s.run())
        graphs.append(g)
    for i in range(3):
        for s in (st, other):
            s.r.copy_(th.rnd(s.rs, s.r.shape, torch.bfloat16))
            s.ids.copy_(torch.from_numpy(s.rs.integers(-1, 4, s.T).astype(np.int32)))
            s.pos.copy_(torch.from_numpy(s.rs.integers(0, 4096, s.T)))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        seen = [[t.clone() for t in o] for o in outs]
        for s, got in zip((st, other), seen):
            for a, b in zip(got, s.run()):
                assert torch.equal(a, b), i


def far(rows, width, gap):
    """[rows, width] of bf16 whose last row lies past 2^31 elements."""
    t = torch.empty((rows - 1) * gap + width, dtype=torch.bfloat16, device=DEV)
    assert (rows - 1) * gap > 2 ** 31
    return t.as_strided((rows, width), (gap, 1))


@pytest.mark.parametrize("rows", [3, 2100])
def test_rows_far_apart(rows):
    """Offsets past 32 bits: the results are those of the rows side by side."""
    rs = np.random.default_rng(rows)
    gap = 2 ** 31 // (rows - 1) + 64
    wide = far(rows, 512, gap)
    near = th.rnd(rs, (rows, 512), torch.bfloat16)
    wide.copy_(near)
    pos = torch.arange(rows, device=DEV)
    table, w = moeq.rope_table(rows, 64), th.rnd(rs, (64,), torch.bfloat16)
    parts = lambda t: t.unflatten(1, (8, 64))  # noqa: E731
    want, _ = moeq.head_norm_rope(parts(near), None, w, pos=pos, table=table)
    got, _ = moeq.head_norm_rope(parts(wide), None, w, pos=pos, table=table)
    assert torch.equal(got, want)
    ids = torch.from_numpy(rs.integers(0, 512, rows)).to(DEV)
    for a, b in zip(moeq.token_logprobs(wide, ids, top=3), moeq.token_logprobs(near, ids, top=3)):
        assert torch.equal(a, b)
    s, _ = ta.make(rs, 2, 64, 512, 512, torch.bfloat16)
    plan = moeq.adapter_plan(torch.from_numpy(rs.integers(-1, 2, rows).astype(np.int32)).to(DEV), 2)
    want = moeq.add_adapters(s, near, plan, near, out=torch.empty_like(near))
    assert torch.equal(moeq.add_adapters(s, wide, plan, wide, out=torch.empty_like(near)), want)
    out = far(rows, 512, gap)
    assert torch.equal(moeq.add_adapters(s, near, plan, near, out=out), want)
    # heads in place, their rows far apart
    moeq.head_norm_rope(parts(wide), None, w, pos=pos, table=table, q_out=parts(wide))
    assert torch.equal(parts(wide), moeq.head_norm_rope(parts(near), None, w, pos=pos, table=table)[0])


def test_two_streams_at_once():
    """Calls in flight together on one set, plan and table, each with its own workspace."""
    rs = np.random.default_rng(3)
    T, K = 2100, 512
    s, _ = ta.make(rs, 3, 64, K, K, torch.bfloat16)
    plan = moeq.adapter_plan(torch.from_numpy(rs.integers(-1, 3, T).astype(np.int32)).to(DEV), 3)
    xs = [th.rnd(rs, (T, K), torch.bfloat16) for _ in range(2)]
    ids = torch.from_numpy(rs.integers(0, K, T)).to(DEV)
    run = lambda x: [moeq.add_adapters(s, x, plan, x, out=torch.empty_like(x)),  # noqa: E731
                     *moeq.token_logprobs(x, ids, top=4)]
    want = [run(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[], []]
    for _ in range(5):
        for i, (x, stream) in enumerate(zip(xs, streams)):
            with torch.cuda.stream(stream):
                got[i].append(run(x))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        for r in runs:
            for a, b in zip(r, w):
                assert torch.equal(a, b)


def test_space_of_a_larger_batch():
    """A workspace and a plan's bytes made for the largest batch serve the smaller ones."""
    rs = np.random.default_rng(4)
    s, _ = ta.make(rs, 2, 64, 300, 100, torch.bfloat16)
    ws = moeq.add_adapters_workspace(s, 4096)
    for T in (1, 1000, 1023, 1024, 2047, 2048, 4096):
        x, y = th.rnd(rs, (T, 300), torch.bfloat16), th.rnd(rs, (T, 100), torch.bfloat16)
        plan = moeq.adapter_plan(torch.from_numpy(rs.integers(-1, 2, T).astype(np.int32)).to(DEV), 2)
        want = moeq.add_adapters(s, x, plan, y, out=torch.empty_like(y))
        assert torch.equal(moeq.add_adapters(s, x, plan, y, out=torch.empty_like(y), ws=ws), want)


@pytest.mark.parametrize("n", [3, 1000])
def test_plans_in_the_bytes_of_a_larger_one(n):
    """The bytes of a larger batch's plan, and its workspace, take any smaller batch's; nothing
    behind them is written.  (At 131073 tokens the sort goes on to fewer slices.)"""
    rs = np.random.default_rng(n)
    most = 131073
    s, _ = ta.make(rs, n, 3, 16, 8, torch.bfloat16)
    L = moeq.lib()
    size = L.moe_adapter_plan_bytes(most, n)
    ws = moeq.add_adapters_workspace(s, most)
    ids = torch.from_numpy(rs.integers(-1, n, most).astype(np.int32)).to(DEV)
    x, y = th.rnd(rs, (most, 16), torch.bfloat16), th.rnd(rs, (most, 8), torch.bfloat16)
    for T in (most, 131072, 100000, 4097, 4096, 1024, 1):
        data = torch.full((size + 64,), 77, dtype=torch.uint8, device=DEV)
        stream = torch.cuda.current_stream().cuda_stream
        assert L.moe_adapter_plan(ids.data_ptr(), T, n, data.data_ptr(), size, stream) == 0
        assert (data[size:] == 77).all()
        got = moeq.add_adapters(s, x[:T], moeq.AdapterPlan(T, n, data), y[:T],
                                out=torch.empty_like(y[:T]), ws=ws)
        want = moeq.add_adapters(s, x[:T], moeq.adapter_plan(ids[:T].clone(), n), y[:T],
                                 out=torch.empty_like(y[:T]))
        assert torch.equal(got, want), T


def test_a_refused_adapter_workspace_leaves_the_output():
    """linear_i8 refuses the adapters' workspace before the product writes."""
    rs = np.random.default_rng(6)
    lin = moeq.I8Linear.quantized(th.rnd(rs, (100, 256), torch.float32))
    s, _ = ta.make(rs, 2, 16, 256, 100, torch.bfloat16)
    x = th.rnd(rs, (9, 256), torch.bfloat16)
    plan = moeq.adapter_plan(torch.zeros(9, dtype=torch.int32, device=DEV), 2)
    ws = moeq.add_adapters_workspace(s, 9)
    want = moeq.linear_i8(lin, x, adapters=s, plan=plan)
    assert torch.equal(moeq.linear_i8(lin, x, adapters=s, plan=plan, adapter_ws=ws), want)
    out = torch.full((9, 100), 7.0, dtype=torch.bfloat16, device=DEV)
    wide = torch.empty(ws.numel() + 256, dtype=torch.uint8, device=DEV)
    for bad in (ws[:256], ws.float(), ws.cpu(), wide[1:]):
        with pytest.raises((ValueError, moeq.MoeError), match="workspace"):
            moeq.linear_i8(lin, x, out=out, adapters=s, plan=plan, adapter_ws=bad)
    torch.cuda.synchronize()
    assert (out == 7).all()
