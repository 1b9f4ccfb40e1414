"""GPU parity of the 8-bit integer products against the oracle.

Codes and scales are held to the exact bits of their fp32 definition.  The
integer sums are exact, so a product is off by its fp32 epilogue (four
roundings, 2^-24 each, and one of the bias' addition) and half a step of the
output type.  In the gated feed-forward the middle rows h are fp32: g and u
carry 4 roundings, exp(-g) is off by |g| 2^-23 (the rounded argument) plus
2^-22 (the instruction), so h is within (|g|max 2^-23 + 2^-20) of a row's
largest; a code of h whose exact value lies that near to the border between
two integers may be either, and the oracle adds up what that can change.
"""

import numpy as np
import pytest
import torch

import bit_quantized_moe_route_amd as moeq
import oracle
from oracle import block as ob
from tests.gpu_common import say

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TINY = {torch.float32: 2.0 ** -140, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def rnd(rs, shape, dtype, scale=1.0):
    return torch.from_numpy((rs.standard_normal(shape) * scale).astype(np.float32)).to(dtype).to(DEV)


def codes(rs, shape):
    """8-bit codes over the whole range, -128 included (weights may hold any)."""
    return torch.from_numpy(rs.integers(-128, 128, shape).astype(np.int8)).to(DEV)


def scales(rs, shape):
    return torch.from_numpy((np.exp(rs.standard_normal(shape) * 0.3) * 0.01).astype(np.float32)).to(DEV)


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def same_codes(x, q, s, what):
    K = x.shape[1]
    rq, rscale = ob.quantize_i8(x.float().cpu().numpy())
    got = q.cpu().numpy()
    assert np.array_equal(got[:, :K], rq), what
    assert np.all(got[:, K:moeq.codes_width(K)] == 0), what
    assert np.array_equal(s.cpu().numpy(), rscale, equal_nan=True), what
    return rq, rscale


# ------------------------------------------------------------------ codes

@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("T,K", [(1, 1), (1, 64), (3, 65), (5, 1003), (2, 6144), (300, 2048),
                                 (2, 8192), (3, 8200), (2, 32768), (2, 40000), (2, 40001)])
def test_quantize(T, K, dt):
    say("quantize", T, K, dt)
    rs = np.random.default_rng(T * K)
    x = rnd(rs, (T, K), TYPES[dt], 5.0)
    q, s = moeq.quantize_i8(x)
    same_codes(x, q, s, (T, K, dt))


def test_quantize_special_rows():
    x = torch.zeros((10, 40), dtype=torch.float32, device=DEV)
    x[1, 3] = -1e-42                       # below the smallest row maximum: codes 0
    x[2, 0], x[2, 1] = 127 * 2.0 ** -126, -1.0 * 2.0 ** -126
    x[3, :] = 3.0e38
    x[4, 7] = float("inf")
    x[5, 7] = float("nan")
    x[6, :5] = torch.tensor([127.0, 0.5, 1.5, -2.5, 126.5])          # ties to even
    x[7, :4] = torch.tensor([1.0, 0.5, -0.5, 0.25])
    x[8, 39] = -float("inf")
    x[9, 39], x[9, 0] = 1.0, -1.0
    q, s = moeq.quantize_i8(x)
    same_codes(x, q, s, "special")
    assert q[6, :5].tolist() == [127, 0, 2, -2, 126]
    assert torch.isnan(s[[4, 5, 8]]).all() and not q[[0, 1, 4, 5, 8]].any()


@pytest.mark.parametrize("dt", sorted(TYPES))
def test_quantize_strided(dt):
    rs = np.random.default_rng(3)
    wide = rnd(rs, (7, 300), TYPES[dt])
    for a, b in ((0, 256), (8, 264), (1, 130), (5, 300)):
        x = wide[:, a:b]
        qw = torch.full((7, 512), 5, dtype=torch.int8, device=DEV)
        q, s = moeq.quantize_i8(x, q=qw[:, 32:32 + 448])
        same_codes(x, q, s, (a, b))
        w = moeq.codes_width(b - a)
        assert torch.all(qw[:, :32] == 5) and torch.all(qw[:, 32 + w:] == 5)


# ------------------------------------------------------------------ linear

def check_linear(lin, W, S, bias, q, s, out, what):
    acc = ob.product_i8(q, W)
    ref = acc * np.asarray(s, np.float64)[:, None] * np.asarray(S, np.float64)
    mag = np.abs(ref)
    if bias is not None:
        ref = ref + np.asarray(bias, np.float64)
        mag = mag + np.abs(ref)
    tol = torch.finfo(out.dtype).eps / 2 * np.abs(ref) + 5 * 2.0 ** -24 * mag + TINY[out.dtype]
    err = np.abs(f64(out) - ref)
    assert np.all(err <= tol), (what, float((err / tol).max()), np.argmax(err / tol))


@pytest.mark.parametrize("T,K,N", [(1, 1, 1), (1, 64, 16), (1, 6144, 48), (2, 100, 33), (16, 65, 17),
                                   (17, 640, 272), (31, 1001, 250), (33, 192, 96), (64, 512, 528),
                                   (65, 128, 1000), (128, 384, 512), (129, 2048, 256),
                                   (257, 320, 640), (300, 72, 100), (513, 1088, 520)])
@pytest.mark.parametrize("dt", sorted(TYPES))
def test_linear(T, K, N, dt):
    say("linear", T, K, N, dt)
    rs = np.random.default_rng(T + K + N)
    W, S = codes(rs, (N, K)), scales(rs, N)
    bias = rnd(rs, (N,), torch.float32) if (T + N) % 2 else None
    lin = moeq.I8Linear(W, S, bias)
    x = rnd(rs, (T, K), TYPES[dt], 2.0)
    out = moeq.linear_i8(lin, x)
    assert out.dtype == TYPES[dt]
    q, s = moeq.quantize_i8(x)
    rq, rscale = same_codes(x, q, s, "x")
    b = None if bias is None else f64(bias)
    check_linear(lin, W.cpu().numpy(), f64(S), b, rq, rscale, out, (T, K, N, dt))
    # codes in: the same product; another output type; other junk behind the codes
    q[:, K:] = 77
    out2 = moeq.linear_i8(lin, q, s, out_dtype=TYPES[dt])
    assert torch.equal(out2, out)


# one case for every kernel that the number of tiles picks: the streaming kernel
# over 1, 4 and 8 input parts, and each GEMM tile
@pytest.mark.parametrize("T,K,N", [(3, 700, 16400), (9, 200, 16400), (4, 333, 4200), (16, 1300, 4112),
                                   (1, 72, 16390), (1300, 192, 4096), (640, 136, 4090),
                                   (640, 328, 2048), (30, 264, 41000), (50, 200, 16384),
                                   (200, 520, 1040), (4, 6144, 100), (4, 6145, 100),
                                   (1, 24576, 33), (1, 24640, 33), (3, 8192, 33)])
def test_linear_every_kernel(T, K, N):
    say("linear kernels", T, K, N)
    rs = np.random.default_rng(T + K + N)
    W, S = codes(rs, (N, K)), scales(rs, N)
    lin = moeq.I8Linear(W, S)
    for dt in ("bf16", "fp32"):
        x = rnd(rs, (T, K), TYPES[dt], 2.0)
        out = moeq.linear_i8(lin, x)
        q, s = moeq.quantize_i8(x)
        check_linear(lin, W.cpu().numpy(), f64(S), None, q.cpu().numpy()[:, :K], s.cpu().numpy(),
                     out, (T, K, N, dt))
        # rows coded inside the product: the bits of coding them apart
        assert torch.equal(moeq.linear_i8(lin, q, s, out_dtype=x.dtype), out)


def test_linear_strided_in_and_out():
    rs = np.random.default_rng(4)
    T, K, N = 37, 96, 80
    W, S = codes(rs, (N, K)), scales(rs, N)
    lin = moeq.I8Linear(W, S)
    wide = rnd(rs, (T, 200), torch.bfloat16)
    for a in (0, 3, 8):
        x = wide[:, a:a + K]
        big = torch.full((T, N + 11), 3.0, dtype=torch.bfloat16, device=DEV)
        out = moeq.linear_i8(lin, x, out=big[:, 5:5 + N])
        assert torch.equal(out, moeq.linear_i8(lin, x.contiguous()))
        assert torch.all(big[:, :5] == 3) and torch.all(big[:, 5 + N:] == 3)


def test_linear_extremes():
    """Sums that only int32 holds, and rows that are zero, infinite or NaN."""
    K, N = 131071, 16
    W = torch.full((N, K), -128, dtype=torch.int8, device=DEV)
    W[3] = 127
    lin = moeq.I8Linear(W, torch.ones(N, device=DEV))
    q = torch.full((2, moeq.codes_width(K)), -128, dtype=torch.int8, device=DEV)
    q[1] = 127
    out = moeq.linear_i8(lin, q, torch.ones(2, device=DEV), out_dtype=torch.float32)
    ref = ob.product_i8(q.cpu().numpy()[:, :K], W.cpu().numpy())
    assert np.array_equal(out.cpu().numpy(), ref.astype(np.float32))
    rs = np.random.default_rng(6)
    W = codes(rs, (48, 72))
    lin = moeq.I8Linear(W, scales(rs, 48))
    x = rnd(rs, (20, 72), torch.bfloat16)
    clean = moeq.linear_i8(lin, x)
    x[3, 4], x[9, 0], x[11] = float("inf"), float("nan"), 0.0
    out = moeq.linear_i8(lin, x)
    for t in range(20):
        if t in (3, 9):
            assert torch.isnan(out[t]).all()
        elif t == 11:
            assert torch.all(out[t] == 0)
        else:
            assert torch.equal(out[t], clean[t])


# ------------------------------------------------------------------ experts

def make_layer(rs, E, H, I):
    w13, w2 = codes(rs, (E, 2 * I, H)), codes(rs, (E, H, I))
    s13, s2 = scales(rs, (E, 2 * I)) / H ** 0.5, scales(rs, (E, H))
    return moeq.I8Layer(w13, s13, w2, s2), (w13, s13, w2, s2)


def check_rows(layer, mats, e, q, s, out, what):
    w13, s13, w2, s2 = (t[e].cpu().numpy() for t in mats)
    I = layer.I
    g = ob.product_i8(q, w13[:I]) * np.asarray(s, np.float64)[:, None] * s13[:I]
    eps_h = np.abs(g).max() * 2.0 ** -23 + 2.0 ** -20
    ref, slack, near = ob.expert_i8(q, s, w13, s13, w2, s2, eps_h)
    tol = (torch.finfo(out.dtype).eps / 2 + 2.0 ** -20) * np.abs(ref) + 1.01 * slack + TINY[out.dtype]
    err = np.abs(f64(out) - ref)
    assert np.all(err <= tol), (what, e, float((err / tol).max()))
    # few codes are that near to a border: 4 * 127 * eps_h of them where the
    # fractions are spread evenly, here at most four times as many and three more
    assert near <= 4 * (4 * 127 * eps_h) * len(q) * I + 3, (what, near)


def run_experts(T, E, k, H, I, x_t, y_t, seed, ids=None):
    rs = np.random.default_rng(seed)
    layer, mats = make_layer(rs, E, H, I)
    x = rnd(rs, (T, H), TYPES[x_t])
    logits = torch.from_numpy((rs.standard_normal((T, E)) * 2).astype(np.float32)).to(DEV)
    if ids is None:
        ids, tw, counts, offsets, perm, inv = moeq.route_permute(logits, k)
    else:
        ids = torch.from_numpy(ids.astype(np.int32)).to(DEV)
        counts, offsets, perm, inv = moeq.permute(ids, E)
    y = moeq.expert_ffn_i8(layer, x, perm, offsets, k, y_dtype=TYPES[y_t])
    q, s = moeq.quantize_i8(x)
    rq, rscale = same_codes(x, q, s, "x")
    off, tok = offsets.cpu().numpy(), perm.cpu().numpy() // k
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        if off[e] < off[e + 1]:
            check_rows(layer, mats, e, rq[tok[rows]], rscale[tok[rows]], y[rows], (T, E, k, H, I))
    y2 = moeq.expert_ffn_i8(layer, q, perm, offsets, k, s, y_dtype=TYPES[y_t])
    assert torch.equal(y2, y)
    return layer, mats, x, y


@pytest.mark.parametrize("T,E,k,H,I", [(1, 1, 1, 16, 16), (1, 8, 2, 256, 128), (2, 4, 4, 272, 80),
                                       (5, 3, 2, 100, 33), (17, 8, 3, 1, 1), (37, 16, 4, 272, 80),
                                       (64, 4, 2, 128, 320), (130, 8, 8, 320, 64),
                                       (200, 70, 5, 192, 48), (300, 4, 1, 144, 112),
                                       (600, 2, 2, 192, 96), (90, 40, 8, 72, 528),
                                       (260, 40, 8, 72, 520), (700, 40, 8, 72, 264),
                                       (4, 40, 4, 1000, 200), (2, 130, 8, 72, 136)])
@pytest.mark.parametrize("x_t,y_t", [("bf16", "bf16"), ("fp32", "fp32"), ("fp16", "fp16")])
def test_expert_ffn(T, E, k, H, I, x_t, y_t):
    say("expert_ffn", T, E, k, H, I, x_t)
    run_experts(T, E, k, H, I, x_t, y_t, T + E + H)


def test_expert_ffn_one_expert_takes_all_and_repeated_ids():
    """Every token on one expert of many, and tokens that name one expert twice
    (more rows than tokens): every row is computed."""
    T, E, k = 150, 64, 2
    ids = np.zeros((T, k), np.int64)
    ids[:, 0], ids[:, 1] = 63, 5
    run_experts(T, E, k, 128, 64, "bf16", "fp32", 1, ids)
    ids[:, 1] = 63
    run_experts(T, E, k, 128, 64, "bf16", "fp32", 2, ids)
    # few rows, all on one expert
    run_experts(8, 3, 2, 136, 72, "bf16", "fp32", 3, np.full((8, 2), 1))


@pytest.mark.parametrize("T,H,I", [(1, 256, 128), (3, 100, 40), (16, 272, 80), (33, 64, 200),
                                   (128, 320, 192), (257, 192, 272), (500, 136, 96)])
@pytest.mark.parametrize("x_t", ["bf16", "fp16"])
def test_shared_ffn(T, H, I, x_t):
    say("shared_ffn", T, H, I, x_t)
    rs = np.random.default_rng(T + H)
    layer, mats = make_layer(rs, 1, H, I)
    x = rnd(rs, (T, H), TYPES[x_t])
    y = moeq.shared_ffn_i8(layer, x)
    assert y.dtype == x.dtype
    q, s = moeq.quantize_i8(x)
    check_rows(layer, mats, 0, q.cpu().numpy()[:, :H], s.cpu().numpy(), y, (T, H, I))
    assert torch.equal(moeq.shared_ffn_i8(layer, q, s, y_dtype=x.dtype), y)
    # the routed call on one expert does the same rows
    ids = torch.zeros((T, 1), dtype=torch.int32, device=DEV)
    _, offsets, perm, _ = moeq.permute(ids, 1)
    assert torch.equal(moeq.expert_ffn_i8(layer, x, perm, offsets, 1), y)


def test_bad_rows_stay_apart():
    rs = np.random.default_rng(12)
    layer, _ = make_layer(rs, 1, 128, 64)
    x = rnd(rs, (40, 128), torch.bfloat16)
    clean = moeq.shared_ffn_i8(layer, x)
    x[7, 3], x[20, 0], x[30] = float("nan"), float("inf"), 0.0
    y = moeq.shared_ffn_i8(layer, x)
    for t in range(40):
        if t in (7, 20):
            assert torch.isnan(y[t]).all()
        elif t == 30:
            assert torch.all(y[t] == 0)
        else:
            assert torch.equal(y[t], clean[t])


def test_empty_batches():
    rs = np.random.default_rng(13)
    layer, _ = make_layer(rs, 1, 64, 32)
    lin = moeq.I8Linear(codes(rs, (48, 64)), scales(rs, 48))
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=DEV)
    assert moeq.linear_i8(lin, x).shape == (0, 48)
    assert moeq.shared_ffn_i8(layer, x).shape == (0, 64)
    r = moeq.forward_i8(layer, x, torch.empty((0, 1), device=DEV), 1, shared=layer)
    assert r["out"].shape == (0, 64) and r["counts"].tolist() == [0]
    q, s = moeq.quantize_i8(x)
    assert q.shape == (0, 64) and s.shape == (0,)


# ------------------------------------------------------------------ together

def test_block_of_a_decoder():
    """norm -> codes -> router -> experts and shared expert -> gated sum, norm
    after, residual, norm before the next: each step against the oracle on the
    step's own inputs, and the whole captured and replayed."""
    T, H, I, E, k = 21, 256, 96, 8, 2
    rs = np.random.default_rng(14)
    layer, mats = make_layer(rs, E, H, I)
    shared, smats = make_layer(rs, 1, H, I)
    router = moeq.I8Linear.quantized(rnd(rs, (E, H), torch.float32))
    r, y = rnd(rs, (T, H), torch.bfloat16), rnd(rs, (T, H), torch.bfloat16)
    w, pw, w2 = (rnd(rs, (H,), torch.bfloat16) for _ in range(3))

    def step():
        r1, _, q, s = moeq.block_residual(r, y, w, post_w=pw, codes=True, out=False)
        logits = moeq.linear_i8(router, q, s, out_dtype=torch.float32)
        ids, tw, _, offsets, perm, inv = moeq.route_permute(logits, k)
        yp = moeq.expert_ffn_i8(layer, q, perm, offsets, k, s)
        ys = moeq.shared_ffn_i8(shared, q, s)
        r2, n = moeq.combine_residual(r1, yp, inv, tw, w2, y_shared=ys, post_w=pw)
        return dict(r1=r1, q=q, s=s, logits=logits, ids=ids, tw=tw, offsets=offsets, perm=perm,
                    inv=inv, yp=yp, ys=ys, r2=r2, n=n)

    v = step()
    torch.cuda.synchronize()
    q, s = v["q"].cpu().numpy()[:, :H], v["s"].cpu().numpy()
    check_rows(shared, smats, 0, q, s, v["ys"], "shared")
    off, tok = v["offsets"].cpu().numpy(), v["perm"].cpu().numpy() // k
    for e in range(E):
        rows = slice(off[e], off[e + 1])
        if off[e] < off[e + 1]:
            check_rows(layer, mats, e, q[tok[rows]], s[tok[rows]], v["yp"][rows], "experts")
    b, bmag = ob.gated_sum(f64(v["yp"]), v["inv"].cpu().numpy(), f64(v["tw"]), f64(v["ys"]))
    ref_r, rmag, ref_n, nmag = ob.block(f64(v["r1"]), b, f64(w2), f64(pw), y_mag=bmag)
    for got, ref, mag in ((v["r2"], ref_r, rmag), (v["n"], ref_n, nmag)):
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -17 * mag
        assert np.all(np.abs(f64(got) - ref) <= tol)

    f = moeq.forward_i8(layer, v["q"], v["logits"], k, shared=shared, scale=v["s"])
    b, bmag = ob.gated_sum(f64(f["y_perm"]), f["inv_perm"].cpu().numpy(), f64(f["topk_w"]),
                           f64(f["y_shared"]))
    assert np.all(np.abs(f64(f["out"]) - b) <= 2.0 ** -18 * bmag)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        held = step()
    for i in range(4):
        y.copy_(rnd(rs, (T, H), torch.bfloat16))
        now = step()
        g.replay()
        torch.cuda.synchronize()
        for name in now:
            if name == "q":
                assert torch.equal(now[name][:, :H], held[name][:, :H])
            else:
                assert torch.equal(now[name], held[name]), (i, name)


def test_codes_or_float_rows_from_slices():
    """A layer fed from columns of a wider tensor, and from code rows that lie
    further apart."""
    rs = np.random.default_rng(17)
    layer, _ = make_layer(rs, 1, 96, 48)
    for T in (3, 30):
        wide = rnd(rs, (T, 300), torch.bfloat16)
        for a in (0, 5):
            x = wide[:, a:a + 96]
            ref = moeq.shared_ffn_i8(layer, x.contiguous())
            assert torch.equal(moeq.shared_ffn_i8(layer, x), ref)
            q, s = moeq.quantize_i8(x)
            big = torch.full((T, 512), 99, dtype=torch.int8, device=DEV)
            big[:, 64:64 + 128] = q
            assert torch.equal(moeq.shared_ffn_i8(layer, big[:, 64:64 + 128], s, y_dtype=x.dtype), ref)


def test_refusals_of_shapes():
    rs = np.random.default_rng(18)
    layer, _ = make_layer(rs, 4, 96, 48)
    lin = moeq.I8Linear(codes(rs, (48, 96)), scales(rs, 48))
    x = rnd(rs, (5, 96), torch.bfloat16)
    q, s = moeq.quantize_i8(x)
    ids = torch.zeros((5, 1), dtype=torch.int32, device=DEV)
    _, off, perm, _ = moeq.permute(ids, 4)
    for call in (lambda: moeq.linear_i8(lin, x[:, :95]), lambda: moeq.linear_i8(lin, x.t()),
                 lambda: moeq.linear_i8(lin, x.double()), lambda: moeq.linear_i8(lin, q),
                 lambda: moeq.linear_i8(lin, x, s), lambda: moeq.linear_i8(lin, q[:, :96], s),
                 lambda: moeq.linear_i8(lin, q, s[:4]),
                 lambda: moeq.linear_i8(lin, x, out=torch.empty((5, 47), device=DEV)),
                 lambda: moeq.linear_i8(lin, x, out=torch.empty((5, 48))),
                 lambda: moeq.linear_i8(lin, x, ws=torch.empty(9999)),
                 lambda: moeq.expert_ffn_i8(layer, x, perm, off[:4], 1),
                 lambda: moeq.expert_ffn_i8(layer, x, perm.long(), off, 1),
                 lambda: moeq.expert_ffn_i8(layer, x, perm, off, 2),
                 lambda: moeq.expert_ffn_i8(layer, x.cpu(), perm, off, 1),
                 lambda: moeq.block_norm(x, torch.ones(95, device=DEV)),
                 lambda: moeq.block_norm(x, torch.ones(96)),
                 lambda: moeq.block_residual(x, x[:4], None),
                 lambda: moeq.block_residual(x, x, torch.ones(96, device=DEV), post_w=x[0]),
                 lambda: moeq.block_residual(x, x, None, gate=torch.ones((3, 1), device=DEV)),
                 lambda: moeq.block_residual(x, x, None, gate=torch.ones(96, device=DEV)),
                 lambda: moeq.block_residual(x, x, None, r_out=x.float()),
                 lambda: moeq.block_norm(x, x[0], codes=True, q=q[:, :96]),
                 lambda: moeq.I8Linear(codes(rs, (48, 96)), scales(rs, 47)),
                 lambda: moeq.I8Layer(codes(rs, (2, 96, 64)), scales(rs, (2, 96)),
                                      codes(rs, (2, 64, 47)), scales(rs, (2, 64)))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: moeq.shared_ffn_i8(layer, x),
                 lambda: moeq.linear_i8(lin, x, ws=torch.empty(8, dtype=torch.uint8, device=DEV)),
                 lambda: moeq.block_norm(x, None)):
        with pytest.raises(moeq.MoeError):
            call()


def test_gated_sum_is_combine():
    """combine_residual without a residual stream gives the bits of combine and
    combine_shared on fp32 rows."""
    T, k, H, E = 13, 4, 200, 8
    rs = np.random.default_rng(19)
    logits = torch.from_numpy(rs.standard_normal((T, E)).astype(np.float32)).to(DEV)
    _, tw, _, _, _, inv = moeq.route_permute(logits, k)
    y, ys = rnd(rs, (T * k, H), torch.float32), rnd(rs, (T, H), torch.float32)
    assert torch.equal(moeq.combine_residual(None, y, inv, tw)[0], moeq.combine(y, inv, tw))
    assert torch.equal(moeq.combine_residual(None, y, inv, tw, y_shared=ys)[0],
                       moeq.combine_shared(y, inv, tw, ys))


def test_side_stream():
    rs = np.random.default_rng(15)
    layer, _ = make_layer(rs, 1, 128, 64)
    x = rnd(rs, (50, 128), torch.bfloat16)
    ref = moeq.shared_ffn_i8(layer, x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = moeq.shared_ffn_i8(layer, x)
    side.synchronize()
    assert torch.equal(y, ref)


def test_routed_oracle_of_the_whole_layer():
    """forward_i8 against forward's fp64 oracle on the dequantised weights, at
    8-bit precision.  A code is off by at most half of 1/127 of its row's
    largest value (about 4 RMS), RMS error 4 / 127 / sqrt(12) = 0.9% of the row's
    RMS; x, the gate and up weights, h and the down weights each add that (x and
    the weights twice, through g and u): 0.9% * sqrt(6) = 2.3%; a row's RMS error
    stays under twice that."""
    T, H, I, E, k = 24, 512, 256, 8, 2
    rs = np.random.default_rng(16)
    gate, up, down = (torch.from_numpy((rs.standard_normal(sh) * 0.05).astype(np.float32)).to(DEV)
                      for sh in ((E, I, H), (E, I, H), (E, H, I)))
    layer = moeq.I8Layer.quantized(gate, up, down)
    x = rnd(rs, (T, H), torch.bfloat16)
    logits = torch.from_numpy(rs.standard_normal((T, E)).astype(np.float32)).to(DEV)
    r = moeq.forward_i8(layer, x, logits, k)
    bits = x.view(torch.int16).cpu().numpy().view(np.uint16)
    mats = [t.cpu().numpy().astype(np.float64) for t in (gate, up, down)]
    out, ids, w, y = oracle.forward(bits, logits.cpu().numpy(), k,
                                    lambda e: [m[e] for m in mats])
    assert np.array_equal(r["topk_ids"].cpu().numpy(), ids)
    err = np.abs(r["out"].cpu().numpy() - out)
    rel = np.sqrt((err ** 2).mean(1) / (out * out).mean(1))
    assert rel.max() <= 0.046, rel.max()


@pytest.mark.parametrize("dt", sorted(TYPES))
def test_rows_do_not_depend_on_the_batch(dt):
    """A row's bits are the same in every kernel that its batch leads to."""
    rs = np.random.default_rng(31)
    K, N, T = 712, 1330, 700
    lin = moeq.I8Linear(codes(rs, (N, K)), scales(rs, N), rnd(rs, (N,), torch.float32))
    shared = moeq.I8Layer(codes(rs, (1, 2 * N, K)), scales(rs, 2 * N).view(1, -1),
                          codes(rs, (1, K, N)), scales(rs, K).view(1, -1))
    x = rnd(rs, (T, K), TYPES[dt], 2.0)
    full, ffn = moeq.linear_i8(lin, x), moeq.shared_ffn_i8(shared, x)
    for a, n in ((0, 1), (5, 4), (300, 16), (1, 30), (400, 120), (350, 350)):
        say("rows", dt, a, n)
        assert torch.equal(moeq.linear_i8(lin, x[a:a + n]), full[a:a + n])
        assert torch.equal(moeq.shared_ffn_i8(shared, x[a:a + n]), ffn[a:a + n])


def test_graphs_of_the_products():
    """Two graphs, each with its own memory, replayed in turn with eager calls
    between them, on new inputs."""
    rs = np.random.default_rng(32)
    E, H, I, k = 8, 328, 200, 2
    layer = moeq.I8Layer(codes(rs, (E, 2 * I, H)), scales(rs, E * 2 * I).view(E, -1),
                         codes(rs, (E, H, I)), scales(rs, E * H).view(E, -1))
    lin = moeq.I8Linear(codes(rs, (264, H)), scales(rs, 264))
    sets = []
    for T in (3, 150):
        x = rnd(rs, (T, H), torch.bfloat16)
        logits = rnd(rs, (T, E), torch.float32)
        _, tw, _, off, src, inv = moeq.route_permute(logits, k)

        def step(x=x, tw=tw, off=off, src=src, inv=inv):
            y = moeq.expert_ffn_i8(layer, x, src, off, k)
            r, n = moeq.combine_residual(x, y, inv, tw, torch.ones_like(x[0]))
            return moeq.linear_i8(lin, n), r

        for _ in range(2):
            step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        sets.append((T, x, step, g, out))
    for i in range(4):
        for T, x, step, g, out in sets:
            say("replay", i, T)
            x.copy_(rnd(rs, (T, H), torch.bfloat16))
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, step()):
                assert torch.equal(a, b), (i, T)
