"""The 8-bit codes of every kernel that makes them, at and next to ties: equal to
the exact quotients' rounding."""

import numpy as np
import pytest
import torch

import bit_quantized_moe_route_amd as moeq
from oracle import block as ob
from tests.gpu_common import say

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def halves(dt, width):
    """A row for every mantissa of dt (512 of fp32's): its largest magnitude, plus
    and minus half of it, and other values of the type."""
    bits = {"bf16": 7, "fp16": 10, "fp32": 9}[dt]
    n = 1 << bits
    rs = np.random.default_rng(width)
    top = 1 + torch.arange(n, dtype=torch.float64) / n
    if dt == "fp32":
        top += torch.from_numpy(rs.integers(0, 1 << 14, n)) * 2.0 ** -23
    x = torch.from_numpy(rs.uniform(-1, 1, (n, width))).to(TYPES[dt]).double() * 0.99
    x[:, 0], x[:, width // 2], x[:, width - 1] = top / 2, -top, -top / 2
    return x.to(TYPES[dt]).to(DEV)


def near_ties(width):
    """fp32 rows of values as near to (n + 1/2) a / 127 as the type comes."""
    rs = np.random.default_rng(7)
    rows = []
    for scale in (1.0, 2.0 ** 127, 2.0 ** -118):
        for _ in range(24):
            a = np.float32(rs.uniform(1, 1.99) * scale)
            v = ((rs.integers(0, 127, width) + 0.5) * float(a) / 127).astype(np.float32)
            step = rs.integers(-1, 2, width)
            v = np.where(step < 0, np.nextafter(v, np.float32(0)),
                         np.where(step > 0, np.nextafter(v, np.float32(np.inf)), v))
            v = np.minimum(v, a) * rs.choice([-1, 1], width)
            v[rs.integers(0, width)] = a
            rows.append(v.astype(np.float32))
    return torch.from_numpy(np.stack(rows)).to(DEV)


def inputs(dt, width):
    x = [halves(dt, width)]
    return x + [near_ties(width)] if dt == "fp32" else x


def same(q, x, what):
    ref, _ = ob.quantize_i8(x.float().cpu().numpy())
    got = q[:, :x.shape[1]].cpu().numpy()
    bad = np.argwhere(got != ref)
    assert len(bad) == 0, (what, len(bad), bad[:3].tolist())


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("width", [5, 64, 203, 1024, 8200, 40000])
def test_quantize_at_ties(dt, width):
    """Rows in registers, in registers four chunks a thread, and read twice; on and
    off 16 bytes."""
    for x in inputs(dt, width):
        say("quantize ties", dt, tuple(x.shape))
        q, _ = moeq.quantize_i8(x)
        same(q, x, (dt, width))
        wide = torch.zeros((x.shape[0], width + 3), dtype=x.dtype, device=DEV)
        wide[:, 1:1 + width] = x
        q, _ = moeq.quantize_i8(wide[:, 1:1 + width])
        same(q, x, (dt, width, "off 16 bytes"))


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("H", [5, 203, 1024, 8200, 20000])
def test_block_norm_codes_at_ties(dt, H):
    """The codes that a block norm makes of its result (here r itself, no weights)."""
    for x in inputs(dt, H):
        say("block ties", dt, tuple(x.shape))
        zero = torch.zeros_like(x)
        r, n, q, s = moeq.block_residual(x, zero, None, codes=True)
        assert n is None and torch.equal(r, x)
        same(q, x, (dt, H))
        assert torch.equal(s, moeq.quantize_i8(x)[1])


def test_codes_of_a_norm_are_those_of_its_fp32_result():
    rs = np.random.default_rng(3)
    r = torch.from_numpy(rs.standard_normal((700, 520))).to(torch.bfloat16).to(DEV)
    w = torch.ones(520, dtype=torch.bfloat16, device=DEV)
    n, q, s = moeq.block_norm(r, w, out_dtype=torch.float32, codes=True)
    same(q, n, "n")
    q2, s2 = moeq.quantize_i8(n)
    assert torch.equal(q2[:, :520], q[:, :520]) and torch.equal(s2, s)


@pytest.mark.parametrize("dt", sorted(TYPES))
@pytest.mark.parametrize("K", [40, 203])
@pytest.mark.parametrize("T", [1, 3, 4])
def test_linear_codes_rows_itself_at_ties(dt, K, T):
    """Few rows are coded inside the product: an identity gives the codes back."""
    lin = moeq.I8Linear(torch.eye(K, dtype=torch.int8, device=DEV), torch.ones(K, device=DEV))
    for x in inputs(dt, K):
        ref, scale = ob.quantize_i8(x.float().cpu().numpy())
        for a in range(0, x.shape[0] - T + 1, T):
            out = moeq.linear_i8(lin, x[a:a + T], out_dtype=torch.float32).cpu().numpy()
            want = ref[a:a + T] * scale[a:a + T, None]
            assert np.array_equal(out, want.astype(np.float32)), (dt, K, a)


def test_shared_ffn_of_rows_with_ties():
    """Two rows that hold a tie, through a shared expert, over many seeds: y stays
    at fp32's rounding (plus what codes of h within rounding of a tie can add)."""
    H, I = 520, 72
    for seed in range(100):
        rs = np.random.default_rng(seed)
        w13 = rs.integers(-128, 128, (1, 2 * I, H)).astype(np.int8)
        w2 = rs.integers(-128, 128, (1, H, I)).astype(np.int8)
        s13 = (np.exp(rs.standard_normal((1, 2 * I)) * 0.3) * 0.01 / H ** 0.5).astype(np.float32)
        s2 = (np.exp(rs.standard_normal((1, H)) * 0.3) * 0.01).astype(np.float32)
        layer = moeq.I8Layer(*(torch.from_numpy(t).to(DEV) for t in (w13, s13, w2, s2)))
        x = torch.from_numpy(rs.standard_normal((2, H))).to(torch.bfloat16)
        top = x.float().abs().amax(1)
        x[:, 1], x[:, H - 2] = (top / 2).to(x.dtype), (-top / 2).to(x.dtype)
        y = moeq.shared_ffn_i8(layer, x.to(DEV), y_dtype=torch.float32)
        q, s = ob.quantize_i8(x.float().numpy())
        g = ob.product_i8(q, w13[0, :I]) * s[:, None].astype(np.float64) * s13[0, :I]
        # h as in the other tests of these products: exp's argument and the division
        eps_h = np.abs(g).max() * 2.0 ** -23 + 2.0 ** -20
        ref, slack, _ = ob.expert_i8(q, s, w13[0], s13[0], w2[0], s2[0], eps_h)
        tol = (2.0 ** -24 + 2.0 ** -20) * np.abs(ref) + 1.01 * slack
        err = np.abs(y.double().cpu().numpy() - ref)
        assert np.all(err <= tol), (seed, float((err / np.maximum(tol, 1e-300)).max()))
