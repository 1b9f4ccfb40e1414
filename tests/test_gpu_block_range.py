"""Block norms of rows whose squares leave fp32's range, against the fp64 oracle at
the tolerance of ordinary rows (the scaling by a power of two rounds nothing)."""

import numpy as np
import pytest
import torch

import bit_quantized_moe_route_amd as moeq
from oracle import block as ob
from tests.gpu_common import say
from tests.test_gpu_block import REL32, close_codes, f64

pytestmark = pytest.mark.gpu

DEV = "cuda"


def close(got, ref, mag, what):
    """The other block norm tests' tolerance for fp32, and for results below fp32's
    normal range: v * rstd rounded to 2^-150 at worst, times |w| < 6, and the
    result's own rounding, 7 * 2^-150."""
    tol = 2.0 ** -24 * np.abs(ref) + (1 + 2.0 ** -24) * REL32 * mag + 2.0 ** -147
    err = np.abs(f64(got) - ref)
    assert np.all(err <= tol), (what, float((err / tol).max()), np.argmax(err / tol))


def rows(T, H, scales, dtype, seed):
    rs = np.random.default_rng(seed)
    x = rs.standard_normal((T, H)).clip(-3, 3) * np.asarray(scales, np.float64)[:, None]
    return torch.from_numpy(x.astype(np.float32)).to(dtype).to(DEV)


SCALES = [1.0, 1e20, 1e38, 1e-25, 1e-19, 1e-37, 1e18, 3e-41]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("eps", [0.0, 1e-42, 1e-31, 1e-5])
@pytest.mark.parametrize("H", [1, 7, 64, 1003, 6144, 8200, 20001, 32768])
def test_norm(H, eps, dt):
    say("range", H, eps, dt)
    T = len(SCALES)
    r = rows(T, H, SCALES, dt, H)
    if eps == 0:
        # no row without a square: every value at least a step of its type
        r = torch.where(r == 0, torch.full_like(r, 1e-37), r)
    w = rows(1, H, [1.0], dt, H + 1)[0]
    n, q, s = moeq.block_norm(r, w, eps=eps, out_dtype=torch.float32, codes=True)
    e = float(np.float32(eps))
    _, _, ref, mag = ob.block(f64(r), None, f64(w), eps=e)
    close(n, ref, mag, (H, eps))
    # a row's codes need its largest above 127 * 2^-126
    live = np.abs(ref).max(1) > 2.0 ** -118
    close_codes(q[live], s[live], ref[live], mag[live], H, (H, eps))
    assert torch.equal(n[:1], moeq.block_norm(r[:1], w, eps=eps, out_dtype=torch.float32))


@pytest.mark.parametrize("H", [7, 1003, 6144, 20001])
@pytest.mark.parametrize("T", [8, 2200])
def test_residual(T, H):
    """Both norms at once, in place, many rows: the norm after from far out of
    range, the residual stream too."""
    say("range residual", T, H)
    if T * H > 20000000:
        T = 64
    ys = [1e25, 1.0, 1e-30, 1e37, 1e-38, 1e19, 1e-22, 1e30] * (T // 8)
    rsc = [1.0, 1e22, 1e-30, 1e-24, 1e37, 1e19, 1e-40, 1.0] * (T // 8)
    y, r = rows(T, H, ys, torch.float32, H), rows(T, H, rsc, torch.float32, H + 1)
    w, pw = rows(1, H, [1.0], torch.float32, 2)[0], rows(1, H, [1.0], torch.float32, 3)[0]
    kw = dict(y_scale=0.7, r_scale=1.3, eps=0.0)
    ref_r, rmag, ref_n, nmag = ob.block(f64(r), f64(y), f64(w), f64(pw), **kw)
    got_r, n = moeq.block_residual(r, y, w, post_w=pw, r_out=r, **kw)
    assert got_r is r
    close(r, ref_r, rmag, "r'")
    close(n, ref_n, nmag, "n")


def test_gated_sum():
    T, k, H = 8, 3, 1003
    scales = [1.0, 1e20, 1e37, 1e-25, 1e-19, 1e-30, 1e18, 1e-22]
    y = rows(T * k, H, np.repeat(scales, k), torch.float32, 5)
    r = rows(T, H, scales, torch.float32, 6)
    w = rows(1, H, [1.0], torch.float32, 7)[0]
    rs = np.random.default_rng(8)
    tw = torch.from_numpy(rs.random((T, k)).astype(np.float32)).to(DEV)
    inv = torch.arange(T * k, dtype=torch.int32, device=DEV)
    b, bmag = ob.gated_sum(f64(y), inv.cpu().numpy(), f64(tw))
    ref_r, rmag, ref_n, nmag = ob.block(f64(r), b, f64(w), f64(w), y_mag=bmag, eps=0.0)
    r2, n = moeq.combine_residual(r, y, inv, tw, w, post_w=w, eps=0.0)
    close(r2, ref_r, rmag, "r'")
    close(n, ref_n, nmag, "n")


@pytest.mark.parametrize("H", [40, 1003, 9000])
def test_rows_without_a_norm_stay_apart(H):
    """Infinities and NaNs keep their rows to themselves, zeros with eps 0 are 0 / 0."""
    r = rows(8, H, SCALES, torch.float32, 9)
    w = rows(1, H, [1.0], torch.float32, 10)[0]
    clean = moeq.block_norm(r, w, eps=1e-31, codes=True)
    bad = r.clone()
    bad[1, H - 1], bad[3, 0], bad[6] = float("inf"), float("nan"), 0.0
    n, q, s = moeq.block_norm(bad, w, eps=1e-31, codes=True)
    for t in (0, 2, 4, 5, 7):
        for a, b in zip((n, q, s), clean):
            assert torch.equal(a[t], b[t]), t
    assert torch.isnan(n[1, H - 1]) and torch.all(n[1, :H - 1] == 0) and torch.isnan(n[3]).all()
    assert torch.isnan(s[1]) and torch.isnan(s[3]) and not q[1].any() and not q[3].any()
    assert torch.all(n[6] == 0) and s[6] == 0
    assert torch.isnan(moeq.block_norm(torch.zeros_like(r), w, eps=0.0)).all()
