"""The oracle's 8-bit codes against rational arithmetic, ties above all."""

from fractions import Fraction

import numpy as np
import torch

from oracle import block as ob


def rational_codes(row):
    a = max(abs(Fraction(float(v))) for v in row)
    return [round(Fraction(float(v)) * 127 / a) for v in row]      # round: ties to even


def test_ties_of_half_the_largest():
    """|v| = a / 2 is the tie 63.5 and goes to 64, for every mantissa of bf16 and fp16."""
    for first, last in ((128, 256), (1024, 2048)):
        for m in range(first, last):
            q, _ = ob.quantize_i8(np.array([[m, m / 2, -m / 2, -m]], np.float32))
            assert q.tolist() == [[127, 64, -64, -127]], m


def test_codes_are_the_quotients_rounded():
    rs = np.random.default_rng(0)
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        x = torch.from_numpy(rs.standard_normal((60, 40))).to(dtype).float().numpy()
        q, _ = ob.quantize_i8(x)
        for t in range(len(x)):
            assert q[t].tolist() == rational_codes(x[t])


def test_codes_next_to_ties():
    """fp32 values at a tie, or as near to one as fp32 comes, on either side; rows
    at both ends of the range."""
    rs = np.random.default_rng(1)
    for scale in (1.0, 2.0 ** 127, 2.0 ** -118):
        for _ in range(40):
            a = np.float32(rs.uniform(1, 1.99) * scale)
            half = (np.arange(127) + 0.5) * float(a) / 127
            v = half.astype(np.float32)
            row = np.concatenate([[a], v, np.nextafter(v, np.float32(0)),
                                  -np.nextafter(v, np.float32(np.inf))[:-1]]).astype(np.float32)
            q, _ = ob.quantize_i8(row[None])
            assert q[0].tolist() == rational_codes(row)
