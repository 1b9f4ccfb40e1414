"""Calls of the block norms that the binding refuses before it looks at a device."""

import pytest
import torch

import bit_quantized_moe_route_amd as moeq


def test_a_gated_sum_needs_slots():
    """No slot at all is not the form without a gated sum (y itself)."""
    r = torch.zeros((3, 64))
    inv = torch.zeros(0, dtype=torch.int32)
    for w in (torch.empty((3, 0)), torch.empty(3)):
        with pytest.raises(ValueError, match="topk_w"):
            moeq.combine_residual(r, r, inv, w, r[0])
