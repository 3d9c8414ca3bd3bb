"""Outputs that a 4-bit call would leave as they were are refused (no GPU needed)."""
import pytest
import torch

import combine_router_top_amd as M


def test_zero_points_that_are_not_made():
    w = torch.zeros((128, 16))
    out = (torch.zeros(M.packed_weights_4bit_shape(128, 16), dtype=torch.int32), torch.zeros((1, 16), dtype=torch.bfloat16),
           torch.zeros((1, 16), dtype=torch.uint8))
    with pytest.raises(ValueError, match="zero points"):
        M.quantize_weights_4bit(w, 128, False, out=out)
