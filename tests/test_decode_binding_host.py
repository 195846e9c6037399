"""moe_decode's checks of shapes, made before anything of the device is asked."""

from types import SimpleNamespace

import pytest
import torch

from combine_top_route_moe_amd import ops


@pytest.mark.parametrize("shape", [(2, 4, 3), (2,), (8,), (1, 4), (2, 4, 1)])
def test_logits_are_a_matrix(shape):
    """(More dimensions would be read as rows of the first two.)"""
    weights = SimpleNamespace(H=256, I=128, num_groups=4, w13=torch.zeros(1))
    x = torch.zeros(2, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match=r"logits must be \[T, num_experts\]"):
        ops.moe_decode(torch.zeros(shape), x, 2, weights)
