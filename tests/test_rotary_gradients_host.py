"""Rotary positions refuse a gradient that they would not give, before they look at the rest."""
import pytest
import torch

import differentiable_image_quality_gb300 as pkg


@pytest.mark.parametrize("asks", ["positions", "frequencies"])
def test_positions_and_frequencies_that_ask_for_a_gradient(asks):
    q, at = torch.zeros(4, 2, 16), torch.zeros(4, 1)
    f = pkg.rotary_frequencies((4,), device="cpu")
    (at if asks == "positions" else f).requires_grad_()
    with pytest.raises(ValueError, match=asks):
        pkg.fused_rotary(q, None, at, f, (4,))
    with torch.no_grad(), pytest.raises(TypeError, match="q must be a CUDA tensor"):
        pkg.fused_rotary(q, None, at, f, (4,))
    with pytest.raises(TypeError, match="q must be a CUDA tensor"):
        pkg.fused_rotary(q, None, at.detach(), f.detach(), (4,))
