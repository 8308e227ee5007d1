"""What the sequence operators keep for their backward passes, on the GPU."""
import pytest
import torch

import log_linear_hierarchical_b200 as llsa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", ["positions", "frequencies"])
def test_rotary_refuses_a_gradient_at_rewritten_positions(which):
    q = torch.randn(1, 2, 8, 64, device="cuda", requires_grad=True)
    held = dict(positions=torch.arange(8, device="cuda"), frequencies=llsa.llsa_rotary_frequencies(64, device="cuda")[0])
    y = llsa.llsa_rotary(q, None, held["positions"], held["frequencies"])
    dy = torch.randn_like(y)
    (before,) = torch.autograd.grad(y, q, dy, retain_graph=True)
    assert torch.equal(torch.autograd.grad(y, q, dy, retain_graph=True)[0], before)
    held[which].mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad(y, q, dy)
