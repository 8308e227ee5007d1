"""Many launches over uneven segment and chunk counts: every one gives the same bits, and no wait of
the kernels gives up (a wait that misses its phase runs into its limit and records a timeout)."""
import pytest
import torch

import log_linear_hierarchical_b200 as llsa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H,N", [(1, 1, 20000), (1, 6, 9000), (3, 5, 2500), (40, 5, 700), (300, 1, 130)])
def test_repeats(D, B, H, N):
    g = torch.Generator(device="cuda").manual_seed(N)
    q, k, v, do = (torch.randn(B, H, N, D, device="cuda", generator=g).bfloat16() for _ in range(4))
    a = torch.linspace(-0.3, -0.001, H, device="cuda")
    s0 = torch.randn(B, H, D, D, device="cuda", generator=g)
    leaves = [t.requires_grad_() for t in (q, k, v)]
    first = None
    for _ in range(60):
        o, fin = llsa.llsa_linear_attention(q, k, v, a, initial_state=s0, return_state=True)
        got = [o.detach(), fin.detach(), *torch.autograd.grad(o, leaves, do)]
        if first is None:
            first = got
        else:
            assert all(torch.equal(x, y) for x, y in zip(got, first))
    assert llsa.llsa_device_status() == 0
