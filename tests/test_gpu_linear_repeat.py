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


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,H,N", [(5, 2, 290), (100, 4, 200), (1, 2, 3000)])
def test_empty_rows_keep_their_state(D, dtype, B, H, N):
    q, k, v, do = (torch.full((B, H, N, D), float("nan"), device="cuda", dtype=dtype) for _ in range(4))
    s0, ds = torch.randn(B, H, D, D, device="cuda"), torch.randn(B, H, D, D, device="cuda")
    a = torch.full((H,), -0.1, device="cuda")
    leaves = [t.requires_grad_() for t in (q, k, v, s0)]
    lengths = torch.zeros(B, device="cuda", dtype=torch.int32)
    for _ in range(20):
        o, fin = llsa.llsa_linear_attention(q, k, v, a, initial_state=s0, lengths=lengths, return_state=True)
        grads = torch.autograd.grad([o, fin], leaves, [do, ds])
        assert torch.equal(fin, s0) and torch.equal(grads[3], ds)
        assert not any(t.any() for t in (o, *grads[:3]))
