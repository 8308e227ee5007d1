"""What the sequence operators keep for their backward passes and refuse at their raw calls, on the GPU."""
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


def test_raw_calls_refuse_states_of_another_size():
    B, H, N, D = 2, 2, 40, 64
    q, k, v, do, o, dq, dk, dv = (torch.randn(B, H, N, D, device="cuda") for _ in range(8))
    a = torch.tensor([-0.1, -0.01], device="cuda")
    shape = llsa.make_linear_shape(B, H, N, D, torch.float32)
    for n in (B - 1, B + 1):  # a pool of other states is not a batch's
        pool = torch.zeros(n, H, D, D, device="cuda")
        for name in ("initial_state", "final_state"):
            with pytest.raises(ValueError, match=name):
                llsa.llsa_linear_forward(shape, q, k, v, a, o, **{name: pool})
        for name in ("initial_state", "d_final", "d_initial"):
            with pytest.raises(ValueError, match=name):
                llsa.llsa_linear_backward(shape, q, k, v, do, a, dq, dk, dv, **{name: pool})
    roomy = torch.zeros(1000, device="cuda")  # scratch may be larger than needed
    llsa.llsa_linear_forward(shape, q, k, v, a, o, states=roomy)
    assert torch.equal(o, llsa.llsa_linear_attention(q, k, v, a)) and llsa.llsa_device_status() == 0


def test_tensors_written_in_place_count_as_written():
    """An earlier operation that saved one of them refuses its backward, as with torch's own in-place
    operations."""
    B, H, N, D = 2, 2, 40, 64
    q, k, v, do, o, dq, dk, dv = (torch.randn(B, H, N, D, device="cuda") for _ in range(8))
    s0, fin, ds0 = (torch.randn(B, H, D, D, device="cuda") for _ in range(3))
    a, f = torch.tensor([-0.1, -0.01], device="cuda"), llsa.llsa_rotary_frequencies(D, device="cuda")[0]
    shape = llsa.make_linear_shape(B, H, N, D, torch.float32)
    one, out = [t[:, :, 0].contiguous() for t in (q, k, v)], torch.empty(B, H, D, device="cuda")
    for call, written in (
            (lambda: llsa.llsa_rotary(q, k, None, f, inplace=True), (q, k)),
            (lambda: llsa.llsa_linear_step(*one, a, s0), (s0,)),
            (lambda: llsa.llsa_linear_step(*one, a, s0, out=out), (s0, out)),
            (lambda: llsa.llsa_linear_forward(shape, q, k, v, a, o, None, None, s0, fin), (o, fin)),
            (lambda: llsa.llsa_linear_backward(shape, q, k, v, do, a, dq, dk, dv, initial_state=s0, d_initial=ds0),
             (dq, dk, dv, ds0))):
        for t in written:
            w = torch.ones_like(t, requires_grad=True)
            y = w * t
            call()
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                y.sum().backward()
    with torch.inference_mode():
        pool = torch.randn(B, H, D, D, device="cuda")
    llsa.llsa_linear_step(*one, a, pool)


def test_gradients_own_their_memory():
    """A gradient that is kept holds no other's memory, and writing one is no write of another."""
    leaves = [torch.randn(1, 2, 200, 64, device="cuda", requires_grad=True) for _ in range(3)]
    o = llsa.llsa_linear_attention(*leaves, torch.tensor([-0.1, -0.01], device="cuda"))
    grads = torch.autograd.grad(o, leaves, torch.randn_like(o))
    for g in grads:
        assert g.untyped_storage().nbytes() == g.numel() * g.element_size() and not g._is_view()
    before = [g._version for g in grads]
    grads[0].mul_(2)
    assert [g._version for g in grads[1:]] == before[1:]
