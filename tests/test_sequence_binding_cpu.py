"""What the Python side of the sequence operators does before and around the kernels, on host
tensors: the kernels' launch is replaced where a call has to get past it."""
import pytest
import torch
from torch.autograd import forward_ad

import log_linear_hierarchical_b200 as llsa
from log_linear_hierarchical_b200 import rotary


def fake_rotate(xs, outs, positions, frequencies, interleaved, first, scale, inverse):
    """A pass that depends on the positions and frequencies of the moment."""
    turn = (positions[:, None] * frequencies[0]).to(xs[0].dtype)
    return [t * (scale - turn if inverse else scale + turn) for t in xs]


@pytest.mark.parametrize("which", ["positions", "frequencies"])
def test_rotary_gradient_sees_a_rewritten_buffer(monkeypatch, which):
    monkeypatch.setattr(rotary, "_rotate", fake_rotate)
    q, k = (torch.randn(1, 2, 8, 64, requires_grad=True) for _ in range(2))
    held = dict(positions=torch.arange(8), frequencies=torch.ones(32, dtype=torch.float64))
    y, z = rotary.llsa_rotary(q, k, held["positions"], held["frequencies"])
    torch.autograd.grad([y, z], [q, k], [torch.ones_like(y)] * 2, retain_graph=True)
    held[which].add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        torch.autograd.grad([y, z], [q, k], [torch.ones_like(y)] * 2)


def test_rotary_gradient_without_positions(monkeypatch):
    seen = []
    monkeypatch.setattr(rotary, "_rotate", lambda xs, outs, *a: seen.append(a) or [t.clone() for t in xs])
    q = torch.randn(1, 2, 8, 64, requires_grad=True)
    f = torch.ones(32, dtype=torch.float64)
    y = rotary.llsa_rotary(q, None, None, f, interleaved=True, first=2, scale=0.5)
    torch.autograd.grad(y, q, torch.ones_like(y))
    assert [(a[0], a[2:]) for a in seen] == [(None, (True, 2, 0.5, False)), (None, (True, 2, 0.5, True))]
    assert all(torch.equal(a[1], f) for a in seen)


def test_rotary_gradient_with_a_table_made_in_inference_mode(monkeypatch):
    monkeypatch.setattr(rotary, "_rotate", fake_rotate)
    with torch.inference_mode():
        pos, f = torch.arange(8), torch.ones(32, dtype=torch.float64)
    q = torch.randn(1, 2, 8, 64, requires_grad=True)
    y = rotary.llsa_rotary(q, None, pos, f)
    (g,) = torch.autograd.grad(y, q, torch.ones_like(y))
    assert torch.equal(g, (1 - torch.arange(8.0))[:, None].expand(1, 2, 8, 64))


DUAL = "forward-mode"


@pytest.mark.parametrize("which", range(3))
def test_rotary_refuses_a_tangent(which):
    args = [torch.randn(1, 2, 8, 64), torch.randn(1, 2, 8, 64), torch.ones(32, dtype=torch.float64)]
    with forward_ad.dual_level():
        args[which] = forward_ad.make_dual(args[which], torch.ones_like(args[which]))
        with pytest.raises(ValueError, match=DUAL):
            llsa.llsa_rotary(args[0], args[1], None, args[2])


@pytest.mark.parametrize("which", range(5))
def test_linear_attention_and_step_refuse_a_tangent(which):
    tokens, state = [torch.randn(1, 2, 8, 64) for _ in range(3)], torch.zeros(1, 2, 64, 64)
    args = [*tokens, torch.zeros(2), state]
    one = [t[:, :, 0] for t in tokens] + args[3:]
    with forward_ad.dual_level():
        for a in (args, one):
            a[which] = forward_ad.make_dual(a[which], torch.ones_like(a[which]))
        with pytest.raises(ValueError, match=DUAL):
            llsa.llsa_linear_attention(*args[:4], initial_state=args[4])
        with pytest.raises(ValueError, match=DUAL):
            llsa.llsa_linear_step(*one)


def test_a_dual_level_alone_refuses_nothing():
    x = torch.randn(1, 2, 8, 64)
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="CUDA tensors"):
            llsa.llsa_linear_attention(x, x, x, torch.zeros(2))


def test_rotary_gradient_refuses_a_tangent(monkeypatch):
    monkeypatch.setattr(rotary, "_rotate", fake_rotate)
    q = torch.randn(1, 2, 8, 64, requires_grad=True)
    y = rotary.llsa_rotary(q, None, torch.arange(8), torch.ones(32, dtype=torch.float64))
    with forward_ad.dual_level():
        dy = forward_ad.make_dual(torch.ones_like(y), torch.ones_like(y))
        with pytest.raises(ValueError, match=DUAL):
            torch.autograd.grad(y, q, dy)


def test_raw_calls_refuse_host_tensors():
    x, a = torch.zeros(1, 2, 8, 64), torch.zeros(2)
    shape = llsa.make_linear_shape(1, 2, 8, 64, torch.float32)
    for call in (lambda: llsa.llsa_linear_forward(shape, x, x, x, a, x.clone()),
                 lambda: llsa.llsa_linear_backward(shape, x, x, x, x, a, x.clone(), x.clone(), x.clone())):
        with pytest.raises(ValueError, match="CUDA tensors"):
            call()


@pytest.mark.parametrize("shape", [(1,), (4,), (3, 2), (3, 2, 8), (2, 1), (1, 2), ()])
def test_a_log_decay_of_another_shape_is_refused(shape):
    """One value a head: a decay for each request or token is another operator."""
    x, a = torch.zeros(3, 2, 8, 64), torch.zeros(shape)
    spec = llsa.make_linear_shape(3, 2, 8, 64, torch.float32)
    for call in (lambda: llsa.llsa_linear_attention(x, x, x, a),
                 lambda: llsa.llsa_linear_attention(x.clone().requires_grad_(), x, x, a),
                 lambda: llsa.llsa_linear_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], a, torch.zeros(3, 2, 64, 64)),
                 lambda: llsa.llsa_linear_forward(spec, x, x, x, a, x.clone()),
                 lambda: llsa.llsa_linear_backward(spec, x, x, x, x, a, x.clone(), x.clone(), x.clone())):
        with pytest.raises(ValueError, match="log_decay"):
            call()


@pytest.mark.parametrize("which", range(2))
def test_rotary_in_place_counts_as_a_write(monkeypatch, which):
    def turn_in_place(xs, outs, *rest):
        for t in outs:
            t.data.mul_(2)  # as the kernel does, unseen by torch
        return outs

    monkeypatch.setattr(rotary, "_rotate", turn_in_place)
    w, f = torch.ones(1, 2, 8, 64, requires_grad=True), torch.ones(32, dtype=torch.float64)
    x = [torch.randn(1, 2, 8, 64) for _ in range(2)]
    y = w * x[which]
    rotary.llsa_rotary(x[0], x[1], None, f, inplace=True)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    with torch.inference_mode():
        free = torch.ones(1, 2, 8, 64)
    assert rotary.llsa_rotary(free, None, None, f, inplace=True) is free  # (counts no versions)


def test_step_refuses_an_output_that_requires_grad():
    x = torch.zeros(1, 2, 64)
    with pytest.raises(ValueError, match="no gradients"):
        llsa.llsa_linear_step(x, x, x, torch.zeros(2), torch.zeros(1, 2, 64, 64), out=x.clone().requires_grad_())


def test_a_q_of_another_rank_is_refused_beside_a_state():
    x, a, s0 = torch.zeros(1, 2, 8, 64), torch.zeros(2), torch.zeros(1, 2, 64, 64)
    for q in (x[0], x[0, 0], x[None]):
        for state in (None, s0):
            with pytest.raises(ValueError, match="expected .B, H, N, D"):
                llsa.llsa_linear_attention(q, x, x, a, initial_state=state)


def test_no_channels_are_refused_as_any_other_head_width():
    assert llsa.llsa_linear_validate(llsa.make_linear_shape(1, 2, 8, 0, torch.float32)) == 1
    assert llsa.llsa_linear_validate(llsa.make_linear_shape(1, 2, 8, -64, torch.float32)) == 1
    x = torch.zeros(1, 2, 8, 0)
    with pytest.raises(llsa.LLSAError):
        llsa.llsa_linear_attention(x, x, x, torch.zeros(2))
    with pytest.raises(ValueError):  # (host tensors; a ZeroDivisionError is none)
        llsa.llsa_linear_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], torch.zeros(2), torch.zeros(1, 2, 0, 0))
