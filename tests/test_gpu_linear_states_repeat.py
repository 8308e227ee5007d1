"""Many launches that return states and their gradients, over uneven segment and chunk counts and on two
streams at once: every one gives the same bits, and no wait of the kernels gives up."""
import pytest
import torch

import log_linear_hierarchical_b200 as llsa

pytestmark = pytest.mark.gpu


def make(B, H, N, D, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = [torch.randn(B, H, N, D, device="cuda", generator=g).bfloat16() for _ in range(4)]
    return x, [torch.randn(B, H, D, D, device="cuda", generator=g) for _ in range(2)]


def step(x, states, a, lengths):
    leaves = [t.detach().requires_grad_() for t in (*x[:3], states[0])]
    o, fin = llsa.llsa_linear_attention(*leaves[:3], a, initial_state=leaves[3], lengths=lengths, return_state=True)
    return [o.detach(), fin.detach(), *torch.autograd.grad([o, fin], leaves, [x[3], states[1]])]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H,N", [(1, 1, 20000), (1, 6, 9000), (3, 5, 2500), (40, 5, 700), (300, 1, 130)])
def test_repeats(D, B, H, N):
    x, states = make(B, H, N, D, N)
    a = torch.linspace(-0.3, -0.001, H, device="cuda")
    lengths = torch.tensor([N - (13 * b) % N for b in range(B)], device="cuda", dtype=torch.int32)
    first = step(x, states, a, lengths)
    for _ in range(40):
        assert all(torch.equal(s, t) for s, t in zip(step(x, states, a, lengths), first))
    assert llsa.llsa_device_status() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H,N", [(2, 3, 3000), (60, 3, 500)])
def test_two_streams(D, B, H, N):
    a = torch.tensor([-0.01, -0.2, 0.0], device="cuda")
    sets = [make(B, H, N, D, s) for s in (1, 2)]
    want = [step(*s, a, None) for s in sets]
    streams, got = [torch.cuda.Stream() for _ in sets], [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(*sets[i], a, None))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(s, t) for r in got[i] for s, t in zip(r, want[i]))
    assert llsa.llsa_device_status() == 0


@pytest.mark.parametrize("D,N", [(64, 300), (128, 300), (64, 3000), (128, 4000)])
def test_outputs_differ_by_roundings_only_whether_or_not_states_are_returned(D, N):
    """Asked for a state, a call whose sequences are whole gives the tokens in it more digits; what of that
    reaches o and dv is a rounding of the state's copy, 2^-8 of a term, and of the result."""
    x, states = make(1, 3, N, D, 5)
    a = torch.tensor([-0.01, -0.2, 0.0], device="cuda")
    with torch.no_grad():
        o, _ = llsa.llsa_linear_attention(*x[:3], a, return_state=True)
        p = llsa.llsa_linear_attention(*x[:3], a)
    # two results, each off by at most sqrt(2 / 3) 2^-8 of it in the mean square
    assert (o.double() - p.double()).norm() <= 2 * (2 / 3) ** 0.5 * 2.0 ** -8 * p.double().norm()
