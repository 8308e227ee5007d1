"""Calls of the sequence operators that a program makes without thinking of them: tensors past
2^32 elements, two streams at once, a thread's first CUDA call, capture while an eager graph lives,
states passed in place, packed projections."""
import threading

import numpy as np
import pytest
import torch

import log_linear_hierarchical_b200 as llsa
from oracle import sequence_ops as so

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def num(t):
    return t.detach().double().cpu().numpy()


def test_offsets_past_32_bits():
    """[3, 12, 2^20, 128] bf16: 4.8e9 elements a tensor.  The last head against the reference on its last
    tokens (a decay of e^-0.7 forgets what is 300 tokens back: e^-210), by the bound of the bf16 path."""
    B, H, N, D = 3, 12, 1 << 20, 128
    assert B * H * N * D > 2 ** 32
    q, k, v = (torch.empty(B, H, N, D, device="cuda", dtype=BF).normal_() for _ in range(3))
    a = torch.full((H,), -0.7, device="cuda")
    with torch.no_grad():
        o, fin = llsa.llsa_linear_attention(q, k, v, a, return_state=True)
        for b, h, t1 in ((B - 1, H - 1, N), (1, 3, N // 2 + 77)):
            t0 = t1 - 600
            x = [num(t[b:b + 1, h:h + 1, t0:t1]) for t in (q, k, v)]
            an = np.array([-0.7])
            want, S, _ = so.linear_forward(*x, an, D ** -0.5)
            size, SS, _ = so.linear_forward(*(np.abs(t) for t in x), an, D ** -0.5)
            got = num(o[b:b + 1, h:h + 1, t0:t1])[:, :, 300:]
            tol = 1.02 * (2.0 ** -8 * (size + np.abs(want)) + 2.0 ** -16 * size)[:, :, 300:]
            assert (np.abs(got - want[:, :, 300:]) <= tol).all()
            if t1 == N:
                assert (np.abs(num(fin)[b:b + 1, h:h + 1] - S) <= (2.0 ** -16 + 2.0 ** -18) * SS).all()
        del o
        f, _ = llsa.llsa_rotary_frequencies(D, device="cuda")
        y = llsa.llsa_rotary(q, None, None, f)
        part = llsa.llsa_rotary(q[-1:, -1:, -1000:].contiguous(), None, torch.arange(N - 1000, N, device="cuda"), f)
        assert torch.equal(y[-1:, -1:, -1000:], part)
    assert llsa.llsa_device_status() == 0


def test_a_pool_past_32_bits():
    H, D = 64, 128
    P = 2 ** 32 // (H * D * D) + 3
    pool = torch.empty(P, H, D, D, device="cuda")
    pool[-2:].normal_()
    old = pool[-2:].clone()
    q, k, v = (torch.randn(2, H, D, device="cuda") for _ in range(3))
    a = torch.full((H,), -0.1, device="cuda")
    slots = torch.tensor([P - 2, P - 1], device="cuda", dtype=torch.int32)
    o = llsa.llsa_linear_step(q, k, v, a, pool, slots=slots)
    small = old.clone()
    assert torch.equal(llsa.llsa_linear_step(q, k, v, a, small), o) and torch.equal(pool[-2:], small)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("rot,first", [(64, 0), (22, 5)])
def test_rows_that_share_their_values(dtype, rot, first):
    """Expanded inputs and gradients: strides of 0 in some or all of the first three dimensions."""
    f, _ = llsa.llsa_rotary_frequencies(rot, device="cuda")
    one = torch.randn(64, device="cuda").to(dtype)
    for x in (one.expand(2, 3, 40, 64), torch.randn(40, 64, device="cuda").to(dtype).expand(2, 3, 40, 64),
              torch.randn(2, 1, 1, 64, device="cuda").to(dtype).expand(2, 3, 40, 64)):
        want = llsa.llsa_rotary(x.contiguous(), None, None, f, first=first)
        assert torch.equal(llsa.llsa_rotary(x, None, None, f, first=first), want)
        leaf = torch.randn(2, 3, 40, 64, device="cuda").to(dtype).requires_grad_()
        y = llsa.llsa_rotary(leaf, None, None, f, first=first)
        (g,) = torch.autograd.grad(y, leaf, x, retain_graph=True)
        assert torch.equal(g, torch.autograd.grad(y, leaf, x.contiguous())[0])
    a = torch.tensor([-0.1, -0.01, 0.0], device="cuda")
    q = torch.randn(2, 3, 40, 64, device="cuda").to(dtype)
    k = one.expand(2, 3, 40, 64)
    assert torch.equal(llsa.llsa_linear_attention(q, k, k, a), llsa.llsa_linear_attention(q, k.contiguous(), k.contiguous(), a))


def inputs(seed, B, H, N, D, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn(B, H, N, D, device="cuda", generator=g).to(dtype) for _ in range(4)]


@pytest.mark.parametrize("D", [64, 128])
def test_two_streams_at_once(D):
    a = torch.tensor([-0.01, -0.2, 0.0], device="cuda")
    sets = [inputs(s, 2, 3, 3000, D, BF) for s in (1, 2)]

    def step(x):
        leaves = [t.detach().requires_grad_() for t in x[:3]]
        o = llsa.llsa_linear_attention(*leaves, a)
        return [o.detach(), *torch.autograd.grad(o, leaves, x[3])]

    want = [step(x) for x in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(8):
        for i, (s, x) in enumerate(zip(streams, sets)):
            with torch.cuda.stream(s):
                got[i].append(step(x))
    torch.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(r, want[i]))


def test_first_call_of_a_thread():
    x = inputs(3, 1, 3, 700, 64, BF)
    a = torch.tensor([-0.01, -0.2, 0.0], device="cuda")
    with torch.no_grad():
        want = llsa.llsa_linear_attention(*x[:3], a)
    torch.cuda.synchronize()
    shape = llsa.make_linear_shape(1, 3, 700, 64, BF)
    o = torch.empty_like(x[0])
    states = torch.empty(llsa.llsa_linear_states_elems(shape), device="cuda")
    torch.cuda.synchronize()
    errors = []

    def work():
        try:
            llsa.llsa_linear_forward(shape, *x[:3], a, o, states)
        except Exception as e:  # pragma: no cover - reported below
            errors.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors and torch.equal(o, want)


def test_capture_while_an_eager_graph_of_the_same_tensors_lives():
    # (of the same storage: torch ties a leaf's gradient to the stream that it was first used on, so
    # a graph of the same leaf objects that lives on another stream cannot be captured with any op)
    x = inputs(4, 1, 3, 700, 64, BF)
    a = torch.tensor([-0.01, -0.2, 0.0], device="cuda")
    f, _ = llsa.llsa_rotary_frequencies(64, device="cuda")
    leaves = [t.requires_grad_() for t in x[:3]]

    def forward(ls):
        q, k = llsa.llsa_rotary(ls[0], ls[1], None, f)
        return llsa.llsa_linear_attention(q, k, ls[2], a)

    def step():
        o = forward(leaves)
        return o.detach(), torch.autograd.grad(o, leaves, x[3])

    _, want = step()
    others = [t.detach().requires_grad_() for t in leaves]
    alive = forward(others)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, grads = step()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, alive) and all(torch.equal(x, y) for x, y in zip(grads, want))
    late = torch.autograd.grad(alive, others, x[3])
    assert all(torch.equal(x, y) for x, y in zip(late, want))


def test_two_captured_graphs_share_nothing():
    a = torch.tensor([-0.01, -0.2, 0.0], device="cuda")
    sets = [inputs(s, 1, 3, 2000, 64, BF) for s in (5, 6)]
    want = [llsa.llsa_linear_attention(*x[:3], a, return_state=True) for x in sets]
    graphs, outs = [], []
    for x in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(llsa.llsa_linear_attention(*x[:3], a, return_state=True))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(4):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N", [100, 1000])
def test_state_in_place_and_packed_projection(dtype, N):
    B, H, D = 2, 3, 64
    g = torch.Generator(device="cuda").manual_seed(N)
    packed = torch.randn(B, N, 3, H, D, device="cuda", generator=g).to(dtype)
    q, k, v = (packed[:, :, i].transpose(1, 2) for i in range(3))
    a = torch.tensor([-0.01, -0.2, 0.0], device="cuda")
    s0 = torch.randn(B, H, D, D, device="cuda", generator=g)
    o, fin = llsa.llsa_linear_attention(q, k, v, a, initial_state=s0, return_state=True)
    shape = llsa.make_linear_shape(B, H, N, D, dtype)
    n = llsa.llsa_linear_states_elems(shape)
    o2, state = torch.empty(B, H, N, D, device="cuda", dtype=dtype), s0.clone()
    llsa.llsa_linear_forward(shape, q, k, v, a, o2, torch.empty(n, device="cuda") if n else None, None, state, state)
    assert torch.equal(o2, o) and torch.equal(state, fin)
    with pytest.raises(llsa.LLSAError):  # an output on an input
        llsa.llsa_linear_forward(shape, o2, k, v, a, o2, torch.empty(n, device="cuda") if n else None)


def test_rows_behind_a_captured_length_follow_the_length_tensor():
    x = inputs(7, 3, 3, 900, 64, BF)
    a = torch.tensor([-0.01, -0.2, 0.0], device="cuda")
    lengths = torch.tensor([900, 3, 500], device="cuda", dtype=torch.int32)
    llsa.llsa_linear_attention(*x[:3], a, lengths=lengths)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, fin = llsa.llsa_linear_attention(*x[:3], a, lengths=lengths, return_state=True)
    lengths.copy_(torch.tensor([0, 900, 129]))
    graph.replay()
    torch.cuda.synchronize()
    w, wf = llsa.llsa_linear_attention(*x[:3], a, lengths=lengths, return_state=True)
    assert torch.equal(o, w) and torch.equal(fin, wf) and not o[0].any() and not o[2, :, 129:].any()


def test_gradients_that_carry_no_gradient_are_refused():
    x = inputs(8, 1, 3, 10, 64, F32)
    f = llsa.llsa_rotary_frequencies(64, device="cuda")[0].requires_grad_()
    with pytest.raises(ValueError):
        llsa.llsa_rotary(x[0], None, None, f)
