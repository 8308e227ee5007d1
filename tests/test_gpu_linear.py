"""Linear attention with a decay for each head on the GPU, forward and backward, against the
fp64 token-by-token reference.

Tolerances.  Let A be the reference with |inputs| and the same decay: the sum of the terms'
magnitudes.  fp32 arithmetic (products, exponentials of relative error (|a| n log2 e + 4) 2^-24 on
weights that e^(-|a| n) makes small, sums over a chunk, the channels and the chunks) stays below
2^-18 A.  bf16 inputs round the masked products and the state to bf16 as tensor-core operands,
at most 2^-8 each of its own part of the terms, hence 2^-8 A together; the weighted tokens enter
the state as two bf16 terms (2^-16).  The bf16 result adds 2^-8 of its value; 1.02 covers the
products of these.  States are fp32: (2^-16 + 2^-18) A for bf16 inputs, 2^-18 A for fp32."""
import numpy as np
import pytest
import torch

import log_linear_hierarchical_b200 as llsa
from oracle import sequence_ops as so

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def num(t):
    return None if t is None else t.detach().double().cpu().numpy()


def mag(t):
    return None if t is None else np.abs(num(t))


def close(got, want, size, dtype, what):
    got = num(got)
    if got.dtype != np.float64:
        got = got.astype(np.float64)
    tol = 2.0 ** -18 * size
    if dtype == BF:
        tol = 1.02 * (2.0 ** -8 * (size + np.abs(want)) + 2.0 ** -16 * size)
    bad = np.abs(got - want) - tol
    assert np.isfinite(got).all(), what
    assert (bad <= 1e-30).all(), (what, float(bad.max()), float(np.abs(got - want).max()))


def close_state(got, want, size, dtype, what):
    tol = (2.0 ** -18 + (2.0 ** -16 if dtype == BF else 0)) * size
    assert (np.abs(num(got) - want) <= tol + 1e-30).all(), (what, float((np.abs(num(got) - want) - tol).max()))


def inputs(B, H, N, D, dtype, seed=0, carry=True, strided=False):
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + N + D)

    def tok():
        if strided:
            return torch.randn(B, N, H, D, device="cuda", generator=g).to(dtype).transpose(1, 2)
        return torch.randn(B, H, N, D, device="cuda", generator=g).to(dtype)

    st = [torch.randn(B, H, D, D, device="cuda", generator=g) if carry else None for _ in range(2)]
    return tok(), tok(), tok(), tok(), st[0], st[1]


DECAYS = [-0.02, 0.0, -0.7, -30.0]


def decays(H):
    return torch.tensor([DECAYS[h % len(DECAYS)] for h in range(H)], device="cuda")


def run_and_check(B, H, N, D, dtype, lengths=None, carry=True, strided=False, log_decay=None, scale=None):
    q, k, v, do, s0, ds = inputs(B, H, N, D, dtype, carry=carry, strided=strided)
    a = decays(H) if log_decay is None else log_decay
    L = None if lengths is None else torch.tensor(lengths, device="cuda", dtype=torch.int32)
    ref_scale = D ** -0.5 if scale is None else scale
    if lengths is not None:  # what stands behind the last token takes no part
        for t in (q, k, v, do):
            for b, n in enumerate(lengths):
                t[b, :, n:] = float("nan")
    leaves = [t.requires_grad_() for t in (q, k, v)] + ([s0.requires_grad_()] if carry else [])
    o, fin = llsa.llsa_linear_attention(q, k, v, a, scale=scale, initial_state=s0, lengths=L, return_state=True)
    grads = torch.autograd.grad([o, fin] if carry else [o], leaves, [do, ds] if carry else [do])
    x = [np.nan_to_num(num(t)) for t in (q, k, v, do)]
    an, s0n, dsn = num(a), num(s0), num(ds) if carry else None
    wo, ws, _ = so.linear_forward(*x[:3], an, ref_scale, s0n, lengths)
    ao, as_, _ = so.linear_forward(*(np.abs(t) for t in x[:3]), an, abs(ref_scale), mag(s0), lengths)
    close(o, wo, ao, dtype, "o")
    close_state(fin, ws, as_, dtype, "final")
    want = so.linear_backward(*x, an, ref_scale, s0n, lengths, dsn)
    size = so.linear_backward(*(np.abs(t) for t in x), an, abs(ref_scale), mag(s0), lengths, mag(ds) if carry else None)
    for n, gt, w, m in zip(("dq", "dk", "dv"), grads, want, size):
        close(gt, w, m, dtype, n)
    if carry:
        close_state(grads[3], want[3], size[3], dtype, "d_initial")
    if lengths is not None:
        for b, n in enumerate(lengths):
            for t in (o, *grads[:3]):
                assert not t[b, :, n:].any()
    assert llsa.llsa_device_status() == 0


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H,N", [(1, 1, 1), (2, 3, 2), (1, 4, 31), (1, 2, 64), (1, 4, 127), (2, 2, 128), (1, 4, 129),
                                   (1, 2, 300)])
def test_matches_the_recurrence(dtype, D, B, H, N):
    run_and_check(B, H, N, D, dtype)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D,N", [(64, 1500), (128, 1025)])
def test_long_sequences_in_segments_without_states(dtype, D, N):
    assert llsa.llsa_linear_states_elems(llsa.make_linear_shape(1, 4, N, D, dtype)) > 0
    run_and_check(1, 4, N, D, dtype, carry=False)
    run_and_check(1, 1, N, D, dtype, carry=True, log_decay=torch.tensor([-0.001], device="cuda"))


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("D", [64, 128])
def test_ragged_batch(dtype, D):
    run_and_check(5, 2, 290, D, dtype, lengths=[290, 0, 1, 128, 173])
    run_and_check(3, 1, 130, D, dtype, lengths=[0, 0, 129], carry=False)


def test_many_heads_in_one_segment():
    assert llsa.llsa_linear_states_elems(llsa.make_linear_shape(40, 4, 260, 64, BF)) == 0
    run_and_check(40, 4, 260, 64, BF, lengths=[260 - 5 * i for i in range(40)])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_strides_and_copies(dtype):
    run_and_check(2, 3, 150, 64, dtype, strided=True)
    run_and_check(2, 2, 140, 128, dtype, strided=True, scale=-1.5)
    q, k, v, _, s0, _ = inputs(2, 4, 140, 64, dtype)
    base = llsa.llsa_linear_attention(q, k, v, decays(4), initial_state=s0)
    odd = torch.empty(q.numel() + 1, device="cuda", dtype=dtype)[1:].view_as(q).copy_(q)
    columns = k.transpose(2, 3).contiguous().transpose(2, 3)
    turned = s0.transpose(2, 3).contiguous().transpose(2, 3)
    assert torch.equal(llsa.llsa_linear_attention(odd, columns, v, decays(4), initial_state=turned), base)


def test_shared_key_heads_get_the_sum_of_their_gradients():
    q, _, _, do, _, _ = inputs(1, 4, 150, 64, F32)
    k, v = (torch.randn(1, 1, 150, 64, device="cuda", requires_grad=True) for _ in range(2))
    o = llsa.llsa_linear_attention(q, k.expand(1, 4, 150, 64), v.expand(1, 4, 150, 64), decays(4))
    dk, dv = torch.autograd.grad(o, [k, v], do)
    kk, vv = (num(t).repeat(4, axis=1) for t in (k, v))
    _, wk, wv, _ = so.linear_backward(num(q), kk, vv, num(do), num(decays(4)), 0.125)
    _, sk, sv, _ = so.linear_backward(mag(q), np.abs(kk), np.abs(vv), mag(do), num(decays(4)), 0.125)
    for got, w, s in ((dk, wk, sk), (dv, wv, sv)):
        assert (np.abs(num(got) - w.sum(1, keepdims=True)) <= 2.0 ** -17 * s.sum(1, keepdims=True)).all()


@pytest.mark.parametrize("dtype", [F32, BF])
def test_no_memory_and_no_decay(dtype):
    q, k, v, _, s0, _ = inputs(1, 2, 200, 64, dtype)
    a = torch.tensor([float("-inf"), -1e9], device="cuda")
    o, fin = llsa.llsa_linear_attention(q, k, v, a, initial_state=s0, return_state=True)
    x = [num(t) for t in (q, k, v)]
    own = 0.125 * (x[0] * x[1]).sum(-1, keepdims=True) * x[2]
    size = 0.125 * np.abs(x[0] * x[1]).sum(-1, keepdims=True) * np.abs(x[2])
    close(o, own, size, dtype, "o")
    close_state(fin, x[1][:, :, -1, :, None] * x[2][:, :, -1, None, :],
                np.abs(x[1][:, :, -1, :, None] * x[2][:, :, -1, None, :]), dtype, "final")


def test_a_bad_length_is_recorded():
    q, k, v, _, _, _ = inputs(2, 1, 40, 64, F32)
    a = decays(1)
    o = llsa.llsa_linear_attention(q, k, v, a, lengths=torch.tensor([41, -3], device="cuda", dtype=torch.int32))
    assert llsa.llsa_device_status() == 5
    want = llsa.llsa_linear_attention(q, k, v, a, lengths=torch.tensor([40, 0], device="cuda", dtype=torch.int32))
    assert torch.equal(o, want) and llsa.llsa_device_status() == 0


def test_gradient_by_differences():
    q, k, v, do, s0, ds = inputs(1, 2, 140, 64, F32)
    a = decays(2)
    leaves = [t.requires_grad_() for t in (q, k, v, s0)]
    o, fin = llsa.llsa_linear_attention(q, k, v, a, initial_state=s0, return_state=True)
    grads = torch.autograd.grad([o, fin], leaves, [do, ds])
    for i, (leaf, g) in enumerate(zip(leaves, grads)):  # the map is linear in each input alone
        e = torch.randn_like(leaf)
        with torch.no_grad():
            args = [t.detach() for t in leaves]
            args[i] = args[i] + e
            o1, f1 = llsa.llsa_linear_attention(*args[:3], a, initial_state=args[3], return_state=True)
        moved = ((o1.double() - o.detach().double()) * do.double()).sum() + \
                ((f1.double() - fin.detach().double()) * ds.double()).sum()
        # both sums have the terms' magnitudes times a few 2^-18
        size = ((o1.abs() + o.detach().abs()).double() * do.abs().double()).sum() + \
               ((f1.abs() + fin.detach().abs()).double() * ds.abs().double()).sum()
        assert abs(moved - (e.double() * g.double()).sum()) < 2.0 ** -17 * size


def test_gradients_of_one_output_alone():
    q, k, v, do, s0, ds = inputs(1, 2, 150, 64, F32)
    leaves = [t.requires_grad_() for t in (q, k, v, s0)]
    o, fin = llsa.llsa_linear_attention(q, k, v, decays(2), initial_state=s0, return_state=True)
    both = torch.autograd.grad([o, fin], leaves, [do, ds], retain_graph=True)
    one = torch.autograd.grad(o, leaves, do, retain_graph=True)
    two = torch.autograd.grad(fin, leaves[1:], ds)
    for i in range(1, 4):  # each is a sum of the same fp32 terms, rounded a few times each
        assert torch.allclose(both[i], one[i] + two[i - 1], rtol=1e-5, atol=1e-4)
    assert torch.equal(both[0], one[0])


def test_results_repeat_and_a_captured_step_replays():
    q, k, v, do, s0, ds = inputs(1, 4, 1000, 64, BF)
    leaves = [t.requires_grad_() for t in (q, k, v, s0)]
    a = decays(4)

    def step():
        o, fin = llsa.llsa_linear_attention(q, k, v, a, initial_state=s0, return_state=True)
        return [o.detach(), fin.detach(), *torch.autograd.grad([o, fin], leaves, [do, ds])]

    first = [t.clone() for t in step()]
    assert all(torch.equal(x, y) for x, y in zip(first, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    with torch.no_grad():
        for t in (q, k, v, do):
            t.copy_(torch.randn_like(t))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(held, step()))


def test_refusals():
    q = torch.zeros(1, 2, 8, 64, device="cuda")
    a = torch.zeros(2, device="cuda")
    for call in (lambda: llsa.llsa_linear_attention(q, q, q[:, :, :4], a), lambda: llsa.llsa_linear_attention(q, q, q.bfloat16(), a),
                 lambda: llsa.llsa_linear_attention(q, q, q, a.double()), lambda: llsa.llsa_linear_attention(q, q, q, a[:1]),
                 lambda: llsa.llsa_linear_attention(q, q, q, a.cpu()),
                 lambda: llsa.llsa_linear_attention(q, q, q, a, lengths=torch.zeros(1, device="cuda")),
                 lambda: llsa.llsa_linear_attention(q, q, q, a, lengths=torch.zeros(2, device="cuda", dtype=torch.int32))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(llsa.LLSAError):
        llsa.llsa_linear_attention(q[:, :, :0], q[:, :, :0], q[:, :, :0], a)
