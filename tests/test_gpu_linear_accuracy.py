"""How accurate linear attention is, beyond the bounds by the terms' magnitudes: fp32 inputs whose
products are exact, and root-mean-square errors over random inputs."""
import numpy as np
import pytest
import torch

import log_linear_hierarchical_b200 as llsa
from oracle import sequence_ops as so

pytestmark = pytest.mark.gpu
F32 = torch.float32


def num(t):
    return t.detach().double().cpu().numpy()


def run(q, k, v, do, a, scale, s0, ds):
    """Outputs and gradients of one call, and the same in 64 bits."""
    leaves = [t.requires_grad_() for t in (q, k, v, s0)]
    o, fin = llsa.llsa_linear_attention(q, k, v, a, scale=scale, initial_state=s0, return_state=True)
    got = [o, fin, *torch.autograd.grad([o, fin], leaves, [do, ds])]
    x = [num(t) for t in (q, k, v, do)]
    wo, ws, _ = so.linear_forward(*x[:3], num(a), scale, num(s0))
    return got, [wo, ws, *so.linear_backward(*x, num(a), scale, num(s0), None, num(ds))]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("N", [1, 2])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_fp32_factors_are_split_by_rounding(D, N, sign):
    """Every value is c = 2 - 2^-23, all of whose low bits are set.  Rounded to 11 bits it is 2, the
    rest -2^-23 is one bit, and of the product c c = 4 - 2^-21 + 2^-46 only the last term is left out: 64 of
    them make 256 - 2^-15, 0.125 of that times c again is 64 - 3 2^-18 (+ 2^-41), and their sums with the same of
    the state and of a second token are short too, all within 24 bits; so a result is off by its own and a
    sum's last rounding, 2^-24 each of values of one sign, and twice that bounds it.  (Cut off to 11 bits, c is 2 - 2^-10
    and the rest loses bits and enters its own square, 2^-21.)"""
    c = torch.tensor(0x3fffffff, dtype=torch.int32).view(F32).item()
    assert c == 2.0 - 2.0 ** -23
    full = lambda *s, by=1.0: torch.full(s, c * by, device="cuda")  # noqa: E731
    q, k, v, do = full(1, 2, N, D, by=sign), full(1, 2, N, D), full(1, 2, N, D, by=sign), full(1, 2, N, D)
    s0, ds = full(1, 2, D, D, by=sign), full(1, 2, D, D, by=sign)
    got, want = run(q, k, v, do, torch.zeros(2, device="cuda"), 0.125, s0, ds)
    for name, g, w in zip(("o", "final", "dq", "dk", "dv", "d_initial"), got, want):
        assert (np.abs(num(g) - w) <= 2.0 ** -22 * np.abs(w)).all(), (name, np.abs(num(g) / w - 1).max())


@pytest.mark.parametrize("D,N", [(64, 1000), (128, 700)])
def test_fp32_root_mean_square_error(D, N):
    """Rounding to 11 bits leaves lo uniform in +-L, L = 2^-11 of x's power of two; of lo TF32 keeps 11
    bits, so what is lost of a factor has a mean square of (2^-10 2^floor(log2 |lo|))^2 / 3, on average (2^-10 L)^2 / 21:
    2^-21 / 4.6 of x's power of two, about 7.5e-8 of x; lo lo, which is left out, has L^2 / 3, 4e-8 of the product.
    A product of two factors is off by 1.1e-7 with either sign, two in a row (the masked products, then
    their product with the tokens) by 1.6e-7, and the additions of groups of 8 on the tensor cores and in fp32 add about
    as much: 2.3e-7.  Twice that, 2^-21, bounds every output."""
    g = torch.Generator(device="cuda").manual_seed(D)
    q, k, v, do = (torch.randn(1, 2, N, D, device="cuda", generator=g) for _ in range(4))
    s0, ds = (torch.randn(1, 2, D, D, device="cuda", generator=g) for _ in range(2))
    got, want = run(q, k, v, do, torch.tensor([-0.02, -0.002], device="cuda"), D ** -0.5, s0, ds)
    for name, x, w in zip(("o", "final", "dq", "dk", "dv", "d_initial"), got, want):
        assert np.linalg.norm(num(x) - w) <= 2.0 ** -21 * np.linalg.norm(w), name


@pytest.mark.parametrize("D,N", [(64, 1500), (128, 700)])
def test_bf16_root_mean_square_error(D, N):
    """A rounding to bf16 is off by a value uniform in half a step, at most 2^-8 of what is rounded: 2^-8 / sqrt(3)
    of it in the mean square.  Over random inputs a result is a sum of terms of either sign, whose rounded factor
    (the masked product, or the state's copy) makes the sum off by that share of its own mean square; the result's
    own rounding comes on top: sqrt(2 / 3) 2^-8 together, for each head alone.  States get tokens in two bf16 terms,
    2^-16 / sqrt(3)."""
    g = torch.Generator(device="cuda").manual_seed(D)
    q, k, v, do = (torch.randn(1, 3, N, D, device="cuda", generator=g).bfloat16() for _ in range(4))
    s0, ds = (torch.randn(1, 3, D, D, device="cuda", generator=g) for _ in range(2))
    got, want = run(q, k, v, do, torch.tensor([0.0, -0.02, -0.7], device="cuda"), D ** -0.5, s0, ds)
    for name, x, w in zip(("o", "final", "dq", "dk", "dv", "d_initial"), got, want):
        bound = 2.0 ** -16 / 3 ** 0.5 if x.dtype == F32 else (2 / 3) ** 0.5 * 2.0 ** -8
        for h in range(3):
            assert np.linalg.norm(num(x)[:, h] - w[:, h]) <= bound * np.linalg.norm(w[:, h]), (name, h)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("B,H,N,cut", [(1, 2, 1, False), (1, 3, 100, False), (1, 2, 1500, True), (100, 2, 290, False),
                                       (3, 2, 1900, True)])
def test_returned_states_of_bf16_inputs_are_fp32(D, B, H, N, cut):
    """The states and their gradients, which are fp32, over ragged rows with NaN behind the last token.  A token
    enters in three bf16 terms (2^-25 of it) times a weight that is off by a few 2^-24 with either sign, 2^-22 at
    most; eight products of 16 tokens make a chunk's sum, each cut off below 2^-23 of what the sum is by then,
    half of that on average and half of the sum over the eight: 2^-22; chunks are added in fp32.  2^-21 together, and
    a chunk's rounding, 2^-24, that the decay forgets.  (Two terms are 2^-17 off a token, 2.4e-6.)"""
    shape = llsa.make_linear_shape(B, H, N, D, torch.bfloat16)
    assert (llsa.llsa_linear_states_elems(shape) > 0) == cut
    g = torch.Generator(device="cuda").manual_seed(N + D)
    q, k, v, do = (torch.randn(B, H, N, D, device="cuda", generator=g).bfloat16() for _ in range(4))
    s0, ds = (torch.randn(B, H, D, D, device="cuda", generator=g) for _ in range(2))
    lengths = [N - (7 * b) % N for b in range(B)]
    for t in (q, k, v, do):
        for b, n in enumerate(lengths):
            t[b, :, n:] = float("nan")
    a = torch.tensor([-0.02, -0.7, -0.003][:H], device="cuda")
    leaves = [t.requires_grad_() for t in (q, k, v, s0)]
    o, fin = llsa.llsa_linear_attention(q, k, v, a, initial_state=s0, return_state=True,
                                        lengths=torch.tensor(lengths, device="cuda", dtype=torch.int32))
    d0 = torch.autograd.grad([o, fin], leaves, [do, ds])[3]
    rows = sorted({0, 1 % B, B - 1})  # (each row's 64-bit reference takes a while)
    x = [np.nan_to_num(num(t[rows])) for t in (q, k, v, do)]
    sub = [lengths[b] for b in rows]
    _, want, _ = so.linear_forward(*x[:3], num(a), D ** -0.5, num(s0[rows]), sub)
    dwant = so.linear_backward(*x, num(a), D ** -0.5, num(s0[rows]), sub, num(ds[rows]))[3]
    for name, got, w in (("final", fin, want), ("d_initial", d0, dwant)):
        for i in range(len(rows)):
            for h in range(H):
                off = np.linalg.norm(num(got[rows[i], h]) - w[i, h])
                assert off <= 2.0 ** -21 * np.linalg.norm(w[i, h]), (name, i, h, off / np.linalg.norm(w[i, h]))
    assert llsa.llsa_device_status() == 0
