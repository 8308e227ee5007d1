"""llsa_rotary on the GPU against the fp64 reference: layouts, parts of the head, far positions,
strides, alignment, gradients, in place.

Tolerance per element: the angle's place in its turn is exact to about 1e-9 and rounded to fp32
relative to itself (at most 2^-25 turns = 2^-22.3 radians), sincospif is within 2 ulp of values of
at most 1 (2^-23), and y = x_a c - x_b s adds three fp32 roundings, so the fp32 value is within
scale (|x_a| + |x_b|) (2^-22.3 + 2^-23 + 2 * 2^-24) < scale (|x_a| + |x_b|) 2^-21; storing it as
bf16 adds at most 2^-8 of it.  Copied channels are equal."""
import numpy as np
import pytest
import torch

import log_linear_hierarchical_b200 as llsa
from oracle import sequence_ops as so

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def check(y, x, pos, f, interleaved, first, scale, inverse=False):
    xn = x.detach().double().cpu().numpy()
    want = so.rotary(xn, pos, f, interleaved, first, scale, inverse)
    got = y.detach().double().cpu().numpy()
    n = len(f)
    size = np.zeros_like(xn)
    for c in range(n):
        a, b = (first + 2 * c, first + 2 * c + 1) if interleaved else (first + c, first + n + c)
        size[..., a] = size[..., b] = np.abs(xn[..., a]) + np.abs(xn[..., b])
    tol = scale * size * 2.0 ** -21 * (1 + 2.0 ** -8) + (2.0 ** -8 * np.abs(want) if y.dtype == BF else 0)
    turned = size > 0
    assert (np.abs(got - want) <= tol)[turned].all(), np.abs(got - want)[turned].max()
    rest = np.ones(xn.shape[-1], bool)
    rest[first:first + 2 * n] = False
    assert np.array_equal(got[..., rest], xn[..., rest])


def freqs(rot, base=10000.0):
    return llsa.llsa_rotary_frequencies(rot, base=base, device="cuda")[0]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("B,H,N,D,rot,first", [
    (1, 1, 1, 64, 64, 0), (2, 3, 37, 64, 32, 16), (1, 2, 130, 128, 128, 0), (3, 5, 7, 128, 64, 64),
    (2, 2, 33, 64, 2, 61), (1, 3, 9, 64, 46, 8), (1, 2, 5, 128, 16, 4), (2, 1, 300, 128, 96, 24), (70, 2, 1, 64, 64, 0)])
def test_matches_the_reference(dtype, interleaved, B, H, N, D, rot, first):
    g = torch.Generator(device="cuda").manual_seed(N + D + rot)
    q = torch.randn(B, H, N, D, device="cuda", generator=g).to(dtype)
    k = torch.randn(B, H + 1, N, D, device="cuda", generator=g).to(dtype)
    f = freqs(rot)
    pos = torch.randint(-50, 1 << 20, (B, N), device="cuda", generator=g)
    y, z = llsa.llsa_rotary(q, k, pos, f, interleaved=interleaved, first=first, scale=1.25)
    assert y.is_contiguous() and z.shape == k.shape
    check(y, q, pos.cpu().numpy(), f.cpu().numpy(), interleaved, first, 1.25)
    check(z, k, pos.cpu().numpy(), f.cpu().numpy(), interleaved, first, 1.25)


def test_positions_forms_agree():
    x = torch.randn(3, 2, 20, 64, device="cuda")
    f = freqs(64)
    p = torch.arange(20, device="cuda")
    y = llsa.llsa_rotary(x, None, None, f)
    for pos in (p, p.int(), p.expand(3, 20), p.repeat(3, 1).int(), torch.arange(40, device="cuda")[::2] // 2):
        assert torch.equal(llsa.llsa_rotary(x, None, pos, f), y)
    check(y, x, np.arange(20), f.cpu().numpy(), False, 0, 1.0)


def test_very_far_positions_keep_their_angle():
    x = torch.randn(1, 1, 4, 64, device="cuda")
    f = freqs(64, base=5e5)
    pos = torch.tensor([2 ** 31 + 12345, 2 ** 33 + 1, 3, -(2 ** 32) - 7], device="cuda")
    # the fp64 product is within 2^-53 of 2^33 radians: 1e-6, which the reference shares
    y = llsa.llsa_rotary(x, None, pos, f).double().cpu().numpy()
    want = so.rotary(x.double().cpu().numpy(), pos.cpu().numpy(), f.cpu().numpy())
    assert np.abs(y - want).max() < 2e-5


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strided_misaligned_and_in_place(dtype):
    f = freqs(64)
    fn = f.cpu().numpy()
    pos = np.arange(11)
    packed = torch.randn(2, 11, 3, 4, 64, device="cuda").to(dtype)      # [B, N, q|k|v, H, D]
    q, k = packed[:, :, 0].transpose(1, 2), packed[:, :, 1].transpose(1, 2)
    y, z = llsa.llsa_rotary(q, k, None, f)
    check(y, q, pos, fn, False, 0, 1.0)
    check(z, k, pos, fn, False, 0, 1.0)
    shared = torch.randn(2, 1, 11, 64, device="cuda").to(dtype).expand(2, 3, 11, 64)   # one head for three
    check(llsa.llsa_rotary(shared, None, None, f), shared, pos, fn, False, 0, 1.0)
    flat = torch.randn(2 * 3 * 11 * 64 + 1, device="cuda").to(dtype)
    odd = flat[1:].view(2, 3, 11, 64)                                    # not 16-byte aligned
    check(llsa.llsa_rotary(odd, None, None, f), odd, pos, fn, False, 0, 1.0)
    column = torch.randn(2, 3, 64, 11, device="cuda").to(dtype).transpose(2, 3)      # channels strided
    check(llsa.llsa_rotary(column, None, None, f), column, pos, fn, False, 0, 1.0)
    a, b = torch.randn(2, 3, 11, 64, device="cuda").to(dtype), torch.randn(2, 1, 11, 64, device="cuda").to(dtype)
    ya, yb = llsa.llsa_rotary(a, b, None, f[:20].contiguous(), first=3)
    ra, rb = llsa.llsa_rotary(a, b, None, f[:20].contiguous(), first=3, inplace=True)
    assert ra is a and rb is b and torch.equal(a, ya) and torch.equal(b, yb)
    with pytest.raises(ValueError):
        llsa.llsa_rotary(q, None, None, f, inplace=True)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("interleaved,rot,first", [(False, 64, 0), (True, 32, 32), (False, 22, 5)])
def test_gradient_is_the_inverse_rotation(dtype, interleaved, rot, first):
    f = freqs(rot)
    pos = torch.randint(0, 1000, (2, 13), device="cuda")
    q = torch.randn(2, 13, 3, 64, device="cuda").to(dtype).transpose(1, 2).requires_grad_()
    k = torch.randn(2, 1, 13, 64, device="cuda").to(dtype).requires_grad_()
    y, z = llsa.llsa_rotary(q, k, pos, f, interleaved=interleaved, first=first, scale=0.75)
    dy, dz = torch.randn_like(y), torch.randn_like(z)
    dq, dk = torch.autograd.grad([y, z], [q, k], [dy, dz])
    check(dq, dy, pos.cpu().numpy(), f.cpu().numpy(), interleaved, first, 0.75, inverse=True)
    check(dk, dz, pos.cpu().numpy(), f.cpu().numpy(), interleaved, first, 0.75, inverse=True)
    (only,) = torch.autograd.grad(llsa.llsa_rotary(q, k.detach(), pos, f, interleaved=interleaved, first=first)[0].sum(), q)
    assert only.shape == q.shape
    # against differences: the map is linear, so <R x, dy> moves by <e, R^T dy> exactly
    if dtype == F32:
        e = torch.randn_like(q)
        lhs = ((llsa.llsa_rotary((q + e).detach(), None, pos, f, interleaved=interleaved, first=first, scale=0.75).double()
                - y.detach().double()) * dy.double()).sum()
        rhs = (e.double() * dq.double()).sum()
        # each of the 2 * 3 * 13 * 64 terms carries a few 2^-22 of values of size ~ 4
        assert abs(lhs - rhs) < 2 * 3 * 13 * 64 * 16 * 2.0 ** -22


def test_refusals():
    x = torch.zeros(1, 2, 8, 64, device="cuda")
    f = freqs(64)
    for call in (lambda: llsa.llsa_rotary(x, x[:, :, :4], None, f), lambda: llsa.llsa_rotary(x, None, None, f.float()),
                 lambda: llsa.llsa_rotary(x, None, torch.zeros(7, device="cuda", dtype=torch.int64), f),
                 lambda: llsa.llsa_rotary(x, None, torch.zeros(8, device="cuda"), f),
                 lambda: llsa.llsa_rotary(x, None, torch.zeros(8, dtype=torch.int64), f),
                 lambda: llsa.llsa_rotary(x.requires_grad_(), None, None, f, inplace=True)):
        with pytest.raises(ValueError):
            call()
    x = x.detach()
    for call in (lambda: llsa.llsa_rotary(x, None, None, f, first=2), lambda: llsa.llsa_rotary(x[:, :, :0], None, None, f),
                 lambda: llsa.llsa_rotary(x[..., :32].contiguous(), None, None, f[:8].contiguous())):
        with pytest.raises(llsa.LLSAError):
            call()
