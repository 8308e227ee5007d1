"""llsa_rotary far from position 0, against angles reduced with 60 decimal digits.

Tolerance as near 0: the angle's place in its turn is rounded to fp32 relative to itself (at most
2^-22.3 radians), sincospif is within 2 ulp (2^-23), and each output is two products and a sum: below
(|x_a| + |x_b|) 2^-21.  The reduction itself is within 2^-50 turns at any position."""
import math
from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

import log_linear_hierarchical_b200 as llsa

pytestmark = pytest.mark.gpu

TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def angle(position, frequency):
    getcontext().prec = 60
    t = (Decimal(position) * Decimal(frequency)) % TWO_PI
    return float(t)


FAR = [0, 1, -1, 2 ** 20 + 7, 2 ** 31 - 1, -(2 ** 31), 2 ** 33 + 1, 2 ** 40 + 12345, -(2 ** 45) - 3, 2 ** 50 + 1, 2 ** 52 - 1,
       2 ** 52 + 3, 2 ** 53 - 1, -(2 ** 53) + 1, 6381956970095103, 411557987]


@pytest.mark.parametrize("base,rot,first", [(10000.0, 64, 0), (5e5, 46, 8)])  # one for each kernel
@pytest.mark.parametrize("inverse", [False, True])
def test_any_position_keeps_its_angle(base, rot, first, inverse):
    f, _ = llsa.llsa_rotary_frequencies(rot, base=base, device="cuda")
    n = rot // 2
    x = torch.randn(1, 2, len(FAR), 64, device="cuda")
    pos = torch.tensor(FAR, device="cuda")
    if inverse:
        leaf = torch.zeros_like(x, requires_grad=True)
        (y,) = torch.autograd.grad(llsa.llsa_rotary(leaf, None, pos, f, first=first), leaf, x)
    else:
        y = llsa.llsa_rotary(x, None, pos, f, first=first)
    got, xn = y.double().cpu().numpy(), x.double().cpu().numpy()
    t = np.array([[angle(p, float(w)) for w in f.tolist()] for p in FAR]) * (-1 if inverse else 1)
    cos, sin = np.vectorize(math.cos)(t), np.vectorize(math.sin)(t)
    a, b = xn[..., first:first + n], xn[..., first + n:first + rot]
    tol = 2.0 ** -21 * (np.abs(a) + np.abs(b))
    assert (np.abs(got[..., first:first + n] - (a * cos - b * sin)) <= tol).all()
    assert (np.abs(got[..., first + n:first + rot] - (b * cos + a * sin)) <= tol).all()


def test_int32_positions_at_their_ends():
    f, _ = llsa.llsa_rotary_frequencies(64, device="cuda")
    x = torch.randn(1, 1, 4, 64, device="cuda").bfloat16()
    pos = torch.tensor([2 ** 31 - 1, -(2 ** 31), 2 ** 30 + 1, -5], device="cuda")
    assert torch.equal(llsa.llsa_rotary(x, None, pos.int(), f), llsa.llsa_rotary(x, None, pos, f))
