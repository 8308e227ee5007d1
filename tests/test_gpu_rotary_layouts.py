"""llsa_rotary on tensors that start at any element, against the aligned call.

Where both go through the same kernel the bits are equal.  With `first` a multiple of 8 and `rot`
of 16 the aligned call takes the kernel of 16-byte accesses, in which the compiler may fuse the
other product of x_a c - x_b s.  Either form rounds one product and the sum, so it is within
2^-24 max(|x_a c|, |x_b s|) + 2^-24 |y| <= 2^-23 (|x_a| + |x_b|) of the exact sum, and the two are
within 2^-22 (|x_a| + |x_b|) of each other; as bf16 each is then rounded by half a step, 2^-8 of it,
so they may differ by 2^-7 |y| more (1.01 for the parts of these roundings that multiply)."""
import pytest
import torch

import log_linear_hierarchical_b200 as llsa

pytestmark = pytest.mark.gpu


def same(got, want, x, rot, first, dtype):
    if first % 8 or rot % 16:
        return torch.equal(got, want)
    pairs = x.float().abs()[..., first:first + rot].unflatten(-1, (2, rot // 2)).sum(-2).repeat(1, 1, 1, 2)
    tol = torch.zeros_like(x, dtype=torch.float32)
    tol[..., first:first + rot] = 1.01 * 2.0 ** -22 * pairs
    if dtype == torch.bfloat16:
        tol[..., first:first + rot] += 1.01 * 2.0 ** -7 * want.float().abs()[..., first:first + rot]
    return ((got.double() - want.double()).abs() <= tol.double()).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,rot,first", [(64, 46, 8), (64, 64, 0), (128, 30, 97), (128, 128, 0)])
def test_any_element_alignment(dtype, D, rot, first):
    B, H, N = 3, 2, 41  # 123 rows: the last group of 32 is not full
    x = torch.randn(B, H, N, D, device="cuda").to(dtype)
    k = torch.randn(B, H + 1, N, D, device="cuda").to(dtype)
    f, _ = llsa.llsa_rotary_frequencies(rot, device="cuda")
    want = llsa.llsa_rotary(x, k, None, f, first=first)
    for shift in range(1, 16 // x.element_size()):
        def moved(t):
            flat = torch.full((t.numel() + 16,), float("nan"), device="cuda", dtype=dtype)
            return flat, flat[shift:shift + t.numel()].view(t.shape).copy_(t)

        (fx, mx), (fk, mk) = moved(x), moved(k)
        got = llsa.llsa_rotary(mx, mk, None, f, first=first)
        for t, g, w in zip((x, k), got, want):
            assert same(g, w, t, rot, first, dtype)
        llsa.llsa_rotary(mx, mk, None, f, first=first, inplace=True)
        assert torch.equal(mx, got[0]) and torch.equal(mk, got[1])
        for flat in (fx, fk):  # nothing beside the tensor is written
            assert flat[:shift].isnan().all() and flat[shift - 16:].isnan().all()
    assert llsa.llsa_device_status() == 0
