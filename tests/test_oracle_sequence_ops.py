"""Pins of the fp64 reference of rotary positions and decayed linear attention: closed forms,
dense masks with torch autograd, finite differences."""
import numpy as np
import pytest
import torch

from log_linear_hierarchical_b200 import llsa_rotary_frequencies
from oracle import sequence_ops as so


def rng(*shape, seed=0):
    return np.random.default_rng(seed).standard_normal(shape)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotary_is_a_complex_product_and_scores_depend_on_distance(interleaved):
    f = np.array([1.0, 0.3, 0.01])
    x = rng(1, 2, 5, 10)
    pos = np.array([3, 0, -7, 1000, 12])
    y = so.rotary(x, pos, f, interleaved, first=2, scale=1.5)
    sel = slice(2, 8)
    part = x[..., sel]
    z = part[..., 0::2] + 1j * part[..., 1::2] if interleaved else part[..., :3] + 1j * part[..., 3:]
    w = 1.5 * z * np.exp(1j * pos[:, None] * f)
    got = y[..., sel]
    g = got[..., 0::2] + 1j * got[..., 1::2] if interleaved else got[..., :3] + 1j * got[..., 3:]
    assert np.abs(g - w).max() < 1e-12
    assert np.array_equal(y[..., :2], x[..., :2]) and np.array_equal(y[..., 8:], x[..., 8:])
    # the inverse undoes it up to scale^2; inner products see position differences only
    assert np.abs(so.rotary(y, pos, f, interleaved, 2, 1.5, inverse=True)[..., sel] - 2.25 * part).max() < 1e-12
    a, b = rng(1, 1, 1, 6, seed=1), rng(1, 1, 1, 6, seed=2)
    s = [(so.rotary(a, [p], f, interleaved) * so.rotary(b, [p - 4], f, interleaved)).sum() for p in (4, 90)]
    assert abs(s[0] - s[1]) < 1e-12


def test_frequency_tables():
    f, s = llsa_rotary_frequencies(64, base=10000.0)
    assert f.dtype == torch.float64 and s == 1.0
    assert np.allclose(f.numpy(), 10000.0 ** (-np.arange(32) / 32), rtol=1e-14)
    lin, _ = llsa_rotary_frequencies(64, scaling="linear", factor=4.0)
    assert torch.equal(lin, f / 4)
    ntk, _ = llsa_rotary_frequencies(64, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0 and abs(ntk[-1] / f[-1] - 0.25) < 1e-12
    y, sy = llsa_rotary_frequencies(64, scaling="yarn", factor=4.0, original_length=4096)
    turns = 4096 * f / (2 * np.pi)
    assert torch.equal(y[turns > 32], f[turns > 32]) and torch.equal(y[turns < 1], f[turns < 1] / 4)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and ((y < f) & (y > f / 4))[mid].all()
    assert abs(sy - (0.1 * np.log(4.0) + 1)) < 1e-15
    for bad in (dict(rot=3), dict(rot=0), dict(rot=2, scaling="ntk"), dict(rot=8, scaling="yarn"),
                dict(rot=8, scaling="x"), dict(rot=8, scaling="linear", factor=0.5), dict(rot=8, base=-1.0)):
        with pytest.raises(ValueError):
            llsa_rotary_frequencies(**bad)


def dense(q, k, v, log_decay, scale, initial, lengths):
    """torch fp64: the explicit N x N decay mask."""
    B, H, N, D = q.shape
    o, fin = [], []
    for b in range(B):
        L = N if lengths is None else int(lengths[b])
        t = torch.arange(L, dtype=torch.float64)
        ob, fb = [], []
        for h in range(H):
            a = log_decay[h]
            mask = torch.where(t[:, None] >= t, torch.exp(a * (t[:, None] - t).clamp(min=0)), 0.0)
            s0 = initial[b, h]
            oo = (q[b, h, :L] @ k[b, h, :L].T * mask) @ v[b, h, :L] + torch.exp(a * (t + 1))[:, None] * (q[b, h, :L] @ s0)
            ob.append(torch.cat((scale * oo, torch.zeros(N - L, D, dtype=torch.float64))))
            fb.append(torch.exp(a * L) * s0 + (torch.exp(a * (L - 1 - t))[:, None] * k[b, h, :L]).T @ v[b, h, :L])
        o.append(torch.stack(ob))
        fin.append(torch.stack(fb))
    return torch.stack(o), torch.stack(fin)


@pytest.mark.parametrize("lengths", [None, [7, 0], [1, 9]])
def test_linear_matches_the_dense_mask_and_its_autograd(lengths):
    B, H, N, D = 2, 2, 9, 4
    q, k, v, do = (rng(B, H, N, D, seed=i) for i in range(4))
    s0, ds = rng(B, H, D, D, seed=5), rng(B, H, D, D, seed=6)
    a = np.array([-0.3, 0.0])
    t = [torch.tensor(x, requires_grad=True) for x in (q, k, v, s0)]
    o, fin = dense(*t[:3], torch.tensor(a), 0.7, t[3], lengths)
    grads = torch.autograd.grad([o, fin], t, [torch.tensor(do), torch.tensor(ds)])
    oo, S, _ = so.linear_forward(q, k, v, a, 0.7, s0, lengths)
    assert np.abs(oo - o.detach().numpy()).max() < 1e-12 and np.abs(S - fin.detach().numpy()).max() < 1e-12
    for got, want in zip(so.linear_backward(q, k, v, do, a, 0.7, s0, lengths, ds), grads):
        assert np.abs(got - want.numpy()).max() < 1e-12


def test_linear_gradients_match_differences():
    B, H, N, D = 1, 2, 5, 3
    x = [rng(B, H, N, D, seed=i) for i in range(3)] + [rng(B, H, D, D, seed=4)]
    do, ds = rng(B, H, N, D, seed=7), rng(B, H, D, D, seed=8)
    a = np.array([-0.2, -1.5])

    def loss(q, k, v, s0):
        o, S, _ = so.linear_forward(q, k, v, a, 0.5, s0)
        return (o * do).sum() + (S * ds).sum()

    grads = so.linear_backward(*x[:3], do, a, 0.5, x[3], None, ds)
    for i in range(4):
        for at in [(0, 0, 0, 0), (0, 1, 2, 1), (0, 1, 1, 2)]:
            plus, minus = [y.copy() for y in x], [y.copy() for y in x]
            plus[i][at] += 1e-5
            minus[i][at] -= 1e-5
            assert abs((loss(*plus) - loss(*minus)) / 2e-5 - grads[i][at]) < 1e-8


def test_step_is_the_recurrence():
    q, k, v = (rng(1, 2, 6, 4, seed=i) for i in range(3))
    a = np.array([-0.1, -2.0])
    o, S, _ = so.linear_forward(q, k, v, a, 0.5)
    pool = np.zeros((3, 2, 4, 4))
    for t in range(6):
        got, pool = so.linear_step(q[:, :, t], k[:, :, t], v[:, :, t], a, 0.5, pool, [2], [2])
        assert np.abs(got - o[:, :, t]).max() < 1e-12
    assert np.abs(pool[2] - S[0]).max() < 1e-12 and not pool[:2].any()
    got, same = so.linear_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], a, 0.5, pool, [-1], [0])
    assert not got.any() and np.array_equal(same, pool)
