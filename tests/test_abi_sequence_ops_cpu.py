"""Refusals of the rotary and linear-attention calls, none of which reaches a launch: the C
checks by raw addresses, the binding's on host tensors."""
import ctypes

import pytest
import torch

import log_linear_hierarchical_b200 as llsa
from log_linear_hierarchical_b200 import _lib
from log_linear_hierarchical_b200._lib import LLSALinearShape, LLSARotaryShape


@pytest.fixture(scope="module")
def lib():
    from log_linear_hierarchical_b200 import build
    build.build()
    return _lib.load()


def rotary(lib, x=4096, xs=None, x2=None, xs2=None, pos=64, ps=0, f=128, y=1 << 30, y2=None, **kw):
    s = dict(B=2, H=3, H2=0, N=8, D=64, dtype=0, rot=64, first=0, flags=0, scale=1.0)
    s.update(kw)
    st = (ctypes.c_int64 * 3)(*xs) if xs else None
    st2 = (ctypes.c_int64 * 3)(*xs2) if xs2 else None
    return lib.llsa_rotary(ctypes.byref(LLSARotaryShape(**s)), x, st, x2, st2, pos, ps, f, y, y2, None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(y=None), 1), (dict(f=None), 1), (dict(f=132), 1), (dict(pos=68), 1),
    (dict(x=4097), 1), (dict(dtype=1, x=4098), 1), (dict(dtype=5), 1), (dict(flags=8), 1),
    (dict(rot=0), 1), (dict(rot=7), 1), (dict(rot=66), 1), (dict(first=-2), 1), (dict(rot=32, first=34), 1),
    (dict(ps=-1), 1), (dict(xs=(-64, 64, 64)), 1), (dict(B=0), 1), (dict(N=0), 1), (dict(H2=3), 1),
    (dict(x2=8192, y2=None, H2=3), 1), (dict(x2=8192, y2=2 << 30), 1),
    (dict(D=96), 2), (dict(B=1 << 16, N=1 << 14), 2),
    (dict(y=4096 + 64), 1),                                     # overlaps x without being x
    (dict(y=4096, xs=(3 * 8 * 64, 64, 3 * 64)), 1),             # in place needs contiguous
    (dict(x2=1 << 20, H2=3, y2=1 << 30), 1),                    # the outputs overlap
    (dict(x2=1 << 20, H2=3, y=1 << 20, y2=1 << 31), 1),         # an output on the other input
])
def test_rotary_refusals(lib, kw, status):
    assert rotary(lib, **kw) == status


def linear(**kw):
    s = dict(B=2, H=3, N=70, D=64, dtype=0, scale=0.125)
    strides = {n: kw.pop(n) for n in ("q_strides", "k_strides", "v_strides", "dO_strides") if n in kw}
    s.update(kw)
    shape = LLSALinearShape(**s)
    for n, v in strides.items():
        getattr(shape, n)[:] = v
    return shape


@pytest.mark.parametrize("kw,status", [
    ({}, 0), (dict(N=1), 0), (dict(D=128, dtype=1), 0), (dict(q_strides=(70 * 3 * 64, 64, 192)), 0),
    (dict(B=1, q_strides=(0, 64, 192)), 0),                     # a dimension of size 1 is not looked at
    (dict(B=0), 1), (dict(N=0), 1), (dict(N=-1), 1), (dict(dtype=2), 1), (dict(D=32), 2), (dict(D=80), 2),
    (dict(q_strides=(70 * 3 * 64, 0, 64)), 1),                  # an expanded dimension
    (dict(k_strides=(70 * 3 * 64, 64, -192)), 1), (dict(v_strides=(70 * 3 * 68, 68, 204)), 1),
    (dict(B=1 << 15, H=1 << 10, N=64), 2), (dict(H=65536), 2),
])
def test_linear_shapes(lib, kw, status):
    s = linear(**kw)
    assert lib.llsa_linear_validate(ctypes.byref(s)) == status
    if status:
        assert lib.llsa_linear_states_elems(ctypes.byref(s)) == 0
        assert lib.llsa_linear_forward(ctypes.byref(s), 16, 16, 16, 16, None, None, 16, None, None, None) == status
        assert lib.llsa_linear_step(ctypes.byref(s), 16, 16, 16, 16, 16, 4, None, None, 16, None) == status


def test_linear_scratch_sizes(lib):
    for B, H, N, D in [(1, 6, 65536, 64), (1, 1, 1, 64), (4, 6, 4096, 128), (64, 24, 4096, 64), (1, 1, 1 << 24, 128)]:
        s = linear(B=B, H=H, N=N, D=D)
        n = lib.llsa_linear_states_elems(ctypes.byref(s))
        assert n % (B * H * D * D) == 0 and lib.llsa_linear_workspace_bytes(ctypes.byref(s)) == 4 * n
        assert n // (B * H * D * D) <= 296 and (n == 0 or N > 128)


def test_linear_refusals(lib):
    s = ctypes.byref(linear(N=4096))
    assert lib.llsa_linear_states_elems(s) > 0
    fwd = lambda *a: lib.llsa_linear_forward(s, *a, None)  # noqa: E731
    good = [16, 16, 16, 16, None, None, 16, None, None]
    assert fwd(*good) == 3                                      # states missing
    for i, bad in [(0, None), (1, 24), (3, None), (3, 18), (4, 18), (5, 24), (6, None), (6, 8), (7, 4), (8, 20)]:
        args = good[:8] + [16]
        args[i] = bad
        assert fwd(*args) == 1, (i, bad)
    ws = lib.llsa_linear_workspace_bytes(s)
    back = [16, 16, 16, 16, 16, None, None, None, 16, 16, 16, 16, None, 16, ws]
    call = lambda a: lib.llsa_linear_backward(s, *a, None)  # noqa: E731
    for i, bad, st in [(3, None, 1), (4, None, 1), (8, None, 3), (9, None, 1), (10, 4, 1), (13, None, 3), (14, ws - 1, 3),
                       (7, 8, 1), (12, 8, 1)]:
        args = list(back)
        args[i] = bad
        assert call(args) == st, (i, bad)
    one = ctypes.byref(linear(N=1))
    step = lambda *a, s=one: lib.llsa_linear_step(s, *a, None)  # noqa: E731
    good = [16, 16, 16, 16, 16, 4, None, None, 16]
    for i, bad in [(0, None), (2, 24), (3, None), (4, None), (4, 20), (5, 0), (5, 1), (6, 2), (7, 2), (8, None)]:
        args = list(good)
        args[i] = bad
        assert step(*args) == 1, (i, bad)
    assert step(*good, s=ctypes.byref(linear(N=2))) == 1
    assert step(*good, s=ctypes.byref(linear(N=1, q_strides=(192, 64, 64)))) == 1
    assert lib.llsa_linear_validate(None) == 1


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(1, 2, 8, 64)
    f = torch.ones(32, dtype=torch.float64)
    a = torch.zeros(2)
    for call in (lambda: llsa.llsa_rotary(x, None, None, f),
                 lambda: llsa.llsa_rotary(x.double(), None, None, f),
                 lambda: llsa.llsa_linear_attention(x, x, x, a),
                 lambda: llsa.llsa_linear_attention(x.half(), x.half(), x.half(), a),
                 lambda: llsa.llsa_linear_attention(x, x, x, a.requires_grad_()),
                 lambda: llsa.llsa_linear_attention(x[0], x[0], x[0], a.detach()),
                 lambda: llsa.llsa_linear_attention(x, x, x, a.detach(), initial_state=torch.zeros(1, 2, 64, 32)),
                 lambda: llsa.llsa_linear_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], a.detach(), torch.zeros(1, 2, 64, 64)),
                 lambda: llsa.llsa_linear_step(x[:, :, 0], x[:, :, 0], x[:, :1, 0], a.detach(), torch.zeros(1, 2, 64, 64)),
                 lambda: llsa.llsa_linear_step(x[:, :, 0], x[:, :, 0], x[:, :, 0], a.detach(), torch.zeros(1, 2, 64, 64).double())):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(llsa.LLSAError):
        llsa.llsa_linear_attention(x[..., :32], x[..., :32], x[..., :32], a.detach())
