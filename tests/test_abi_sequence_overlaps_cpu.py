"""Outputs that overlap an input or another output are refused before any launch, by raw
addresses."""
import ctypes

import pytest

from log_linear_hierarchical_b200 import _lib
from log_linear_hierarchical_b200._lib import LLSALinearShape


@pytest.fixture(scope="module")
def lib():
    from log_linear_hierarchical_b200 import build
    build.build()
    return _lib.load()


B, H, N, D = 2, 3, 4096, 64
TOK, ST = B * H * N * D * 2, B * H * D * D * 4
MB = 1 << 20


def shape(n=N):
    return LLSALinearShape(B, H, n, D, 0, 0.125)


@pytest.mark.parametrize("i,value", [
    (6, 64 * MB), (6, 64 * MB + TOK - 16), (6, 192 * MB - TOK + 16),       # o on q, its end, v's start
    (7, 192 * MB + 16), (8, 256 * MB + 32), (8, 320 * MB), (7, 256 * MB)])  # states and final state
def test_forward(lib, i, value):
    s = shape()
    # q, k, v, log_decay, lengths, initial, o, final, states
    args = [64 * MB, 128 * MB, 192 * MB, 16, None, 320 * MB, 256 * MB, 384 * MB, 448 * MB]
    args[i] = value
    assert lib.llsa_linear_forward(ctypes.byref(s), *args, None) == 1


@pytest.mark.parametrize("i,value", [(9, 64 * MB), (10, 576 * MB + 16), (11, 256 * MB), (12, 320 * MB), (12, 384 * MB),
                                     (13, 448 * MB), (13, 512 * MB), (12, 704 * MB)])
def test_backward(lib, i, value):
    s = shape()
    ws = lib.llsa_linear_workspace_bytes(ctypes.byref(s))
    # q, k, v, dO, log_decay, lengths, initial, d_final, states, dq, dk, dv, d_initial, workspace
    args = [64 * MB, 128 * MB, 192 * MB, 256 * MB, 16, None, 320 * MB, 384 * MB, 448 * MB, 512 * MB, 576 * MB, 640 * MB,
            768 * MB, 704 * MB]
    args[i] = value if i != 10 else 512 * MB + 16
    assert lib.llsa_linear_backward(ctypes.byref(s), *args, ws, None) == 1


@pytest.mark.parametrize("i,value", [(8, 64), (8, 4096), (4, 4096), (8, MB + 16), (6, MB), (7, MB + 64)])
def test_step(lib, i, value):
    s = shape(1)
    # q, k, v, log_decay, pool, rows, slots, out_slots, o
    args = [4096, 8192, 12288, 64, MB, 4, None, None, 65536]
    args[i] = value
    assert lib.llsa_linear_step(ctypes.byref(s), *args, None) == 1
