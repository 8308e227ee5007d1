"""Outputs that cover the small inputs of the sequence operators -- decays, lengths, positions,
frequencies -- are refused before any launch, by raw addresses."""
import ctypes

import pytest

from log_linear_hierarchical_b200 import _lib
from log_linear_hierarchical_b200._lib import LLSALinearShape, LLSARotaryShape

B, H, N, D = 2, 3, 4096, 64
TOK, ST = B * H * N * D * 2, B * H * D * D * 4
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from log_linear_hierarchical_b200 import build
    build.build()
    return _lib.load()


# q, k, v, log_decay, lengths, initial, o, final, states
FORWARD = [64 * MB, 128 * MB, 192 * MB, 16, None, 320 * MB, 256 * MB, 384 * MB, 448 * MB]
# q, k, v, dO, log_decay, lengths, initial, d_final, states, dq, dk, dv, d_initial, workspace
BACKWARD = [64 * MB, 128 * MB, 192 * MB, 256 * MB, 16, None, 320 * MB, 384 * MB, 448 * MB, 512 * MB, 576 * MB, 640 * MB,
            768 * MB, 704 * MB]


def ends(lo, size, own):
    """Addresses of a table of `own` bytes that touch an output's first and last bytes."""
    return lo, lo + 4 - own, lo + size - 4


@pytest.mark.parametrize("table,own", [(3, 4 * H), (4, 4 * B)])
@pytest.mark.parametrize("out", [6, 7, 8])
def test_forward(lib, table, own, out):
    s = LLSALinearShape(B, H, N, D, 0, 0.125)
    size = {6: TOK, 7: ST, 8: 4 * lib.llsa_linear_states_elems(ctypes.byref(s))}[out]
    assert size > 0
    for at in ends(FORWARD[out], size, own):
        args = list(FORWARD)
        args[table] = at
        assert lib.llsa_linear_forward(ctypes.byref(s), *args, None) == 1
    args = list(FORWARD)
    args[5], args[3] = args[7], args[7] + 64   # the state in place, with the decays inside it
    assert lib.llsa_linear_forward(ctypes.byref(s), *args, None) == 1


@pytest.mark.parametrize("table,own", [(4, 4 * H), (5, 4 * B)])
@pytest.mark.parametrize("out", [9, 10, 11, 12, 13])
def test_backward(lib, table, own, out):
    s = LLSALinearShape(B, H, N, D, 0, 0.125)
    ws = lib.llsa_linear_workspace_bytes(ctypes.byref(s))
    size = ST if out == 12 else ws if out == 13 else TOK
    for at in ends(BACKWARD[out], size, own):
        args = list(BACKWARD)
        args[table] = at
        assert lib.llsa_linear_backward(ctypes.byref(s), *args, ws, None) == 1


@pytest.mark.parametrize("pos32,stride", [(False, 0), (False, 11), (True, 0), (True, 9)])
@pytest.mark.parametrize("second", [False, True])
def test_rotary(lib, pos32, stride, second):
    n, rot, width = 8, 46, 4 if pos32 else 8
    y = {False: 64 * MB, True: 128 * MB}
    size = {False: 2 * 3 * n * 64 * 2, True: 2 * 5 * n * 64 * 2}[second]
    s = LLSARotaryShape(B=2, H=3, H2=5, N=n, D=64, dtype=0, rot=rot, first=0, flags=4 if pos32 else 0, scale=1.0)

    def call(pos, freq):
        return lib.llsa_rotary(ctypes.byref(s), 16 * MB, None, 32 * MB, None, pos, stride, freq, y[False], y[True], None)

    lo, reach = y[second], (stride + n) * width    # (two batch rows of positions)
    for at in (lo, lo + width - reach, lo + size - width):
        assert call(at, 4096) == 1
    for at in (lo, lo + 8 - 8 * (rot // 2), lo + size - 8):
        assert call(8192, at) == 1
