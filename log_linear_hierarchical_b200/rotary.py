"""Rotary positions for q and k: binding of llsa_rotary (include/llsa.h), its autograd op and
the frequency tables."""
from __future__ import annotations

import ctypes
import functools
import math

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version

from . import _lib
from ._lib import LLSARotaryShape
from .api import _DTYPES, _check


def llsa_rotary_frequencies(rot: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                            original_length: int | None = None, low: float = 1.0, high: float = 32.0,
                            device=None) -> tuple[torch.Tensor, float]:
    """Radians per position of the rot/2 pairs (an fp64 tensor) and the factor of the rotated
    channels, both as ``llsa_rotary`` takes them.  Pair c has base^(-2c / rot), scaled for
    contexts ``factor`` times as long as the ones trained on:

    - ``"linear"``: every frequency divided by ``factor`` (positions squeezed into the old range);
    - ``"ntk"``: the base multiplied by factor^(rot / (rot - 2)), which divides the slowest pair by
      ``factor`` and leaves the fastest;
    - ``"yarn"``: pairs that turn fewer than ``low`` times in ``original_length`` positions divided by
      ``factor``, those that turn more than ``high`` times kept, the ones between blended linearly in
      their turns; the rotated channels are multiplied by 0.1 ln(factor) + 1.
    """
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    if not base > 0 or not factor >= 1:
        raise ValueError("base must be positive and factor at least 1")
    n = rot // 2
    if scaling == "ntk":
        if n < 2:
            raise ValueError("ntk scaling needs rot of at least 4")
        base = base * factor ** (rot / (rot - 2))
    f = torch.tensor([base ** (-c / n) for c in range(n)], dtype=torch.float64)
    scale = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "yarn":
        if original_length is None or not 0 <= low < high:
            raise ValueError("yarn scaling needs original_length and 0 <= low < high")
        turns = original_length * f / (2.0 * math.pi)
        keep = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        f = f * keep + f / factor * (1.0 - keep)
        scale = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError(f"scaling {scaling!r} is none of 'linear', 'ntk', 'yarn'")
    return f.to(device) if device is not None else f, scale


def _on_device(t: torch.Tensor, name: str) -> torch.Tensor:
    """A CUDA tensor on the current device (the kernels read and write its address)."""
    if not t.is_cuda:
        raise ValueError(f"{name}: LLSA buffers must be CUDA tensors (the kernels read device memory)")
    if t.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")
    return t


def _current_stream(t: torch.Tensor) -> int:
    """The current stream of t's device as an address (without torch.cuda's wrapper object, which
    costs as much as a launch)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _torch_stream(stream) -> torch.cuda.Stream:
    return stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))


def _no_tangents(*tensors) -> None:
    """Refuses forward-mode dual tensors: the kernels read the primal's address, and the tangent would
    be lost without a word."""
    if forward_ad._current_level >= 0 and any(
            t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors):
        raise ValueError("forward-mode gradients (dual tensors) are not supported")


def _heads(t: torch.Tensor, name: str, like: torch.Tensor) -> torch.Tensor:
    """A [B, H, N, D] tensor of like's batch, length, channels and dtype (any head count)."""
    if t.dim() != 4:
        raise ValueError(f"{name}: {t.dim()} dimensions, expected [B, H, N, D]")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name}: dtype {t.dtype}, expected bfloat16 or float32")
    if t.dtype != like.dtype or t.shape[0] != like.shape[0] or t.shape[2:] != like.shape[2:]:
        raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype} does not go with {tuple(like.shape)} {like.dtype}")
    return _on_device(t, name)


_Strides = ctypes.c_int64 * 3


@functools.lru_cache(maxsize=1024)
def _shape(*fields):
    """A (constant) llsa_rotary_shape, by reference."""
    return ctypes.byref(LLSARotaryShape(*fields))


def _rotate(xs, outs, positions, frequencies, interleaved, first, scale, inverse) -> list:
    """One launch over one or two tensors; ``outs`` None makes new contiguous ones."""
    x = xs[0]
    B, H, N, D = x.shape
    _heads(x, "q", x)
    if len(xs) == 2:
        _heads(xs[1], "k", x)
    if frequencies.dtype != torch.float64 or frequencies.dim() != 1 or not frequencies.is_contiguous():
        raise ValueError("frequencies: expected a contiguous 1-D float64 tensor, one value for each pair")
    _on_device(frequencies, "frequencies")
    flags = (_lib.LLSA_ROTARY_INTERLEAVED if interleaved else 0) | (_lib.LLSA_ROTARY_INVERSE if inverse else 0)
    pos, pos_stride = None, 0
    if positions is not None:
        if positions.dtype not in (torch.int64, torch.int32):
            raise ValueError(f"positions: dtype {positions.dtype}, expected int64 or int32")
        if tuple(positions.shape) not in ((N,), (B, N)):
            raise ValueError(f"positions: {tuple(positions.shape)}, expected ({N},) or ({B}, {N})")
        if N > 1 and positions.stride(-1) != 1:
            positions = positions.contiguous()
        pos = _on_device(positions, "positions").data_ptr()
        pos_stride = positions.stride(0) if positions.dim() == 2 and B > 1 else 0
        if positions.dtype == torch.int32:
            flags |= _lib.LLSA_ROTARY_POSITIONS_I32
    xs = [t if t.stride(-1) == 1 else t.contiguous() for t in xs]
    if outs is None:
        outs = [t.new_empty(t.shape) for t in xs]
    two = len(xs) == 2
    stream = _current_stream(x)
    shape = _shape(B, H, xs[1].shape[1] if two else 0, N, D, _DTYPES[x.dtype], 2 * frequencies.numel(), int(first),
                   flags, float(scale))
    strides = [None if t.is_contiguous() else _Strides(*t.stride()[:3]) for t in xs]
    _check("llsa_rotary", _lib.load().llsa_rotary(
        shape, xs[0].data_ptr(), strides[0], xs[1].data_ptr() if two else None,
        strides[1] if two else None, pos, pos_stride, frequencies.data_ptr(), outs[0].data_ptr(),
        outs[1].data_ptr() if two else None, stream))
    return outs


class _Rotary(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, frequencies, interleaved, first, scale):
        ctx.set_materialize_grads(False)
        # torch refuses a backward after either is written again, and tensors of inference mode at all
        if frequencies.is_inference():
            frequencies = frequencies.clone()
        if positions is not None and positions.is_inference():
            positions = positions.clone()
        ctx.save_for_backward(positions, frequencies)
        ctx.args = (interleaved, first, scale)
        outs = _rotate([q] if k is None else [q, k], None, positions, frequencies, interleaved, first, scale, False)
        return outs[0] if k is None else tuple(outs)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, *grads):
        _no_tangents(*grads)
        positions, frequencies = ctx.saved_tensors
        interleaved, first, scale = ctx.args
        there = [i for i, g in enumerate(grads) if g is not None and ctx.needs_input_grad[i]]
        back = [None, None]
        if there:
            outs = _rotate([grads[i] for i in there], None, positions, frequencies, interleaved, first, scale, True)
            for i, o in zip(there, outs):
                back[i] = o
        return (*back, None, None, None, None, None)


def llsa_rotary(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor | None, frequencies: torch.Tensor,
                *, interleaved: bool = False, first: int = 0, scale: float = 1.0, inplace: bool = False,
                stream=None):
    """q and k ([B, H, N, D] and [B, Hk, N, D] CUDA tensors, bf16 or fp32, D = 64 or 128, any
    strides of the first three dimensions) turned by their positions, as new contiguous
    [B, H, N, D] tensors, in one launch; only q if ``k`` is None.

    ``positions``: int64 or int32, [N] or [B, N]; None for 0..N-1.  ``frequencies``: fp64, one for
    each pair of channels, radians per position (``llsa_rotary_frequencies``); the 2 * len channels
    from ``first`` on are turned, in the half layout (c with c + len) or ``interleaved`` (2c with
    2c + 1), and multiplied by ``scale``; the others are copied.  Gradients reach q and k by the
    inverse rotation (under grad, on the current stream); forward-mode dual tensors are refused, and
    so is a backward pass after ``positions`` or ``frequencies`` were written again.  Before a backward pass is
    captured into a CUDA graph, drop eager graphs of the same leaves (torch ties a leaf's gradient to the
    stream that the leaf was first used on).  ``inplace`` (contiguous tensors, no gradients): q and k
    themselves are overwritten and returned."""
    if stream is not None:  # copies and new tensors belong to the stream that uses them
        with torch.cuda.stream(_torch_stream(stream)):
            return llsa_rotary(q, k, positions, frequencies, interleaved=interleaved, first=first, scale=scale,
                               inplace=inplace)
    _no_tangents(q, k, frequencies)
    if frequencies.requires_grad and torch.is_grad_enabled():
        raise ValueError("frequencies get no gradient: pass them detached")
    if torch.is_grad_enabled() and (q.requires_grad or (k is not None and k.requires_grad)):
        if inplace:
            raise ValueError("inplace is for calls without gradients")
        return _Rotary.apply(q, k, positions, frequencies, interleaved, first, scale)
    xs = [q] if k is None else [q, k]
    if inplace and not all(t.is_contiguous() for t in xs):
        raise ValueError("inplace needs contiguous tensors")
    outs = _rotate(xs, xs if inplace else None, positions, frequencies, interleaved, first, scale, False)
    if inplace:  # torch sees no write through an address: a backward that saved q or k would not either
        increment_version(xs)
    return outs[0] if k is None else tuple(outs)
