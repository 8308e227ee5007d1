"""Linear attention with a decay for each head: binding of llsa_linear_forward, _backward and
_step (include/llsa.h) and the autograd op."""
from __future__ import annotations

import ctypes
import functools

import torch
from torch.autograd.graph import increment_version

from . import _lib
from ._lib import LLSALinearShape
from .api import _DTYPES, LLSAError, _check, _stream
from .rotary import _current_stream, _no_tangents, _on_device, _torch_stream


def make_linear_shape(B: int, H: int, N: int, D: int, dtype, scale: float | None = None) -> LLSALinearShape:
    """``scale``: the factor of every output, 1 / sqrt(D) by default.  The strides of q, k, v and
    dO are filled in by the calls that take the tensors."""
    code = _DTYPES[dtype] if isinstance(dtype, torch.dtype) else int(dtype)
    return LLSALinearShape(B, H, N, D, code, _scale(D, scale))


def _scale(D: int, scale: float | None) -> float:
    """(a D that is refused later has no root)"""
    return (D ** -0.5 if D > 0 else 1.0) if scale is None else float(scale)


def llsa_linear_validate(shape: LLSALinearShape) -> int:
    return _lib.load().llsa_linear_validate(ctypes.byref(shape))


def llsa_linear_states_elems(shape: LLSALinearShape) -> int:
    return _lib.load().llsa_linear_states_elems(ctypes.byref(shape))


def llsa_linear_workspace_bytes(shape: LLSALinearShape) -> int:
    return _lib.load().llsa_linear_workspace_bytes(ctypes.byref(shape))


@functools.lru_cache(maxsize=1024)
def _sizes(B: int, H: int, N: int, D: int, code: int) -> tuple[int, int, int]:
    """(status, states elements, workspace bytes) of a shape, which need no device to ask."""
    ref = ctypes.byref(LLSALinearShape(B, H, N, D, code, 1.0))
    lib = _lib.load()
    return lib.llsa_linear_validate(ref), lib.llsa_linear_states_elems(ref), lib.llsa_linear_workspace_bytes(ref)


def _tokens(shape, t: torch.Tensor, name: str, strides) -> int:
    """Address of a [B, H, N, D] input whose strides (written to ``strides``; zeros stand for
    contiguous) the kernels take."""
    if t.shape != (shape.B, shape.H, shape.N, shape.D):
        raise ValueError(f"{name}: {tuple(t.shape)}, but the shape is {(shape.B, shape.H, shape.N, shape.D)}")
    if _DTYPES.get(t.dtype) != shape.dtype:
        raise ValueError(f"{name}: dtype {t.dtype} is not the shape's")
    _on_device(t, name)
    if not _readable(t):
        raise ValueError(f"{name}: strides {t.stride()} or alignment not taken (see include/llsa.h); make it contiguous")
    strides[:] = (0, 0, 0) if t.is_contiguous() else t.stride()[:3]
    return t.data_ptr()


def _readable(t: torch.Tensor) -> bool:
    """Whether the kernels read this view in place: channels contiguous, rows of whole 16 bytes."""
    if t.data_ptr() % 16:
        return False
    if t.is_contiguous():
        return True
    per16 = 16 // t.element_size()
    return t.stride(3) == 1 and all(n == 1 or (s > 0 and s % per16 == 0) for n, s in zip(t.shape[:3], t.stride()[:3]))


def _laid_out(t: torch.Tensor) -> torch.Tensor:
    return t if t.dim() != 4 or _readable(t) else t.clone(memory_format=torch.contiguous_format)


def _dense(t: torch.Tensor) -> torch.Tensor:
    return t if t.is_contiguous() and t.data_ptr() % 16 == 0 else t.clone(memory_format=torch.contiguous_format)


def _output(shape, t: torch.Tensor, name: str) -> int:
    if _DTYPES.get(t.dtype) != shape.dtype or t.numel() != shape.B * shape.H * shape.N * shape.D:
        raise ValueError(f"{name}: {tuple(t.shape)} {t.dtype}, but the shape needs B*H*N*D elements of its dtype")
    return _address(t, name)


def _address(t: torch.Tensor, name: str) -> int:
    if not t.is_contiguous():
        raise ValueError(f"{name}: LLSA buffers must be contiguous")
    return _on_device(t, name).data_ptr()


def _f32(t: torch.Tensor | None, need: int, name: str, scratch: bool = False) -> int | None:
    """Address of ``need`` fp32 values (scratch may have more)."""
    if t is None:
        return None
    if t.dtype != torch.float32 or t.numel() < need or (t.numel() > need and not scratch):
        raise ValueError(f"{name}: {t.numel()} elements of {t.dtype}, expected {need} of float32")
    return _address(t, name)


def _decay(t: torch.Tensor, H: int) -> int:
    """Address of log_decay: one value a head, shared by the batch (decays of another shape are other
    operators, not longer tables)."""
    if t.shape != (H,):
        raise ValueError(f"log_decay: {tuple(t.shape)}, expected ({H},), one value a head")
    return _f32(t, H, "log_decay")


def _i32(t: torch.Tensor | None, need: int, name: str) -> int | None:
    if t is None:
        return None
    if t.dtype != torch.int32 or t.numel() != need:
        raise ValueError(f"{name}: {t.numel()} elements of {t.dtype}, expected {need} of int32")
    return _address(t, name)


def _states(shape) -> int:
    return shape.B * shape.H * shape.D * shape.D


# Writes through an address, which torch does not see, are counted with increment_version as torch counts its
# own in-place operations: a backward that saved such a tensor before refuses to run.
def llsa_linear_forward(shape, q, k, v, log_decay, o, states=None, lengths=None, initial_state=None,
                        final_state=None, stream=None) -> None:
    sd = _states(shape)
    a = _decay(log_decay, shape.H)
    args = [_tokens(shape, q, "q", shape.q_strides), _tokens(shape, k, "k", shape.k_strides),
            _tokens(shape, v, "v", shape.v_strides), a,
            _i32(lengths, shape.B, "lengths"), _f32(initial_state, sd, "initial_state"), _output(shape, o, "o"),
            _f32(final_state, sd, "final_state"), _f32(states, _sizes(shape.B, shape.H, shape.N, shape.D, shape.dtype)[1], "states", True)]
    stream = _current_stream(q) if stream is None else _stream(stream)  # (q is on the device by now)
    _check("llsa_linear_forward", _lib.load().llsa_linear_forward(ctypes.byref(shape), *args, stream))
    increment_version(o if final_state is None else (o, final_state))


def llsa_linear_backward(shape, q, k, v, do, log_decay, dq, dk, dv, states=None, workspace=None, lengths=None,
                         initial_state=None, d_final=None, d_initial=None, stream=None) -> None:
    sd = _states(shape)
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    a = _decay(log_decay, shape.H)
    args = [_tokens(shape, q, "q", shape.q_strides), _tokens(shape, k, "k", shape.k_strides),
            _tokens(shape, v, "v", shape.v_strides), _tokens(shape, do, "do", shape.dO_strides),
            a, _i32(lengths, shape.B, "lengths"),
            _f32(initial_state, sd, "initial_state"), _f32(d_final, sd, "d_final"),
            _f32(states, _sizes(shape.B, shape.H, shape.N, shape.D, shape.dtype)[1], "states", True), _output(shape, dq, "dq"),
            _output(shape, dk, "dk"), _output(shape, dv, "dv"), _f32(d_initial, sd, "d_initial"),
            None if workspace is None else _address(workspace, "workspace")]
    stream = _current_stream(q) if stream is None else _stream(stream)
    _check("llsa_linear_backward", _lib.load().llsa_linear_backward(ctypes.byref(shape), *args, nbytes, stream))
    increment_version((dq, dk, dv) if d_initial is None else (dq, dk, dv, d_initial))


def _forward(q, k, v, log_decay, scale, initial_state, lengths, want_state):
    if q.dtype not in _DTYPES:
        raise ValueError(f"q: dtype {q.dtype}, expected bfloat16 or float32")
    shape = make_linear_shape(*q.shape, q.dtype, scale)
    st, n, _ = _sizes(shape.B, shape.H, shape.N, shape.D, shape.dtype)
    if st != 0:
        raise LLSAError("llsa_linear_validate", st)
    o = q.new_empty(q.shape)
    final = q.new_empty((shape.B, shape.H, shape.D, shape.D), dtype=torch.float32) if want_state else None
    states = q.new_empty(n, dtype=torch.float32) if n else None
    llsa_linear_forward(shape, q, k, v, log_decay, o, states, lengths, initial_state, final)
    return shape, o, final, states


class _LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay, scale, initial_state, lengths, want_state):
        ctx.set_materialize_grads(False)
        shape, o, final, states = _forward(q, k, v, log_decay, scale, initial_state, lengths, want_state)
        ctx.save_for_backward(q, k, v, log_decay, initial_state, lengths, states)
        ctx.scale = scale
        return (o, final) if want_state else o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do, d_final=None):
        _no_tangents(do, d_final)
        q, k, v, log_decay, initial_state, lengths, states = ctx.saved_tensors
        if do is None and d_final is None:
            return (None,) * 8
        shape = make_linear_shape(*q.shape, q.dtype, ctx.scale)
        do = q.new_zeros(q.shape) if do is None else _laid_out(do)
        d_final = None if d_final is None else _dense(d_final)
        dq, dk, dv = (q.new_empty(q.shape) for _ in range(3))  # (a kept gradient holds no other's memory or version)
        d_initial = torch.empty_like(initial_state) if ctx.needs_input_grad[5] else None
        n = _sizes(shape.B, shape.H, shape.N, shape.D, shape.dtype)[2]
        workspace = q.new_empty(n // 4, dtype=torch.float32) if n else None
        llsa_linear_backward(shape, q, k, v, do, log_decay, dq, dk, dv, states, workspace, lengths, initial_state,
                             d_final, d_initial)
        return dq, dk, dv, None, None, d_initial, None, None


def llsa_linear_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                          scale: float | None = None, initial_state: torch.Tensor | None = None,
                          lengths: torch.Tensor | None = None, return_state: bool = False):
    """Linear attention with a decay for each head over [B, H, N, D] CUDA tensors (D = 64 or 128,
    bf16 or fp32): with S = exp(log_decay[h]) S + k_t v_t^T after each token, o_t = scale * S^T q_t
    (``scale`` 1/sqrt(D) by default).  Cost is linear in N; gradients reach q, k, v and
    ``initial_state`` (forward-mode dual tensors are refused).

    ``log_decay``: [H] fp32, at most 0 in ordinary use; a constant (it gets no gradient).
    ``initial_state``: [B, H, D, D] fp32, the state before the first token (default 0).
    ``lengths``: [B] int32, the tokens of each row of a padded batch; the positions behind them
    take no part and get 0.  ``return_state``: returns (o, state after the last token), which
    ``llsa_linear_step`` or the next call's ``initial_state`` carries on from (for bf16 the last bits of o may
    depend on it: a state that is returned keeps more digits of its tokens).

    A NaN or infinity at a token may reach the earlier outputs of its chunk of 128 tokens (fp32: 64).
    Before a backward pass is captured into a CUDA graph, drop eager graphs of the same leaves (torch
    ties a leaf's gradient to the stream that the leaf was first used on).
    Views whose rows are whole 16-byte pieces (a [B, N, H, D] projection transposed) are read in
    place; others are copied first."""
    _no_tangents(q, k, v, log_decay, initial_state)
    if q.dim() != 4:
        raise ValueError(f"q: {tuple(q.shape)}, expected [B, H, N, D]")
    if log_decay.requires_grad and torch.is_grad_enabled():
        raise ValueError("log_decay gets no gradient: pass it detached")
    q, k, v = _laid_out(q), _laid_out(k), _laid_out(v)
    if initial_state is not None:
        if tuple(initial_state.shape) != (q.shape[0], q.shape[1], q.shape[3], q.shape[3]):
            raise ValueError(f"initial_state: {tuple(initial_state.shape)}, expected [B, H, D, D]")
        initial_state = _dense(initial_state)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in (q, k, v, initial_state)):
        return _LinearAttention.apply(q, k, v, log_decay, scale, initial_state, lengths, return_state)
    _, o, final, _ = _forward(q, k, v, log_decay, scale, initial_state, lengths, return_state)
    return (o, final) if return_state else o


def llsa_linear_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                     pool: torch.Tensor, scale: float | None = None, slots: torch.Tensor | None = None,
                     out_slots: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """One token of ``llsa_linear_attention`` for each of B requests: q, k, v are [B, H, D], ``pool``
    the fp32 states [P, H, D, D], updated in place.  Row b's state is pool[slots[b]] (default: slot b)
    and goes to pool[out_slots[b]] (default: the same slot); rows with a negative slot take no part
    and get 0.  Slots must not collide (see include/llsa.h).  Returns o, [B, H, D].  No gradients."""
    if stream is not None:  # copies and a new o belong to the stream that uses them
        with torch.cuda.stream(_torch_stream(stream)):
            return llsa_linear_step(q, k, v, log_decay, pool, scale, slots, out_slots, out)
    _no_tangents(q, k, v, log_decay, pool)
    size, dtype = q.shape, q.dtype
    if len(size) != 3 or dtype not in _DTYPES:
        raise ValueError(f"q: {tuple(size)} {dtype}, expected [B, H, D] of bfloat16 or float32")
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad or log_decay.requires_grad
                                    or pool.requires_grad or (out is not None and out.requires_grad)):
        raise ValueError("llsa_linear_step has no gradients: call it under no_grad")
    if k.shape != size or k.dtype != dtype or v.shape != size or v.dtype != dtype:
        raise ValueError(f"k, v: {tuple(k.shape)} {k.dtype} and {tuple(v.shape)} {v.dtype} do not go with q "
                         f"{tuple(size)} {dtype}")
    B, H, D = size
    if pool.dim() != 4 or pool.shape[1:] != (H, D, D) or pool.dtype != torch.float32:
        raise ValueError(f"pool: {tuple(pool.shape)} {pool.dtype}, expected [P, {H}, {D}, {D}] of float32")
    shape = _step_shape(B, H, D, _DTYPES[dtype], _scale(D, scale))
    a = _decay(log_decay, H)
    q, k, v = _dense(q), _dense(k), _dense(v)
    _on_device(q, "q")
    o = q.new_empty(size) if out is None else out
    status = _lib.load().llsa_linear_step(
        shape, _address(q, "q"), _address(k, "k"), _address(v, "v"), a,
        _address(pool, "pool"), pool.shape[0], _i32(slots, B, "slots"), _i32(out_slots, B, "out_slots"),
        o.data_ptr() if out is None else _step_output(q, out), _current_stream(q))
    if status:
        _check("llsa_linear_step", status)
    increment_version(pool if out is None else (pool, out))
    return o


def _step_output(q: torch.Tensor, out: torch.Tensor) -> int:
    if out.shape != q.shape or out.dtype != q.dtype:
        raise ValueError(f"out: {tuple(out.shape)} {out.dtype} is not q's {tuple(q.shape)} {q.dtype}")
    return _address(out, "out")


@functools.lru_cache(maxsize=1024)
def _step_shape(B: int, H: int, D: int, code: int, scale: float):
    """The (constant) shape of a single-token call, by reference."""
    return ctypes.byref(LLSALinearShape(B, H, 1, D, code, scale))
