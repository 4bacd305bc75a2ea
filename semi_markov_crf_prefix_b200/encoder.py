"""What makes emissions of long sequences: linear attention with a decay for each
head, and group norm with an activation on channels-last rows.

``linear_attention`` and ``group_norm`` are differentiable (torch.autograd); the
``*_forward`` / ``*_backward`` pairs are the library's calls, with the workspace in
the caller's hands when given.  ``linear_attention_step`` is the form for single
positions, with the state updated in place.  Argument marshalling only: every step
runs in libsemicrf.so (C ABI in ``include/semicrf.h``), on the current CUDA stream
of the tensors' device.

Layout: q, k [B,T,H,dk], v, o [B,T,H,dv] with a dense last axis and any strides
before it; states float32 [B,H,dk,dv]; log_decay float32 [H]; x, y [N,...,C]
contiguous; lengths int32, as everywhere in this package: what lies behind a
sequence's end is not read, and is zero in outputs.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import _lib

ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2}
_TYPES = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16, torch.float16: _lib.F16}
_SAME = contextlib.nullcontext()


def _guard(device):
    return _SAME if device.index == torch.cuda.current_device() else torch.cuda.device(device)


def _call(name, device, *args):
    """One library call on the device's current stream (appended as the last argument)."""
    with _guard(device):
        status = getattr(_lib.load(), "semicrf_" + name)(*args, torch.cuda.current_stream(device).cuda_stream)
    if status:
        _lib.check(status, name)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _want(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _workspace(ws, need, device):
    if ws is None:
        return torch.empty(need, dtype=torch.uint8, device=device)
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise TypeError("ws must be a contiguous CUDA uint8 tensor")
    if ws.device != device:
        raise ValueError(f"ws is on {ws.device}, expected {device}")
    return ws


# ---------------------------------------------------------------- linear attention

def _operand(t, name, first, width=None):
    """Checks one of q, k, v (or an upstream gradient) against `first`."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != first.dtype:
        raise TypeError(f"{name} must be {first.dtype} like q, got {t.dtype}")
    if t.dim() != first.dim() or t.shape[:-1] != first.shape[:-1] or (width is not None and t.shape[-1] != width):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, which does not match q {tuple(first.shape)}")
    if t.device != first.device:
        raise ValueError(f"{name} is on {t.device}, expected {first.device}")
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"the last axis of {name} must be dense")


def _attention_dims(q, k, v, log_decay, scale, reverse, axes):
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise TypeError("q must be a CUDA tensor")
    if q.dtype not in _TYPES:
        raise TypeError(f"q must be float32, bfloat16 or float16, got {q.dtype}")
    if q.dim() != axes:
        raise ValueError(f"q must have {axes} axes, got {q.dim()}")
    dk, dv = q.shape[-1], v.shape[-1]
    _operand(q, "q", q)
    _operand(k, "k", q, dk)
    _operand(v, "v", q)
    if log_decay.requires_grad:
        raise ValueError("log_decay is a constant: it has no gradient")
    H = q.shape[-2]
    _want(log_decay, "log_decay", torch.float32, (H,), q.device)
    d = _lib.AttentionDims(q.shape[0], q.shape[1] if axes == 4 else 1, H, dk, dv, _TYPES[q.dtype], int(bool(reverse)),
                           dk ** -0.5 if scale is None else scale)
    _strides(d.q_stride, q)
    _strides(d.k_stride, k)
    _strides(d.v_stride, v)
    return d


def _strides(to, t):
    if t.dim() == 4:
        to[0], to[1], to[2], _ = t.stride()
    else:
        to[0], to[2], _ = t.stride()


def _extras(q, dv, lengths, state, state_name):
    B, H, dk = q.shape[0], q.shape[-2], q.shape[-1]
    if lengths is not None:
        _want(lengths, "lengths", torch.int32, (B,), q.device)
    if state is not None:
        _want(state, state_name, torch.float32, (B, H, dk, dv), q.device)


def linear_attention_workspace_bytes(q, v, backward=False) -> int:
    """Bytes of workspace of a call with operands like q [B,T,H,dk] and v [B,T,H,dv]."""
    d = _lib.AttentionDims(*q.shape[:3], q.shape[3], v.shape[3], _TYPES[q.dtype], 0, 1.0)
    return _attention_ws(d, backward)


def _attention_ws(d, backward):
    n = _lib.load().semicrf_linear_attention_workspace_bytes(ctypes.byref(d), int(backward))
    if n == 0:
        bad = max(d.dk, d.dv) > _lib.MAX_HEAD
        raise ValueError(f"unsupported dimensions: B {d.B}, T {d.T}, H {d.H}, dk {d.dk}, dv {d.dv}"
                         + (f" (at most {_lib.MAX_HEAD} wide)" if bad else ""))
    return n


def linear_attention_forward(q, k, v, log_decay, lengths=None, scale=None, initial_state=None, return_state=False,
                             reverse=False, ws=None):
    """(o [B,T,H,dv], state [B,H,dk,dv] float32 or None): S = lam S + k v^T, o = scale q S
    with lam = exp(log_decay) (at most 1), from the first position on or, reversed, from
    the last valid one; scale None: dk ** -0.5."""
    d = _attention_dims(q, k, v, log_decay, scale, reverse, 4)
    _extras(q, d.dv, lengths, initial_state, "initial_state")
    ws = _workspace(ws, _attention_ws(d, False), q.device)
    o = torch.empty((d.B, d.T, d.H, d.dv), dtype=q.dtype, device=q.device)
    _strides(d.o_stride, o)
    state = torch.empty((d.B, d.H, d.dk, d.dv), dtype=torch.float32, device=q.device) if return_state else None
    _call("linear_attention", q.device, ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(lengths),
          _ptr(initial_state), _ptr(o), _ptr(state), _ptr(ws), ws.numel())
    return o, state


def linear_attention_backward(grad_o, q, k, v, log_decay, lengths=None, scale=None, initial_state=None,
                              grad_state=None, reverse=False, want_initial_state=False, ws=None):
    """(dq, dk, dv, d initial_state or None) for the upstream grad_o [B,T,H,dv] and, where
    the returned state was used, grad_state [B,H,dk,dv] float32."""
    d = _attention_dims(q, k, v, log_decay, scale, reverse, 4)
    _operand(grad_o, "grad_o", q, d.dv)
    _extras(q, d.dv, lengths, initial_state, "initial_state")
    _extras(q, d.dv, None, grad_state, "grad_state")
    _strides(d.o_stride, grad_o)
    ws = _workspace(ws, _attention_ws(d, True), q.device)
    new = lambda width: torch.empty((d.B, d.T, d.H, width), dtype=q.dtype, device=q.device)  # noqa: E731
    dq, dk, dv = new(d.dk), new(d.dk), new(d.dv)
    ds = (torch.empty((d.B, d.H, d.dk, d.dv), dtype=torch.float32, device=q.device) if want_initial_state else None)
    _call("linear_attention_backward", q.device, ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay),
          _ptr(lengths), _ptr(initial_state), _ptr(grad_o), _ptr(grad_state), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ds),
          _ptr(ws), ws.numel())
    return dq, dk, dv, ds


class LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, initial_state, log_decay, lengths, scale, reverse, return_state):
        o, state = linear_attention_forward(q, k, v, log_decay, lengths, scale, initial_state, return_state, reverse)
        ctx.save_for_backward(q, k, v, initial_state, log_decay, lengths)
        ctx.how = (scale, reverse)
        ctx.set_materialize_grads(False)
        return (o, state) if return_state else o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_o, grad_state=None):
        q, k, v, initial_state, log_decay, lengths = ctx.saved_tensors
        scale, reverse = ctx.how
        if grad_o is None and grad_state is None:
            return (None,) * 9
        if grad_o is None:
            grad_o = torch.zeros((*q.shape[:3], v.shape[3]), dtype=q.dtype, device=q.device)
        elif grad_o.stride(-1) != 1:
            grad_o = grad_o.contiguous()
        if grad_state is not None:
            grad_state = grad_state.contiguous()
        want = initial_state is not None and ctx.needs_input_grad[3]
        dq, dk, dv, ds = linear_attention_backward(grad_o, q, k, v, log_decay, lengths, scale, initial_state,
                                                   grad_state, reverse, want)
        return dq, dk, dv, ds, None, None, None, None, None


def linear_attention(q, k, v, log_decay, lengths=None, scale=None, initial_state=None, return_state=False,
                     reverse=False):
    """o [B,T,H,dv], or (o, state) with return_state; differentiable with respect to q, k, v
    and initial_state.  Arguments as for linear_attention_forward."""
    return _differentiable(LinearAttention, (q, k, v, initial_state), (q, k, v, initial_state, log_decay, lengths,
                                                                       scale, reverse, return_state),
                           lambda: _drop(linear_attention_forward(q, k, v, log_decay, lengths, scale, initial_state,
                                                                  return_state, reverse), return_state))


def _drop(pair, both):
    return pair if both else pair[0]


def _differentiable(function, inputs, args, plain):
    """function.apply where a gradient may be asked for, else the call alone."""
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs):
        return function.apply(*args)
    return plain()


def linear_attention_step(q, k, v, log_decay, state, scale=None):
    """One position: state [B,H,dk,dv] float32 becomes lam state + k v^T in place; returns
    o [B,H,dv] = scale q state.  q, k [B,H,dk], v [B,H,dv].  No gradient is recorded."""
    d = _attention_dims(q, k, v, log_decay, scale, False, 3)
    _want(state, "state", torch.float32, (d.B, d.H, d.dk, d.dv), q.device)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad or state.requires_grad):
        raise ValueError("linear_attention_step records no gradient: use linear_attention, or torch.no_grad()")
    o = torch.empty((d.B, d.H, d.dv), dtype=q.dtype, device=q.device)
    _strides(d.o_stride, o)
    _call("linear_attention_step", q.device, ctypes.byref(d), _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(state),
          _ptr(o))
    return o


# ---------------------------------------------------------------- group norm

def _norm_dims(x, groups, weight, bias, lengths, eps, activation):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise TypeError("x must be a CUDA tensor")
    if x.dtype not in _TYPES:
        raise TypeError(f"x must be float32, bfloat16 or float16, got {x.dtype}")
    if x.dim() < 2 or x.numel() == 0:
        raise ValueError(f"x must be [N,...,C] and not empty, got shape {tuple(x.shape)}")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    N, C = x.shape[0], x.shape[-1]
    if groups < 1 or C % groups:
        raise ValueError(f"{C} channels do not split into {groups} groups")
    some = weight if weight is not None else bias
    wtype = torch.float32 if some is None else some.dtype
    if wtype != torch.float32 and wtype != x.dtype:
        raise TypeError(f"weight and bias must be float32 or {x.dtype}, got {wtype}")
    for t, name in ((weight, "weight"), (bias, "bias")):
        if t is not None:
            _want(t, name, wtype, (C,), x.device)
    if lengths is not None:
        if x.dim() != 3:
            raise ValueError("lengths need x of shape [N,S,C]")
        _want(lengths, "lengths", torch.int32, (N,), x.device)
    return _lib.NormDims(N, x.numel() // (N * C), C, groups, _TYPES[x.dtype], _TYPES[wtype], ACTIVATIONS[activation],
                         eps)


def group_norm_workspace_bytes(x, groups, backward=False) -> int:
    """Bytes of workspace of a call with rows like x [N,...,C]."""
    return _norm_ws(_norm_dims(x, groups, None, None, None, 1e-5, "none"), backward)


def _norm_ws(d, backward):
    n = _lib.load().semicrf_group_norm_workspace_bytes(ctypes.byref(d), int(backward))
    if n == 0:
        raise ValueError(f"unsupported arguments: N {d.N}, S {d.S}, C {d.C}, groups {d.G}, eps {d.eps}")
    return n


def group_norm_forward(x, groups, weight=None, bias=None, lengths=None, eps=1e-5, activation="none", ws=None):
    """(y like x, stats [N,groups,2] float32: mean and 1/std of the valid positions)."""
    d = _norm_dims(x, groups, weight, bias, lengths, eps, activation)
    ws = _workspace(ws, _norm_ws(d, False), x.device)
    y = torch.empty_like(x)
    stats = torch.empty((d.N, d.G, 2), dtype=torch.float32, device=x.device)
    _call("group_norm", x.device, ctypes.byref(d), _ptr(x), _ptr(weight), _ptr(bias), _ptr(lengths), _ptr(y),
          _ptr(stats), _ptr(ws), ws.numel())
    return y, stats


def group_norm_backward(dy, x, stats, groups, weight=None, bias=None, lengths=None, eps=1e-5, activation="none",
                        want_params=True, ws=None):
    """(dx like x, dweight [C] float32, dbias [C] float32); the last two None without want_params."""
    d = _norm_dims(x, groups, weight, bias, lengths, eps, activation)
    _want(dy, "dy", x.dtype, x.shape, x.device)
    _want(stats, "stats", torch.float32, (d.N, d.G, 2), x.device)
    ws = _workspace(ws, _norm_ws(d, True), x.device)
    dx = torch.empty_like(x)
    dw, db = (torch.empty((2, d.C), dtype=torch.float32, device=x.device) if want_params else (None, None))
    _call("group_norm_backward", x.device, ctypes.byref(d), _ptr(dy), _ptr(x), _ptr(weight), _ptr(bias),
          _ptr(lengths), _ptr(stats), _ptr(dx), _ptr(dw), _ptr(db), _ptr(ws), ws.numel())
    return dx, dw, db


class GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, groups, lengths, eps, activation):
        y, stats = group_norm_forward(x, groups, weight, bias, lengths, eps, activation)
        ctx.save_for_backward(x, weight, bias, lengths, stats)
        ctx.how = (groups, eps, activation)
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, weight, bias, lengths, stats = ctx.saved_tensors
        groups, eps, activation = ctx.how
        want = ctx.needs_input_grad[1] or ctx.needs_input_grad[2]
        dx, dw, db = group_norm_backward(dy.contiguous(), x, stats, groups, weight, bias, lengths, eps, activation,
                                         want)
        return (dx, dw.to(weight.dtype) if ctx.needs_input_grad[1] else None,
                db.to(bias.dtype) if ctx.needs_input_grad[2] else None, None, None, None, None)


def group_norm(x, groups, weight=None, bias=None, lengths=None, eps=1e-5, activation="none"):
    """act((x - mean) / std * weight + bias) of x [N,...,C], with the statistics of each n and
    each of the `groups` groups of channels over all positions (over the first lengths[n] of
    x [N,S,C], zero behind them); activation "none", "silu" or "gelu".  Differentiable with
    respect to x, weight and bias."""
    return _differentiable(GroupNorm, (x, weight, bias), (x, weight, bias, groups, lengths, eps, activation),
                           lambda: group_norm_forward(x, groups, weight, bias, lengths, eps, activation)[0])
