"""What makes emissions of long sequences: linear attention with a decay for each
head, and group norm with an activation on channels-last rows.

``linear_attention`` and ``group_norm`` are differentiable (torch.autograd, once and in
reverse mode; forward-mode tangents and second derivatives are refused); the
``*_forward`` / ``*_backward`` pairs are the library's calls, with the workspace in
the caller's hands when given.  ``linear_attention_step`` is the form for single
positions, with the state updated in place.  Argument marshalling only: every step
runs in libsemicrf.so (C ABI in ``include/semicrf.h``), on the current CUDA stream
of the tensors' device.

Layout: q, k [B,T,H,dk], v, o [B,T,H,dv] with a dense last axis and any strides
before it; states float32 [B,H,dk,dv]; log_decay float32 [H]; x, y [N,...,C]
contiguous; lengths int32, as everywhere in this package: what lies behind a
sequence's end is not read, and is zero in outputs.  A length outside its range is found on
the device: it is taken as the nearest one inside, and ``device_status()`` of this package
returns the code, for any call until ``clear_device_status()``.  A workspace given as `ws` has
a status word of its own, which its owner clears before the first call.
"""
from __future__ import annotations

import torch
from torch._C import _cuda_getCurrentRawStream as _raw_stream
from torch.autograd import forward_ad

from . import _lib

ACTIVATIONS = {"none": 0, "silu": 1, "gelu": 2}
_TYPES = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16, torch.float16: _lib.F16}
_functions = {}


def _call(name, device, *args):
    """One library call on the device's current stream (appended as the last argument)."""
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(_lib.load(), "semicrf_" + name)
    index = device.index
    if index == torch.cuda.current_device():
        status = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            status = f(*args, _raw_stream(index))
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

def _operand(t, name, q, shape):
    """Checks k, v or an upstream gradient against q and the shape it has to have."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != q.dtype:
        raise TypeError(f"{name} must be {q.dtype} like q, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, which does not match q {tuple(q.shape)}")
    if t.device != q.device:
        raise ValueError(f"{name} is on {t.device}, expected {q.device}")
    strides = t.stride()
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"the last axis of {name} must be dense")
    return strides


def _constant(log_decay):
    if isinstance(log_decay, torch.Tensor) and log_decay.requires_grad and torch.is_grad_enabled():
        raise ValueError("log_decay is a constant: it has no gradient (detach it, or call under torch.no_grad())")


def _attention(q, k, v, log_decay, axes):
    """(device, type, shape of q, width of v, strides of q, k and v) of checked operands."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise TypeError("q must be a CUDA tensor")
    kind = _TYPES.get(q.dtype)
    if kind is None:
        raise TypeError(f"q must be float32, bfloat16 or float16, got {q.dtype}")
    shape = q.shape
    if len(shape) != axes:
        raise ValueError(f"q must have {axes} axes, got {len(shape)}")
    device = q.device
    qs = _operand(q, "q", q, shape)
    ks = _operand(k, "k", q, shape)
    dv = v.shape[-1] if isinstance(v, torch.Tensor) and v.dim() else 0
    vs = _operand(v, "v", q, (*shape[:-1], dv))
    _constant(log_decay)
    _want(log_decay, "log_decay", torch.float32, shape[-2:-1], device)
    return device, kind, shape, dv, qs, ks, vs


def _dims(kind, shape, dv, scale, reverse, qs, ks, vs, os):
    B, T, H, dk = shape
    return _lib.ATTENTION_DIMS.pack(B, T, H, dk, dv, kind, 1 if reverse else 0, dk ** -0.5 if scale is None else scale,
                                    *qs[:3], *ks[:3], *vs[:3], *os[:3])


def _extras(shape, dv, device, lengths, state, state_name):
    if lengths is not None:
        _want(lengths, "lengths", torch.int32, shape[:1], device)
    if state is not None:
        _want(state, state_name, torch.float32, (shape[0], shape[2], shape[3], dv), device)


def linear_attention_workspace_bytes(q, v, backward=False) -> int:
    """Bytes of workspace that serve any call with operands like q [B,T,H,dk] and v [B,T,H,dv],
    whatever their strides and addresses (the calls themselves make what theirs need)."""
    none = (0, 0, 0)
    d = _dims(_TYPES[q.dtype], q.shape, v.shape[3], 1.0, False, none, none, none, none)
    return _supported(_lib.load().semicrf_linear_attention_workspace_bytes(d, 1 if backward else 0), q.shape, v.shape[3])


def _supported(n, shape, dv):
    if n == 0:
        bad = max(shape[3], dv) > _lib.MAX_HEAD
        raise ValueError(f"unsupported arguments: q {tuple(shape)}, width of v {dv}"
                         + (f" (at most {_lib.MAX_HEAD} wide)" if bad else ""))
    return n


def _attention_ws_at(dims, shape, dv, backward, q, k, v, o):
    return _supported(_lib.load().semicrf_linear_attention_workspace_bytes_at(dims, backward, q, k, v, o), shape, dv)


def _walk(name, dims, shape, dv, backward, q, k, v, o, device, ws, *args):
    """A call with the workspace given, or with one of the operands' size: args, ws and its bytes."""
    own = ws is None
    need = _attention_ws_at(dims, shape, dv, backward, q, k, v, o)
    ws = _workspace(ws, need, device)
    try:
        _call(name, device, *args, ws.data_ptr(), ws.numel())
    except _lib.SemiCRFError as e:
        if not own or e.status != _lib.SEMICRF_ERR_WORKSPACE_TOO_SMALL:
            raise
        # the copy engine's maps were refused: the size for any operands
        ws = _workspace(None, _lib.load().semicrf_linear_attention_workspace_bytes(dims, backward), device)
        _call(name, device, *args, ws.data_ptr(), ws.numel())


def _dense(shape, width):
    return shape[1] * shape[2] * width, shape[2] * width, width


def linear_attention_forward(q, k, v, log_decay, lengths=None, scale=None, initial_state=None, return_state=False,
                             reverse=False, ws=None):
    """(o [B,T,H,dv], state [B,H,dk,dv] float32 or None): S = lam S + k v^T, o = scale q S
    with lam = exp(log_decay) (at most 1), from the first position on or, reversed, from
    the last valid one; scale None: dk ** -0.5."""
    device, kind, shape, dv, qs, ks, vs = _attention(q, k, v, log_decay, 4)
    _extras(shape, dv, device, lengths, initial_state, "initial_state")
    d = _dims(kind, shape, dv, scale, reverse, qs, ks, vs, _dense(shape, dv))
    return _attention_run(q, k, v, log_decay, lengths, initial_state, return_state, d, shape, dv, device, ws)


def _attention_run(q, k, v, log_decay, lengths, initial_state, return_state, d, shape, dv, device, ws):
    B, T, H, dk = shape
    qp, kp, vp = q.data_ptr(), k.data_ptr(), v.data_ptr()
    _supported(B * T * H * dk * dv, shape, dv)
    o = torch.empty((B, T, H, dv), dtype=q.dtype, device=device)
    state = torch.empty((B, H, dk, dv), dtype=torch.float32, device=device) if return_state else None
    op = o.data_ptr()
    _walk("linear_attention", d, shape, dv, 0, qp, kp, vp, op, device, ws, d, qp, kp, vp, log_decay.data_ptr(),
          _ptr(lengths), _ptr(initial_state), op, _ptr(state))
    return o, state


def linear_attention_backward(grad_o, q, k, v, log_decay, lengths=None, scale=None, initial_state=None,
                              grad_state=None, reverse=False, want_initial_state=False, ws=None):
    """(dq, dk, dv, d initial_state or None) for the upstream grad_o [B,T,H,dv] and, where
    the returned state was used, grad_state [B,H,dk,dv] float32."""
    device, kind, shape, dv, qs, ks, vs = _attention(q, k, v, log_decay, 4)
    os = _operand(grad_o, "grad_o", q, (*shape[:3], dv))
    _extras(shape, dv, device, lengths, initial_state, "initial_state")
    _extras(shape, dv, device, None, grad_state, "grad_state")
    d = _dims(kind, shape, dv, scale, reverse, qs, ks, vs, os)
    B, T, H, dk = shape
    qp, kp, vp, gp = q.data_ptr(), k.data_ptr(), v.data_ptr(), grad_o.data_ptr()
    _supported(B * T * H * dk * dv, shape, dv)
    new = lambda width: torch.empty((B, T, H, width), dtype=q.dtype, device=device)  # noqa: E731
    dq, dk_, dv_ = new(dk), new(dk), new(dv)
    ds = torch.empty((B, H, dk, dv), dtype=torch.float32, device=device) if want_initial_state else None
    _walk("linear_attention_backward", d, shape, dv, 1, qp, kp, vp, gp, device, ws, d, qp, kp, vp, log_decay.data_ptr(),
          _ptr(lengths), _ptr(initial_state), gp, _ptr(grad_state), dq.data_ptr(), dk_.data_ptr(), dv_.data_ptr(), _ptr(ds))
    return dq, dk_, dv_, ds


def _first_order(backward):
    """once_differentiable, whose wrapper is left out where nothing records the backward pass."""
    once = torch.autograd.function.once_differentiable(backward)

    def run(ctx, *grads):
        return once(ctx, *grads) if torch.is_grad_enabled() else backward(ctx, *grads)
    return run


class LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, initial_state, log_decay, lengths, scale, reverse, return_state):
        o, state = linear_attention_forward(q, k, v, log_decay, lengths, scale, initial_state, return_state, reverse)
        ctx.save_for_backward(q, k, v, initial_state, log_decay, lengths)
        ctx.how = (scale, reverse)
        ctx.set_materialize_grads(False)
        return (o, state) if return_state else o

    @staticmethod
    @_first_order
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
    _no_tangents((log_decay,))
    _constant(log_decay)
    return _differentiable(LinearAttention, (q, k, v, initial_state), (q, k, v, initial_state, log_decay, lengths,
                                                                       scale, reverse, return_state),
                           lambda: _drop(linear_attention_forward(q, k, v, log_decay, lengths, scale, initial_state,
                                                                  return_state, reverse), return_state))


def _drop(pair, both):
    return pair if both else pair[0]


def _no_tangents(inputs):
    """Refuses forward-mode derivatives: the library's calls would drop the tangents without a word."""
    if forward_ad._current_level >= 0 and any(isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None
                                              for t in inputs):
        raise NotImplementedError("linear attention and group norm have no forward-mode derivative")


def _differentiable(function, inputs, args, plain):
    """function.apply where a gradient may be asked for, else the call alone."""
    _no_tangents(inputs)
    if torch.is_grad_enabled() and any(t is not None and t.requires_grad for t in inputs):
        return function.apply(*args)
    return plain()


def linear_attention_step(q, k, v, log_decay, state, scale=None):
    """One position: state [B,H,dk,dv] float32 becomes lam state + k v^T in place; returns
    o [B,H,dv] = scale q state.  q, k [B,H,dk], v [B,H,dv].  No gradient is recorded."""
    _no_tangents((q, k, v, log_decay, state))
    device, kind, (B, H, dk), dv, qs, ks, vs = _attention(q, k, v, log_decay, 3)
    _want(state, "state", torch.float32, (B, H, dk, dv), device)
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad or state.requires_grad):
        raise ValueError("linear_attention_step records no gradient: use linear_attention, or torch.no_grad()")
    o = torch.empty((B, H, dv), dtype=q.dtype, device=device)
    d = _lib.ATTENTION_DIMS.pack(B, 1, H, dk, dv, kind, 0, dk ** -0.5 if scale is None else scale, qs[0], 0, qs[1], ks[0],
                                 0, ks[1], vs[0], 0, vs[1], H * dv, 0, dv)
    _call("linear_attention_step", device, d, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(),
          state.data_ptr(), o.data_ptr())
    torch.autograd.graph.increment_version(state)   # autograd refuses a graph that saved it
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
    if not isinstance(groups, int) or groups < 1 or C % groups:
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
    shape = (N, x.numel() // (N * C), C, groups)
    return shape, _lib.NORM_DIMS.pack(*shape, _TYPES[x.dtype], _TYPES[wtype], ACTIVATIONS[activation], eps)


def group_norm_workspace_bytes(x, groups, backward=False) -> int:
    """Bytes of workspace of a call with rows like x [N,...,C]."""
    return _norm_ws(*_norm_dims(x, groups, None, None, None, 1e-5, "none"), backward)


def _norm_ws(shape, dims, backward):
    n = _lib.load().semicrf_group_norm_workspace_bytes(dims, 1 if backward else 0)
    if n == 0:
        raise ValueError(f"unsupported arguments: rows, positions, channels, groups {shape}, or eps")
    return n


def group_norm_forward(x, groups, weight=None, bias=None, lengths=None, eps=1e-5, activation="none", ws=None):
    """(y like x, stats [N,groups,2] float32: mean and 1/std of the valid positions)."""
    shape, d = _norm_dims(x, groups, weight, bias, lengths, eps, activation)
    return _norm_forward(x, weight, bias, lengths, shape, d, ws)


def _norm_forward(x, weight, bias, lengths, shape, d, ws=None):
    device = x.device
    ws = _workspace(ws, _norm_ws(shape, d, False), device)
    y = torch.empty_like(x)
    stats = torch.empty((shape[0], shape[3], 2), dtype=torch.float32, device=device)
    _call("group_norm", device, d, x.data_ptr(), _ptr(weight), _ptr(bias), _ptr(lengths), y.data_ptr(),
          stats.data_ptr(), ws.data_ptr(), ws.numel())
    return y, stats


def _norm_alone(x, weight, bias, lengths, shape, d):
    """y, with the statistics behind the workspace (whose size is a multiple of 256)."""
    need = _norm_ws(shape, d, False)
    ws = torch.empty(need + 8 * shape[0] * shape[3], dtype=torch.uint8, device=x.device)
    y = torch.empty_like(x)
    at = ws.data_ptr()
    _call("group_norm", x.device, d, x.data_ptr(), _ptr(weight), _ptr(bias), _ptr(lengths), y.data_ptr(), at + need, at,
          need)
    return y


def group_norm_backward(dy, x, stats, groups, weight=None, bias=None, lengths=None, eps=1e-5, activation="none",
                        want_params=True, ws=None):
    """(dx like x, dweight [C] float32, dbias [C] float32); the last two None without want_params."""
    shape, d = _norm_dims(x, groups, weight, bias, lengths, eps, activation)
    _want(dy, "dy", x.dtype, x.shape, x.device)
    _want(stats, "stats", torch.float32, (shape[0], groups, 2), x.device)
    return _norm_backward(dy, x, stats, weight, bias, lengths, shape, d, want_params, ws)


def _norm_backward(dy, x, stats, weight, bias, lengths, shape, d, want_params, ws=None):
    device = x.device
    ws = _workspace(ws, _norm_ws(shape, d, True), device)
    dx = torch.empty_like(x)
    dw = db = None
    if want_params:
        dw = torch.empty(shape[2], dtype=torch.float32, device=device)
        db = torch.empty(shape[2], dtype=torch.float32, device=device)
    _call("group_norm_backward", device, d, dy.data_ptr(), x.data_ptr(), _ptr(weight), _ptr(bias), _ptr(lengths),
          stats.data_ptr(), dx.data_ptr(), _ptr(dw), _ptr(db), ws.data_ptr(), ws.numel())
    return dx, dw, db


class GroupNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, groups, lengths, eps, activation):
        ctx.shape, ctx.dims = _norm_dims(x, groups, weight, bias, lengths, eps, activation)
        y, stats = _norm_forward(x, weight, bias, lengths, ctx.shape, ctx.dims)
        ctx.save_for_backward(x, weight, bias, lengths, stats)
        return y

    @staticmethod
    @_first_order
    def backward(ctx, dy):
        x, weight, bias, lengths, stats = ctx.saved_tensors
        _, want_w, want_b = ctx.needs_input_grad[:3]
        if not dy.is_contiguous():
            dy = dy.contiguous()
        dx, dw, db = _norm_backward(dy, x, stats, weight, bias, lengths, ctx.shape, ctx.dims, want_w or want_b)
        if want_w and weight.dtype != torch.float32:
            dw = dw.to(weight.dtype)
        if want_b and bias.dtype != torch.float32:
            db = db.to(bias.dtype)
        return dx, dw if want_w else None, db if want_b else None, None, None, None, None


def group_norm(x, groups, weight=None, bias=None, lengths=None, eps=1e-5, activation="none"):
    """act((x - mean) / std * weight + bias) of x [N,...,C], with the statistics of each n and
    each of the `groups` groups of channels over all positions (over the first lengths[n] of
    x [N,S,C], zero behind them); activation "none", "silu" or "gelu".  Differentiable with
    respect to x, weight and bias."""
    return _differentiable(GroupNorm, (x, weight, bias), (x, weight, bias, groups, lengths, eps, activation),
                           lambda: _norm_alone(x, weight, bias, lengths,
                                               *_norm_dims(x, groups, weight, bias, lengths, eps, activation)))
