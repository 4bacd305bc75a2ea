"""AdamW over many tensors in one launch, with states in 32 or 8 bits: what turns the
gradients of the loss (dA, dD in float64 as the library returns them, or any of the
floating types) into new parameters.

    m, v, ms, vs = sc.new_adamw_state(params, bits=8)        # ms, vs None for 32 bits
    sc.adamw_step(params, grads, m, v, step, lr=1e-3, exp_avg_scale=ms, exp_avg_sq_scale=vs)

Everything is updated in place on the current CUDA stream.  In 8 bits a moment moves
only when an update passes half of its code's spacing (1/16 of its value at most), so
beta2 near 1 makes the second moment follow slowly growing or shrinking gradients in
steps; 32 bits are the exact form.  Where a moment of a block of 256 values is not finite, or
passes float32, the whole block's moments read as NaN, and its parameters are NaN after the
next step: gradients that may overflow are to be checked before the call.
"""
from __future__ import annotations

import array
import ctypes
import itertools
import operator

import torch

from . import _lib
from .encoder import _call

BLOCK = 256   # values that share a scale
_PARAMS = frozenset((torch.float32, torch.bfloat16, torch.float16))
_GRADS = _PARAMS | {torch.float64}
_SINGLE, _CODES = frozenset((torch.float32,)), frozenset((torch.uint8,))
_dtype, _shape = operator.attrgetter("dtype"), operator.attrgetter("shape")
_TYPES = {torch.float32: _lib.F32, torch.bfloat16: _lib.BF16, torch.float16: _lib.F16, torch.float64: _lib.F64}


def new_adamw_state(params, bits=32):
    """(exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale): zero states for `params`; the
    scales are None for 32 bits."""
    if bits == 32:
        return ([torch.zeros(p.shape, dtype=torch.float32, device=p.device) for p in params],
                [torch.zeros(p.shape, dtype=torch.float32, device=p.device) for p in params], None, None)
    if bits != 8:
        raise ValueError(f"bits must be 32 or 8, got {bits}")
    code = lambda p: torch.zeros(p.shape, dtype=torch.uint8, device=p.device)  # noqa: E731
    scale = lambda p: torch.zeros(-(-p.numel() // BLOCK), dtype=torch.float32, device=p.device)  # noqa: E731
    return [code(p) for p in params], [code(p) for p in params], [scale(p) for p in params], [scale(p) for p in params]


def _same_length(lists):
    n = len(lists[0][1])
    for name, ts in lists:
        if ts is not None and len(ts) != n:
            raise ValueError(f"{n} params, but {len(ts)} of {name}")


def _check(ts, name, sizes, dtypes, device):
    """Types, sizes, device and layout of a list's tensors: all together, then one by one for the error."""
    if (set(map(_dtype, ts)) <= dtypes and list(map(torch.Tensor.numel, ts)) == sizes
            and set(map(torch.Tensor.get_device, ts)) <= {device.index} and all(map(torch.Tensor.is_contiguous, ts))):
        return
    for t, n in zip(ts, sizes):
        if t.dtype in dtypes and t.numel() == n and t.device == device and t.is_contiguous():
            continue
        if t.dtype not in dtypes:
            raise TypeError(f"{name} has type {t.dtype}, expected {' or '.join(sorted(map(str, dtypes)))}")
        if t.numel() != n:
            raise ValueError(f"{name} has a tensor of {t.numel()} values, expected {n}")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")
        raise ValueError(f"{name} must be contiguous")


def _pointers(ts, n):
    return [0] * n if ts is None else list(map(torch.Tensor.data_ptr, ts))


def _table(params, grads, m, v, ms, vs, sizes):
    """The library's array of semicrf_adamw_tensor, one of eight 64-bit words each."""
    n = len(params)
    kinds = [_TYPES[p.dtype] for p in params]
    if grads is not None:
        kinds = [k | _TYPES[g.dtype] << 32 for k, g in zip(kinds, grads)]
    rows = zip(_pointers(params, n), _pointers(grads, n), _pointers(m, n), _pointers(v, n), _pointers(ms, n),
               _pointers(vs, n), sizes, kinds)
    return array.array("q", list(itertools.chain.from_iterable(rows)))


def _refuse_overlaps(written, grads):
    """Says which tensors of a refused call overlap, if any do."""
    span = lambda t: (t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())  # noqa: E731
    spans = sorted((*span(t), name) for name, ts in [*written, ("grads", grads)] for t in ts or [] if t.numel())
    end, last, wrote, writer = 0, None, 0, None   # of all so far, of those that are written
    for a, b, name in spans:
        if a < (wrote if name == "grads" else end):
            raise ValueError(f"the same tensor is given twice, or one overlaps another: {name} and {writer if name == 'grads' else last}")
        if b > end:
            end, last = b, name
        if name != "grads" and b > wrote:
            wrote, writer = b, name


def _scalar(x, name, dtype, device):
    if x.dtype != dtype or x.numel() != 1 or x.device != device:
        raise TypeError(f"{name} must be a number or one {dtype} value on {device}")
    return x.data_ptr()


def adamw_step(params, grads, exp_avg, exp_avg_sq, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
               grad_scale=1.0, exp_avg_scale=None, exp_avg_sq_scale=None):
    """One step over lists of tensors, in place; `step` counts from 1.

    params: float32, bfloat16 or float16; grads: those or float64, of the params' shapes
    (None: the parameter had no part in the loss and stays as it is, its states too);
    exp_avg, exp_avg_sq: float32, or uint8 with the lists exp_avg_scale and
    exp_avg_sq_scale (new_adamw_state).  step and lr may be CUDA scalars (int64 and
    float32), which the kernel reads: a captured step then follows them.
    """
    eight = exp_avg_scale is not None
    if eight != (exp_avg_sq_scale is not None):
        raise ValueError("exp_avg_scale and exp_avg_sq_scale come together")
    _same_length([("params", params), ("grads", grads), ("exp_avg", exp_avg), ("exp_avg_sq", exp_avg_sq),
                  ("exp_avg_scale", exp_avg_scale), ("exp_avg_sq_scale", exp_avg_sq_scale)])
    if any(g is None for g in grads):
        at = [i for i, g in enumerate(grads) if g is not None]
        params, grads, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale = (
            ts and [ts[i] for i in at] for ts in (params, grads, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale))
    if not params:
        return
    device = params[0].device
    if not params[0].is_cuda:
        raise TypeError("params must be CUDA tensors")
    kind = _CODES if eight else _SINGLE
    sizes = list(map(torch.Tensor.numel, params))
    _check(params, "params", sizes, _PARAMS, device)
    _check(grads, "grads", sizes, _GRADS, device)
    if list(map(_shape, grads)) != list(map(_shape, params)):
        p, g = next((p, g) for p, g in zip(params, grads) if g.shape != p.shape)
        raise ValueError(f"a gradient of shape {tuple(g.shape)} for a tensor of shape {tuple(p.shape)}")
    _check(exp_avg, "exp_avg", sizes, kind, device)
    _check(exp_avg_sq, "exp_avg_sq", sizes, kind, device)
    if eight:
        blocks = [-(-n // BLOCK) for n in sizes]
        _check(exp_avg_scale, "exp_avg_scale", blocks, _SINGLE, device)
        _check(exp_avg_sq_scale, "exp_avg_sq_scale", blocks, _SINGLE, device)
    c = _lib.AdamWConfig(0.0, betas[0], betas[1], eps, weight_decay, grad_scale, 0)
    if isinstance(step, torch.Tensor):
        c.step_ptr = _scalar(step, "step", torch.int64, device)
    else:
        c.step = step
    if isinstance(lr, torch.Tensor):
        c.lr_ptr = _scalar(lr, "lr", torch.float32, device)
    else:
        c.lr = lr
    words = _table(params, grads, exp_avg, exp_avg_sq, exp_avg_scale, exp_avg_sq_scale, sizes)
    try:
        _call("adamw", device, words.buffer_info()[0], len(params), ctypes.byref(c))
    except _lib.SemiCRFError:
        _refuse_overlaps([("params", params), ("exp_avg", exp_avg), ("exp_avg_sq", exp_avg_sq),
                          ("exp_avg_scale", exp_avg_scale), ("exp_avg_sq_scale", exp_avg_sq_scale)], grads)
        raise
    # autograd refuses a graph that saved what was just overwritten
    torch.autograd.graph.increment_version([*params, *exp_avg, *exp_avg_sq, *(exp_avg_scale or ()),
                                            *(exp_avg_sq_scale or ())])


def adamw_state_values(codes, scales, which):
    """The float32 values that 8-bit states stand for; which: "exp_avg" or "exp_avg_sq"."""
    if which not in ("exp_avg", "exp_avg_sq"):
        raise ValueError(f"which must be exp_avg or exp_avg_sq, got {which!r}")
    _same_length([("codes", codes), ("scales", scales)])
    if not codes:
        return []
    device = codes[0].device
    if not codes[0].is_cuda:
        raise TypeError("codes must be CUDA tensors")
    sizes = list(map(torch.Tensor.numel, codes))
    _check(codes, "codes", sizes, _CODES, device)
    _check(scales, "scales", [-(-n // BLOCK) for n in sizes], _SINGLE, device)
    # one allocation, each tensor at a multiple of 256 bytes
    starts = list(itertools.accumulate([n + 63 & -64 for n in sizes], initial=0))
    flat = torch.empty(starts[-1], dtype=torch.float32, device=device)
    out = [flat.as_strided(c.shape, c.stride(), at) for c, at in zip(codes, starts)]
    second = which == "exp_avg_sq"
    words = _table(out, None, None if second else codes, codes if second else None, None if second else scales,
                   scales if second else None, sizes)
    _call("adamw_state_values", device, words.buffer_info()[0], len(out), int(second))
    return out
