"""Norms around a block on torch tensors: ``norm`` and ``add_norm``.

    norm(x, weight, bias)       N(x), before a block
    add_norm(x, h, gate, ...)   r = scale x + gate * N_post(h), behind a block with its
                                gate and the residual stream's scale, and N(r), before
                                the next, in one pass

    N(v) = (v - mean) / sqrt(mean((v - mean)^2) + eps) * weight + bias

per row, with the mean for kind "layer" and without it for "rms".  x and h are M x D,
row-major, float32, bfloat16 or float16, one type per call.  Weights, biases and
gates are of that type or all float32, and have D elements, or G x D: a row for each
of G sequences of M / G rows (conditioned blocks).

Everything is float32 and rounded once.  With gradients enabled and an input that
requires one the operators are differentiable (once); ``norm_backward`` and
``add_norm_backward`` are those passes by themselves.  Streams, captured graphs and
what is refused are as in ``linear``.
"""
from __future__ import annotations

import struct

import torch
from torch.autograd.function import once_differentiable

from .fused import (DTYPES, _call, _launch, _matrix, _no_capture, _on, _recorded_elsewhere, _rows,
                    _wants_grad, _written)

# tra_norm_kind
KINDS = {"none": 0, "rms": 1, "layer": 2}

# tra_norm_args and tra_norm_grad_args, field by field
_ARGS = struct.Struct("@4i3q2fPqPq5P5qPqPq")
_GRAD_ARGS = struct.Struct("@4i3q2fPqPq5P5qPqPqPqPq5PPQ")

_VECTORS = ("weight", "bias", "gate", "post_weight", "post_bias")


def _kind(kind, name, least=0) -> int:
    try:
        code = KINDS[kind]
    except (KeyError, TypeError):
        code = -1
    if code < least:
        known = [k for k, c in KINDS.items() if c >= least]
        raise ValueError(f"{name} must be one of {', '.join(known)}; got {kind!r}")
    return code


def _vectors(vectors, x, M, D):
    """Checks the vectors; returns (type, groups, addresses, strides of their rows)."""
    device, own = x.device, x.dtype
    dtype, groups = None, 1
    at, ld = [0] * 5, [0] * 5
    for i, v in enumerate(vectors):
        if v is None:
            continue
        if not isinstance(v, torch.Tensor):
            raise TypeError(f"{_VECTORS[i]} must be a torch.Tensor")
        if v.dtype is not dtype:
            if dtype is not None:
                raise TypeError("weights, biases and gates must be of one type")
            dtype = v.dtype
            if dtype is not own and dtype is not torch.float32:
                raise TypeError(f"{_VECTORS[i]} must be {own} or float32")
        if v.device != device:
            raise TypeError(f"{_VECTORS[i]} must be on {device}")
        shape = v.shape
        n = len(shape)
        if n not in (1, 2) or shape[-1] != D or (n == 2 and shape[0] < 1):
            raise ValueError(f"{_VECTORS[i]} must have {D} elements, or a row of them per sequence")
        if not v.is_contiguous() and D > 1 and v.stride(-1) != 1:
            raise ValueError(f"{_VECTORS[i]} must have contiguous rows")
        if n == 2 and shape[0] > 1:
            if M % shape[0] != 0 or groups not in (1, shape[0]):
                raise ValueError(f"{_VECTORS[i]} has {shape[0]} rows: not one for each of some "
                                 f"equal parts of {M} rows, or not as many as another vector's")
            if v.stride(0) < max(1, D):
                raise ValueError(f"{_VECTORS[i]} must be row-major")
            groups = shape[0]
            ld[i] = v.stride(0)
        at[i] = v.data_ptr()
    return DTYPES[own if dtype is None else dtype], groups, at, ld


def _number(v, name) -> float:
    if type(v) is float:
        return v
    if isinstance(v, torch.Tensor):
        raise TypeError(f"{name} must be a number")
    return float(v)


def _given(t, name, x):
    """Checks an M x D tensor beside x; returns (address, leading dimension)."""
    ld = _matrix(t, name, x)
    if t.shape != x.shape:
        raise ValueError(f"{name} must be {x.shape[0]} x {x.shape[1]}")
    return t.data_ptr(), ld


def _fields(x, h, vectors, kind, post, scale, eps):
    """The arguments that both directions begin with."""
    ldx = _matrix(x, "x")
    M, D = x.shape
    H, ldh = (0, 0) if h is None else _given(h, "h", x)
    pdtype, groups, at, ld = _vectors(vectors, x, M, D)
    return (DTYPES[x.dtype], pdtype, kind, post, M, D, groups, scale, eps, x.data_ptr(), ldx, H,
            ldh, *at, *ld)


def _forward(x, h, vectors, kind, post, scale, eps, r=None, y=None):
    """One forward call; returns (r, y), None for what there is not."""
    fields = _fields(x, h, vectors, kind, post, scale, eps)
    M, D = fields[4], fields[5]
    R = Y = 0
    ldr = ldy = D
    if h is not None:
        if r is None:
            r = x.new_empty(M, D)
            R = r.data_ptr()
        else:
            R, ldr = _given(r, "r_out", x)
    if kind:
        if y is None:
            y = x.new_empty(M, D)
            Y = y.data_ptr()
        else:
            Y, ldy = _given(y, "out", x)
    _launch("tra_norm", _ARGS.pack(*fields, R, ldr, Y, ldy), x.device.index)
    return r, y


def _backward(dr, dy, x, h, vectors, kind, post, scale, eps, need_dx, need_dh, need):
    """One backward call; returns (dx, dh, [gradients of the vectors])."""
    fields = _fields(x, h, vectors, kind, post, scale, eps)
    R, ldr = (0, 0) if dr is None else _given(dr, "dr", x)
    Y, ldy = (0, 0) if dy is None else _given(dy, "dy", x)
    dx = dh = None
    X = H = 0
    if need_dx:
        dx = x.new_empty(x.shape)
        X = dx.data_ptr()
    if need_dh and h is not None:
        dh = x.new_empty(x.shape)
        H = dh.data_ptr()
    grads = [v.new_empty(v.shape) if v is not None and n else None
             for v, n in zip(vectors, need)]
    D = x.shape[1]
    _call("tra_norm_backward", _GRAD_ARGS,
          (*fields, R, ldr, Y, ldy, X, D, H, D, *(0 if g is None else g.data_ptr() for g in grads)),
          x.device)
    return dx, dh, grads


class _AddNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, h, weight, bias, gate, post_weight, post_bias, kind, post, scale, eps):
        vectors = (weight, bias, gate, post_weight, post_bias)
        r, y = _forward(x, h, vectors, kind, post, scale, eps)
        ctx.plan = (kind, post, scale, eps)
        ctx.save_for_backward(x, h, *vectors)
        ctx.set_materialize_grads(False)
        if h is None:
            return y
        return (r, y) if kind else r

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        _no_capture()
        kind, post, scale, eps = ctx.plan
        x, h, *vectors = ctx.saved_tensors
        dr, dy = (None, grads[0]) if h is None else grads if kind else (grads[0], None)
        if dr is None and dy is None:
            return (None,) * 11
        need = ctx.needs_input_grad
        dx, dh, dv = _backward(None if dr is None else _rows(dr), None if dy is None else _rows(dy),
                               x, h, vectors, kind, post, scale, eps, need[0], need[1], need[2:7])
        return (dx, dh, *dv, None, None, None, None)


def norm(x, weight=None, bias=None, kind="rms", eps=1e-6, out=None, stream=None):
    """N(x), as a new M x D tensor or in ``out``.

    ``weight`` and ``bias``, D elements or G x D, are optional.  ``kind``: rms or layer.
    ``stream`` as in ``linear``.  ``out`` is refused where autograd records the call.
    """
    _recorded_elsewhere(x, weight, bias, out)
    if stream is not None:
        return _on(stream, lambda: norm(x, weight, bias, kind, eps, out), x, weight, bias, out)
    code, eps = _kind(kind, "kind", 1), _number(eps, "eps")
    if _wants_grad(x, weight, bias, out):
        if out is not None:
            raise ValueError("out cannot be given where gradients are recorded")
        return _AddNorm.apply(x, None, weight, bias, None, None, None, code, 0, 1.0, eps)
    y = _forward(x, None, (weight, bias, None, None, None), code, 0, 1.0, eps, None, out)[1]
    if out is not None:
        _written(out)
    return y


def add_norm(x, h, gate=None, scale=1.0, post="none", post_weight=None, post_bias=None,
             kind="rms", weight=None, bias=None, eps=1e-6, r_out=None, out=None, stream=None):
    """(r, y): r = scale x + gate * N_post(h) and y = N(r), as new M x D tensors or in
    ``r_out`` and ``out``.

    x is the residual stream and h a block's output.  ``post`` and ``kind`` are none,
    rms or layer: with post "none" h is taken as it is, with kind "none" y is None.
    ``gate``, ``post_weight``, ``post_bias``, ``weight`` and ``bias``, D elements or G x D,
    are optional.  ``scale`` is a number.  ``r_out`` may be x itself.  y is taken from r
    before its rounding.  ``stream`` as in ``linear``.  ``r_out`` and ``out`` are refused
    where autograd records the call.
    """
    tensors = (x, h, gate, post_weight, post_bias, weight, bias, r_out, out)
    _recorded_elsewhere(*tensors)
    if stream is not None:
        return _on(stream, lambda: add_norm(x, h, gate, scale, post, post_weight, post_bias, kind,
                                            weight, bias, eps, r_out, out), *tensors)
    if not isinstance(h, torch.Tensor):
        raise TypeError("h must be a torch.Tensor")
    code, post_code = _kind(kind, "kind"), _kind(post, "post")
    scale, eps = _number(scale, "scale"), _number(eps, "eps")
    if not code and (weight is not None or bias is not None or out is not None):
        raise ValueError("weight, bias and out belong to y, which kind none leaves out")
    if not post_code and (post_weight is not None or post_bias is not None):
        raise ValueError("post_weight and post_bias belong to the norm that post none leaves out")
    if _wants_grad(*tensors):
        if r_out is not None or out is not None:
            raise ValueError("r_out and out cannot be given where gradients are recorded")
        got = _AddNorm.apply(x, h, weight, bias, gate, post_weight, post_bias, code, post_code,
                             scale, eps)
        return got if code else (got, None)
    r, y = _forward(x, h, (weight, bias, gate, post_weight, post_bias), code, post_code, scale,
                    eps, r_out, out)
    if r_out is not None or out is not None:
        _written(r_out, out)
    return r, y


def norm_backward(dy, x, weight=None, bias=None, kind="rms", eps=1e-6, need_dx=True,
                  need_dweight=True, need_dbias=True, stream=None):
    """(dx, dweight, dbias) of ``norm`` for dy, the gradient of its result; None for what is
    not there or not asked for.  ``bias`` gives its gradient's shape only.  ``stream`` as in
    ``linear``."""
    _recorded_elsewhere(dy, x, weight, bias)
    if stream is not None:
        return _on(stream, lambda: norm_backward(dy, x, weight, bias, kind, eps, need_dx,
                                                 need_dweight, need_dbias), dy, x, weight, bias)
    dx, _, grads = _backward(None, dy, x, None, (weight, bias, None, None, None),
                             _kind(kind, "kind", 1), 0, 1.0, _number(eps, "eps"), need_dx, False,
                             (need_dweight, need_dbias, False, False, False))
    return dx, grads[0], grads[1]


def add_norm_backward(dr, dy, x, h, gate=None, scale=1.0, post="none", post_weight=None,
                      post_bias=None, kind="rms", weight=None, bias=None, eps=1e-6, need_dx=True,
                      need_dh=True, need_vectors=True, stream=None):
    """(dx, dh, dgate, dpost_weight, dpost_bias, dweight, dbias) of ``add_norm`` for dr and
    dy, the gradients of its results (either may be None, for zero); None for what is not
    there or not asked for.  ``bias`` gives its gradient's shape only.  ``stream`` as in
    ``linear``."""
    tensors = (dr, dy, x, h, gate, post_weight, post_bias, weight, bias)
    _recorded_elsewhere(*tensors)
    if stream is not None:
        return _on(stream, lambda: add_norm_backward(dr, dy, x, h, gate, scale, post, post_weight,
                                                     post_bias, kind, weight, bias, eps, need_dx,
                                                     need_dh, need_vectors), *tensors)
    if not isinstance(h, torch.Tensor):
        raise TypeError("h must be a torch.Tensor")
    code, post_code = _kind(kind, "kind"), _kind(post, "post")
    if not code and (dy is not None or weight is not None or bias is not None):
        raise ValueError("dy, weight and bias belong to y, which kind none leaves out")
    if not post_code and (post_weight is not None or post_bias is not None):
        raise ValueError("post_weight and post_bias belong to the norm that post none leaves out")
    dx, dh, (dw, db, dg, dpw, dpb) = _backward(
        dr, dy, x, h, (weight, bias, gate, post_weight, post_bias), code, post_code,
        _number(scale, "scale"), _number(eps, "eps"), need_dx, need_dh, (need_vectors,) * 5)
    return dx, dh, dg, dpw, dpb, dw, db
