"""Fused linear operators on torch tensors: ``linear`` and ``gated_linear``.

    linear(x, w, bias, act, residual)   act(x w + bias) + residual
    gated_linear(x, w_gate, w_up, act)  act(x w_gate) * (x w_up)

Like ``matmul`` these check the tensors, pass their device pointers and torch's
current stream to the library, and raise TraError on a non-OK status; scratch
comes from torch's allocator, so calls may be captured into a graph.

``stream`` is a torch.cuda.Stream, or None for torch's current stream.  A call
runs behind what is on that stream already, as under ``torch.cuda.stream``: it
waits for no other stream, so the caller orders it behind whatever still writes its
inputs elsewhere, and orders whatever reads its results behind it.  Memory needs no
care: tensors may be dropped, and reused by the allocator, once the call returns.

With gradients enabled and an input that requires one they are differentiable
(once): the backward pass runs in the library too.  ``linear_backward`` and
``gated_linear_backward`` are those passes by themselves, for callers that
keep their own order of work (a pipeline, a captured training step: autograd
itself is refused inside a capture).  Forward-mode derivatives and torch.jit.trace
are refused.

x is M x K, the weights K x N: row-major, or the transposed view of a row-major
N x K tensor (``w.t()`` of a torch.nn.Linear weight).  float32, bfloat16 or
float16, one type per call.  Every element is summed in float32 and rounded
once; the gradients of x and of the weights are sums over dz, the gradient of
the pre-activations, which is itself rounded to the type (in float16 under a
scale of its own, so that its range does not limit them).
"""
from __future__ import annotations

import ctypes
import struct

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import TRA_ERR_INVALID_ARG, TRA_OK, TraError, _row_major_ld, load

# tra_act
ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "sigmoid": 5}
# tra_dtype
DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

# tra_linear_args and tra_linear_grad_args, field by field
_ARGS = struct.Struct("@4i3qPqPPqPPqPqPqPQ")
_GRAD_ARGS = struct.Struct("@4i3qPqPqPqPPqPqPPqPPQ")


def _act(act) -> int:
    try:
        return ACTS[act]
    except (KeyError, TypeError):
        raise ValueError(f"act must be one of {', '.join(ACTS)}; got {act!r}") from None


def _matrix(t, name, like=None, dtype=None) -> int:
    """Checks a row-major 2-D tensor; returns its leading dimension."""
    if (like is not None and isinstance(t, torch.Tensor) and t.dim() == 2
            and t.dtype is (dtype or like.dtype) and t.device == like.device):
        rows, cols = t.shape
        s0, s1 = t.stride()
        return s0 if s1 == 1 and s0 >= cols > 0 else _row_major_ld((rows, cols), (s0, s1), name)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2 or not t.is_cuda:
        raise TypeError(f"{name} must be a 2-D tensor on a GPU")
    if like is None:
        if t.dtype not in DTYPES:
            raise TypeError(f"{name} must be float32, bfloat16 or float16")
    else:
        if t.dtype != (dtype or like.dtype):
            raise TypeError(f"{name} must be {dtype or like.dtype}, not {t.dtype}")
        if t.device != like.device:
            raise ValueError(f"{name} must be on {like.device}")
    rows, cols = t.shape
    s0, s1 = t.stride()
    if s1 == 1 and s0 >= cols > 0:
        return s0
    return _row_major_ld((rows, cols), (s0, s1), name)


def _weight(w, name, x):
    """Checks a weight; returns (w_trans, leading dimension)."""
    if not isinstance(w, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if w.dim() != 2 or not w.is_cuda:
        raise TypeError(f"{name} must be a 2-D tensor on a GPU")
    if w.dtype != x.dtype:
        raise TypeError(f"{name} must be {x.dtype}, not {w.dtype}")
    if w.device != x.device:
        raise ValueError(f"{name} must be on {x.device}")
    K, N = w.shape
    if K != x.shape[1]:
        raise ValueError(f"inner dimensions differ: x is {tuple(x.shape)}, {name} is {(K, N)}")
    s0, s1 = w.stride()
    if s0 == 1 and (s1 >= K if N > 1 else K > 1):
        if s1 != 1 or K > 1:
            return 1, s1 if N > 1 else K
    try:
        return 0, _row_major_ld((K, N), (s0, s1), name)
    except ValueError:
        if K == 1 and s1 >= 1:
            return 1, s1
        raise ValueError(f"{name} must be row-major or the transposed view of a row-major "
                         "tensor") from None


def _vector(b, name, x, N):
    if not isinstance(b, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if b.dtype != x.dtype or b.dim() != 1 or b.device != x.device:
        raise TypeError(f"{name} must be a 1-D {x.dtype} tensor on {x.device}")
    if b.shape[0] != N or (N > 1 and b.stride(0) != 1):
        raise ValueError(f"{name} must be {N} contiguous elements")


# Workspace bytes of the calls seen so far, by name, type, layout and sizes: what
# to allocate before a call.  Alignment and which gradients are asked for count
# too, so a call may need more; the library then refuses it, before anything is
# enqueued, and says how much.
_seen: dict = {}


def _call(name, fmt, fields, device, count=7):
    """Takes a workspace from torch's allocator, packs the arguments and makes
    the call.  Of the fields, the first `count` are types, layout and sizes."""
    index = device.index
    if torch.cuda.current_device() != index:
        with torch.cuda.device(device):
            return _call(name, fmt, fields, device, count)
    lib = load()
    stream = torch._C._cuda_getCurrentRawStream(index)
    call = getattr(lib, name)
    key = (name, fields[:count])
    need = _seen.get(key, 0)
    # torch's blocks are 512-byte aligned, and 256 are wanted
    ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    st = call(fmt.pack(*fields, ws.data_ptr() if need else 0, need), stream)
    if st == TRA_ERR_INVALID_ARG:
        size = ctypes.c_size_t(0)
        ok = getattr(lib, name + "_workspace_size")(fmt.pack(*fields, 0, 0), ctypes.byref(size))
        if ok == TRA_OK and size.value > need:
            if len(_seen) >= 4096:
                _seen.clear()
            need = _seen[key] = size.value
            ws = torch.empty(need, dtype=torch.uint8, device=device)
            st = call(fmt.pack(*fields, ws.data_ptr(), need), stream)
    if st != TRA_OK:
        raise TraError(st, name)


def _launch(name, packed, index):
    """A call that takes no workspace, on torch's current stream of device `index`."""
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            return _launch(name, packed, index)
    st = getattr(load(), name)(packed, torch._C._cuda_getCurrentRawStream(index))
    if st != TRA_OK:
        raise TraError(st, name)


_KEEP = object()


def _forward(x, w, w2, bias, residual, act, out, z):
    """One forward call; z (_KEEP: allocate it) keeps the pre-activations."""
    gated = w2 is not None
    code = _act(act)
    ldx = _matrix(x, "x")
    M, K = x.shape
    trans, ldw = _weight(w, "w_gate" if gated else "w", x)
    N = w.shape[1]
    if gated:
        if _weight(w2, "w_up", x) != (trans, ldw) or w2.shape != w.shape:
            raise ValueError("w_gate and w_up must have the same shape and strides")
    if bias is not None:
        _vector(bias, "bias", x, N)
    ldr = 0
    if residual is not None:
        ldr = _matrix(residual, "residual", x)
        if residual.shape[0] != M or residual.shape[1] != N:
            raise ValueError(f"residual must be {M} x {N}")
    if out is None:
        out = x.new_empty(M, N)
        ldy = N
    else:
        ldy = _matrix(out, "out", x)
        if out.shape[0] != M or out.shape[1] != N:
            raise ValueError(f"out must be {M} x {N}")
    ldz = 0
    if z is not None:
        width = 2 * N if gated else N
        if z is _KEEP:
            z = torch.empty((M, width), dtype=torch.float32, device=x.device)
        ldz = _matrix(z, "z", x, torch.float32)
        if z.shape[0] != M or z.shape[1] != width:
            raise ValueError(f"z must be {M} x {width}")
    fields = (DTYPES[x.dtype], code, trans, int(gated), M, N, K, x.data_ptr(), ldx, w.data_ptr(),
              w2.data_ptr() if gated else 0, ldw, 0 if bias is None else bias.data_ptr(),
              0 if residual is None else residual.data_ptr(), ldr, out.data_ptr(), ldy,
              0 if z is None else z.data_ptr(), ldz)
    _call("tra_linear", _ARGS, fields, x.device)
    return out, z


def _backward(dy, x, w, w2, z, act, need_dx, need_dw, need_bias):
    """Checks the tensors of a backward call and makes it."""
    gated = w2 is not None
    code = _act(act)
    ldx = _matrix(x, "x")
    lddy = _matrix(dy, "dy", x)
    trans, ldw = _weight(w, "w_gate" if gated else "w", x)
    M, N = x.shape[0], w.shape[1]
    if gated and (_weight(w2, "w_up", x) != (trans, ldw) or w2.shape != w.shape):
        raise ValueError("w_gate and w_up must have the same shape and strides")
    if dy.shape[0] != M or dy.shape[1] != N:
        raise ValueError(f"dy must be {M} x {N}")
    ldz = 0
    if gated or code != 0:
        if z is None:
            raise ValueError("z, the kept pre-activations, is needed")
        width = 2 * N if gated else N
        ldz = _matrix(z, "z", x, torch.float32)
        if z.shape[0] != M or z.shape[1] != width:
            raise ValueError(f"z must be {M} x {width}")
    else:
        z = None
    K = x.shape[1]
    dx = dw = dw2 = db = None
    pdx = pdw = pdw2 = pdb = 0
    if need_dx:
        dx = x.new_empty(M, K)
        pdx = dx.data_ptr()
    if need_dw:
        dw = x.new_empty(N, K) if trans else x.new_empty(K, N)
        pdw = dw.data_ptr()
        if w2 is not None:
            dw2 = torch.empty_like(dw)
            pdw2 = dw2.data_ptr()
    if need_bias:
        db = x.new_empty(N)
        pdb = db.data_ptr()
    fields = (DTYPES[x.dtype], code, trans, 0 if w2 is None else 1, M, N, K, dy.data_ptr(), lddy,
              0 if z is None else z.data_ptr(), ldz, x.data_ptr(), ldx, w.data_ptr(),
              0 if w2 is None else w2.data_ptr(), ldw, pdx, K, pdw, pdw2, K if trans else N, pdb)
    _call("tra_linear_backward", _GRAD_ARGS, fields, x.device)
    if trans:
        dw, dw2 = (None if t is None else t.t() for t in (dw, dw2))
    return dx, dw, dw2, db


def _rows(dy):
    """dy as the library takes it: autograd may pass an expanded or transposed one."""
    s0, s1 = dy.stride()
    return dy if s1 == 1 and s0 >= dy.shape[1] else dy.contiguous()


class _Linear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, residual, act):
        need = any(ctx.needs_input_grad[:3])
        y, z = _forward(x, w, None, bias, residual, act, None,
                        _KEEP if need and act != "none" else None)
        ctx.act = act
        ctx.save_for_backward(x, w, z)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        _no_capture()
        need_x, need_w, need_b, need_r, _ = ctx.needs_input_grad
        if not (need_x or need_w or need_b):
            return None, None, None, dy, None
        # (saved-tensor hooks may have changed the strides: all is checked again)
        x, w, z = ctx.saved_tensors
        dx, dw, _, db = _backward(_rows(dy), x, w, None, z, ctx.act, need_x, need_w, need_b)
        return dx, dw, db, dy if need_r else None, None


class _GatedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w_gate, w_up, act):
        h, z = _forward(x, w_gate, w_up, None, None, act, None, _KEEP)
        ctx.act = act
        ctx.save_for_backward(x, w_gate, w_up, z)
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        _no_capture()
        x, w_gate, w_up, z = ctx.saved_tensors
        need_x, need_g, need_u, _ = ctx.needs_input_grad
        dx, dg, du, _ = _backward(_rows(dh), x, w_gate, w_up, z, ctx.act, need_x,
                                  need_g or need_u, False)
        return dx, dg if need_g else None, du if need_u else None, None


def _wants_grad(*tensors) -> bool:
    if torch.is_grad_enabled():
        for t in tensors:
            if isinstance(t, torch.Tensor) and t.requires_grad:
                if t.is_cuda:
                    _no_capture()
                return True
    return False


_tracing = torch._C._is_tracing


def _recorded_elsewhere(*tensors):
    """Refuses what would lose the call without a word: forward-mode derivatives,
    which the operators do not have, and torch.jit.trace, which records torch's own
    operations only."""
    if forward_ad._current_level >= 0 and torch._C._is_fwd_grad_enabled():
        for t in tensors:
            if isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None:
                raise NotImplementedError("the fused operators have no forward-mode derivatives")
    if _tracing():
        raise RuntimeError("torch.jit.trace cannot record the fused operators")


def _on(stream, call, *tensors):
    """call() on a caller's stream, which is one of the tensors' device.

    The allocator is told that ``stream`` uses the tensors given, and that the
    caller's current stream uses the results, which are allocated on ``stream``:
    either may be dropped once the call has returned.
    """
    device = next((t.device for t in tensors if isinstance(t, torch.Tensor) and t.is_cuda),
                  stream.device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        result = call()
    if current != stream:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        for t in result if isinstance(result, tuple) else (result,):
            if t is not None:
                t.record_stream(current)
    return result


def _written(*tensors):
    """Tells autograd that these were written in place."""
    for t in tensors:
        if t is not None:
            torch.autograd.graph.increment_version(t)


def _no_capture():
    # Autograd's engine orders a leaf's gradient behind the stream that the leaf
    # was first used on.  Inside a capture, with an eager graph of the same leaf
    # alive, that stream is outside the capture, and the process ends.
    if torch.cuda.is_current_stream_capturing():
        raise RuntimeError("gradients cannot be recorded into a captured graph: capture the call "
                           "without gradients (a linear one with z=...) and the operator's "
                           "backward function, such as linear_backward")


def linear(x, w, bias=None, act="none", residual=None, out=None, z=None, stream=None):
    """act(x w + bias) + residual, as a new M x N tensor or in ``out``.

    ``bias`` (N elements) and ``residual`` (M x N; ``out`` may be the same
    tensor) are optional.  ``act``: none, relu, gelu, gelu_tanh, silu or
    sigmoid.  ``z``, if given, is a float32 M x N tensor that receives
    x w + bias for ``linear_backward``.  ``stream``, None for the current
    one, is not made to wait for others: inputs written elsewhere have to be done,
    or waited for by it.  ``out`` and ``z`` are refused where autograd records the
    call.
    """
    _recorded_elsewhere(x, w, bias, residual, out, z)
    if stream is not None:
        return _on(stream, lambda: linear(x, w, bias, act, residual, out, z), x, w, bias,
                   residual, out, z)
    if _wants_grad(x, w, bias, residual, out, z):
        if out is not None or z is not None:
            raise ValueError("out and z cannot be given where gradients are recorded")
        return _Linear.apply(x, w, bias, residual, act)
    y = _forward(x, w, None, bias, residual, act, out, z)[0]
    if out is not None or z is not None:
        _written(out, z)
    return y


def gated_linear(x, w_gate, w_up, act="silu", out=None, z=None, stream=None):
    """act(x w_gate) * (x w_up), as a new M x N tensor or in ``out``.

    The weights have the same shape and strides (two tensors, or the halves of
    a packed one).  ``z``, if given, is a float32 M x 2N tensor that receives
    [x w_gate | x w_up] for ``gated_linear_backward``.  Other arguments, and
    what is asked of the caller of ``stream``, as in ``linear``.
    """
    _recorded_elsewhere(x, w_gate, w_up, out, z)
    if stream is not None:
        return _on(stream, lambda: gated_linear(x, w_gate, w_up, act, out, z), x, w_gate, w_up,
                   out, z)
    if w_up is None:
        raise TypeError("w_up must be a torch.Tensor")
    if _wants_grad(x, w_gate, w_up, out, z):
        if out is not None or z is not None:
            raise ValueError("out and z cannot be given where gradients are recorded")
        return _GatedLinear.apply(x, w_gate, w_up, act)
    h = _forward(x, w_gate, w_up, None, None, act, out, z)[0]
    if out is not None or z is not None:
        _written(out, z)
    return h


def linear_backward(dy, x, w, z=None, act="none", need_dx=True, need_dw=True, need_dbias=False,
                    stream=None):
    """(dx, dw, dbias) of ``linear`` for dy, the gradient of its result (that
    of the residual is dy itself); None for each not asked for.  ``z`` is what
    ``linear`` kept, needed unless act is "none".  dw has w's layout.  ``stream``
    as in ``linear``."""
    _recorded_elsewhere(dy, x, w, z)
    if stream is not None:
        return _on(stream, lambda: linear_backward(dy, x, w, z, act, need_dx, need_dw, need_dbias),
                   dy, x, w, z)
    dx, dw, _, db = _backward(dy, x, w, None, z, act, need_dx, need_dw, need_dbias)
    return dx, dw, db


def gated_linear_backward(dh, x, w_gate, w_up, z, act="silu", need_dx=True, need_dw=True,
                          stream=None):
    """(dx, dw_gate, dw_up) of ``gated_linear`` for dh, the gradient of its
    result; ``z`` is what it kept.  None for what is not asked for.  ``stream`` as in
    ``linear``."""
    _recorded_elsewhere(dh, x, w_gate, w_up, z)
    if stream is not None:
        return _on(stream, lambda: gated_linear_backward(dh, x, w_gate, w_up, z, act, need_dx,
                                                         need_dw), dh, x, w_gate, w_up, z)
    if w_up is None:
        raise TypeError("w_up must be a torch.Tensor")
    dx, dg, du, _ = _backward(dh, x, w_gate, w_up, z, act, need_dx, need_dw, False)
    return dx, dg, du
