"""Matrices in 8-bit floating point with a scale for each block of 128, on torch tensors:
``quantize`` makes them and ``scaled_linear`` multiplies them.

    scaled_linear(x, w, x_scales, w_scales, bias, residual)      x w + bias + residual

A block is 128 consecutive elements along the axis that a product sums over, of one row
(activations, gradients) or of 128 rows (weights).  Its scale is float32 or, as the
matrix units of MI355X take it, float8_e8m0fnu, a power of two.  A matrix is a pair of
plain tensors: values (float8_e4m3fn or float8_e5m2, rows x columns filled up with zeros to
a multiple of 16) and scales (rows, or rows / 128 rounded up, x columns / 128 rounded up).

Serving: w is the transposed view of the values of an N x K weight that was quantized once,
w_scales that of its scales; x is a tensor, quantized in the call, or values with x_scales.
Training: x and w are tensors of one type; the call quantizes both (w in blocks of
128 x 128) and is differentiable (once).  Each product sums over quantized operands,
every one with blocks along that product's sum:

    y = Q(x) Q(w)        dx = Q(dy) Q(w)^T        dw = Q(x)^T Q(dy)  (blocks along the rows)

with the gradients passed on as if quantizing were the identity.

Sums of float32 results are float32.  bfloat16 and float16 results, gradients among them, come
from the matrix units' 8-bit instructions, which add 8 neighbouring products at a time, each
cut off 13 binary places below the largest one's exponent: about 1e-5 of a sum of normally
distributed products, well below the rounding to 16 bits, but more where large products cancel.
``dtype=torch.float32`` has none of that.

Streams, captured graphs and what is refused are as in ``linear``.
"""
from __future__ import annotations

import struct

import torch
from torch.autograd.function import once_differentiable

from . import _row_major_ld, fused
from .fused import (DTYPES, _launch, _matrix, _no_capture, _on, _recorded_elsewhere, _rows, _vector,
                    _wants_grad, _weight, _written)

# tra_fp8, tra_scale
FP8 = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}
SCALES = {torch.float32: 0, torch.float8_e8m0fnu: 1}
FORMS = ("rows", "columns", "both")
BLOCK = 128

# tra_quantize_args, field by field
_QUANTIZE = struct.Struct("@4i2qPqPqPqqPqPqq")
# tra_scaled_args
_SCALED = struct.Struct("@6i3qPqPqqPqPqqPPqPqPQ")
X_SCALED = -1


def _up(n, m):
    return -(-n // m)


def _code(table, key, name):
    try:
        return table[key]
    except (KeyError, TypeError):
        raise ValueError(f"{name} must be one of {', '.join(map(str, table))}; got {key!r}") from None


def _block_rows(block) -> int:
    if block in (1, (1, BLOCK)):
        return 1
    if block in (BLOCK, (BLOCK, BLOCK)):
        return BLOCK
    raise ValueError(f"block must be (1, 128) or (128, 128); got {block!r}")


def _empty(x, rows, cols, block_rows, dtype, scale_dtype):
    """An 8-bit matrix: values, scales and the scales' strides.  Scales of rows lie next
    to each other for one block of columns: a product reads them so."""
    values = x.new_empty(rows, _up(cols, 16) * 16, dtype=dtype)
    r, b = _up(rows, block_rows), _up(cols, BLOCK)
    stride = (1, max(1, r)) if block_rows == 1 else (max(1, b), 1)
    return values, x.new_empty_strided((r, b), stride, dtype=scale_dtype), *stride


def _quantize(x, block_rows, dtype, scale_dtype, rows, columns):
    """The forms asked for of a checked x: [values, scales] each."""
    ldx = _matrix(x, "x")
    M, K = x.shape
    fields, got = [], []
    for want, r, c in ((rows, M, K), (columns, K, M)):
        if not want:
            fields += [0, 0, 0, 0, 0]
            continue
        values, scales, ss_row, ss_block = _empty(x, r, c, block_rows, dtype, scale_dtype)
        fields += [values.data_ptr(), values.shape[1], scales.data_ptr(), ss_row, ss_block]
        got += [values, scales]
    _launch("tra_quantize", _QUANTIZE.pack(DTYPES[x.dtype], FP8[dtype], SCALES[scale_dtype],
                                           block_rows, M, K, x.data_ptr(), ldx, *fields),
            x.device.index)
    return got


def quantize(x, block=(1, 128), dtype=torch.float8_e4m3fn, scale_dtype=torch.float8_e8m0fnu,
             form="rows", stream=None):
    """(values, scales) of x, M x K row-major, float32, bfloat16 or float16.

    ``block``: (1, 128), a scale for each row, or (128, 128).  ``dtype``: float8_e4m3fn or
    float8_e5m2.  ``scale_dtype``: float8_e8m0fnu, the least power of two that fits a
    block's largest finite magnitude, or float32, that magnitude over the type's largest
    value; 1 for a block of zeros.  Values are rounded once, to nearest even.  NaN stays
    NaN; an infinity becomes NaN in float8_e4m3fn, which has none.

    ``form``: "rows", blocks along K; "columns", the transpose of x (K rows) with blocks
    along M; "both", as (values, scales, column values, column scales) from one pass.
    Values have K (M) rounded up to a multiple of 16 columns, zeros at the end.  Not
    differentiable: gradients stop here (``scaled_linear`` quantizes tensors by itself).
    ``stream`` as in ``linear``.
    """
    _recorded_elsewhere(x)
    if stream is not None:
        return _on(stream, lambda: quantize(x, block, dtype, scale_dtype, form), x)
    block_rows = _block_rows(block)
    _code(FP8, dtype, "dtype")
    _code(SCALES, scale_dtype, "scale_dtype")
    if form not in FORMS:
        raise ValueError(f"form must be one of {', '.join(FORMS)}; got {form!r}")
    return tuple(_quantize(x, block_rows, dtype, scale_dtype, form != "columns", form != "rows"))


# --- products ---------------------------------------------------------------------

def _values(t, name, rows, K, stride, device):
    """Checks 8-bit values, rows x K with these strides; returns their leading dimension."""
    if t.device != device or not t.is_cuda:
        raise TypeError(f"{name} must be on {device}")
    if K % 16 != 0:
        raise ValueError(f"rows of {name} must be a multiple of 16 long (zeros at the end, as "
                         "quantize leaves them)")
    s0, s1 = stride
    ld = s0 if s1 == 1 and s0 >= K > 0 else _row_major_ld((rows, K), stride, name)
    if K > 0 and ((ld % 16 != 0 and rows > 1) or t.data_ptr() % 16 != 0):
        raise ValueError(f"rows of {name} must start 16-byte aligned")
    return ld


def _scales(s, name, shape, stride, rows, cols, device):
    """Checks scales, of this shape and strides, of rows x cols values; returns (block rows,
    type, row's and block's strides)."""
    if s.dtype not in SCALES or s.device != device:
        raise TypeError(f"{name} must be a float32 or float8_e8m0fnu tensor on {device}")
    blocks = _up(cols, BLOCK)
    if shape[1] != blocks or shape[0] not in (rows, _up(rows, BLOCK)):
        raise ValueError(f"{name} must be of {rows} or {_up(rows, BLOCK)} rows by {blocks} blocks")
    # (of a single row, either is the same)
    block_rows = 1 if shape[0] == rows and rows > 1 else BLOCK
    ss_row, ss_block = stride
    if ss_row != 1 and ss_block != 1 and shape[0] > 1 and blocks > 1:
        raise ValueError(f"{name} must have contiguous rows or columns")
    return block_rows, SCALES[s.dtype], ss_row, ss_block


def _two_dim(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise TypeError(f"{name} must be a 2-D torch.Tensor")


def _product(x, x_scales, w, w_scales, bias, residual, dtype, out):
    """x w + bias + residual: w K x N, the transposed view of values, w_scales of theirs; x
    values with scales, or a tensor."""
    device = x.device
    if w.dtype not in FP8:
        raise TypeError("w must be 8-bit values")
    _two_dim(x, "x")
    _two_dim(w, "w")
    _two_dim(w_scales, "w_scales")
    K, N = w.shape
    ldw = _values(w, "w", N, K, w.stride()[::-1], device)
    block_rows, scale, sw_row, sw_block = _scales(w_scales, "w_scales", w_scales.shape[::-1],
                                                  w_scales.stride()[::-1], N, K, device)
    M, kx = x.shape
    if x_scales is None:
        ldx = _matrix(x, "x")
        if _up(kx, 16) * 16 != K:
            raise ValueError(f"inner dimensions differ: x has {kx} columns, w {K} rows")
        head = (DTYPES[x.dtype], 0)
        sx = (0, 0, 0)
    else:
        ldx = _values(x, "x", M, kx, x.stride(), device)
        if kx != K:
            raise ValueError(f"inner dimensions differ: x has {kx} columns, w {K} rows")
        _two_dim(x_scales, "x_scales")
        one, kind, sx_row, sx_block = _scales(x_scales, "x_scales", x_scales.shape,
                                              x_scales.stride(), M, K, device)
        if (one != 1 and M > 1) or kind != scale:
            raise ValueError("x_scales must have a row for each of x's, and w_scales' type")
        head = (X_SCALED, FP8[x.dtype])
        sx = (x_scales.data_ptr(), sx_row, sx_block)
    if scale == 0 and block_rows == 1:
        raise ValueError("float32 w_scales must be of blocks of 128 x 128")
    w_fp8 = FP8[w.dtype]
    if w_fp8 and (head[1] or scale == 0 or x_scales is None):
        raise ValueError("float8_e5m2 w goes with float8_e4m3fn x and float8_e8m0fnu scales only")
    B = R = 0
    ldr = ldy = N
    if out is None:
        out = x.new_empty(M, N, dtype=dtype)
    else:
        ldy = _matrix(out, "out", x, dtype)
        if out.shape[0] != M or out.shape[1] != N:
            raise ValueError(f"out must be {M} x {N}")
    if bias is not None:
        _vector(bias, "bias", out, N)
        B = bias.data_ptr()
    if residual is not None:
        ldr = _matrix(residual, "residual", out)
        if residual.shape[0] != M or residual.shape[1] != N:
            raise ValueError(f"residual must be {M} x {N}")
        R = residual.data_ptr()
    fields = (DTYPES[dtype], *head, w_fp8, scale, block_rows, M, N, kx, x.data_ptr(), ldx, *sx,
              w.data_ptr(), ldw, w_scales.data_ptr(), sw_row, sw_block, B, R, ldr, out.data_ptr(),
              ldy)
    fused._call("tra_scaled_linear", _SCALED, fields, device, 9)
    return out


def _weights(w, need_w, need_wt):
    """([N x K values, scales], [K x N values, scales]) of a weight tensor, None for what is
    not asked for: one set of blocks of 128 x 128."""
    transposed = _is_transposed(w)
    stored = w.t() if transposed else w
    rows, columns = (need_w, need_wt) if transposed else (need_wt, need_w)
    if not (rows or columns):
        return None, None
    got = _quantize(stored, BLOCK, torch.float8_e4m3fn, torch.float8_e8m0fnu, rows, columns)
    first = got[:2] if rows else None
    second = (got[2:] if rows else got) if columns else None
    return (first, second) if transposed else (second, first)


def _activations(x, dtype, rows, columns):
    if not (rows or columns):
        return None, None
    got = _quantize(x, 1, dtype, torch.float8_e8m0fnu, rows, columns)
    return got[:2] if rows else None, (got[2:] if rows else got) if columns else None


def _column_sums(dy):
    """The bias' gradient: sums of dy's columns, in float32."""
    db = dy.new_empty(dy.shape[1])
    fields = (DTYPES[dy.dtype], 0, 0, 0, dy.shape[0], dy.shape[1], 0, dy.data_ptr(),
              _matrix(dy, "dy"), 0, 0, 0, 0, 0, 0, dy.shape[1], 0, 0, 0, 0, dy.shape[1],
              db.data_ptr())
    fused._call("tra_linear_backward", fused._GRAD_ARGS, fields, dy.device)
    return db


def _gradients(dy, xt, wt, transposed, grad_dtype, need_dx, need_dw, need_dbias):
    """(dx, dw, dbias) from the column forms of x and of the weight."""
    dx = dw = None
    rows, columns = _activations(dy, grad_dtype, need_dx, need_dw)
    if need_dx:
        dx = _product(*rows, wt[0].t(), wt[1].t(), None, None, dy.dtype, None)
    if need_dw:
        if transposed:
            dw = _product(*columns, xt[0].t(), xt[1].t(), None, None, dy.dtype, None).t()
        else:
            dw = _product(*xt, columns[0].t(), columns[1].t(), None, None, dy.dtype, None)
    return dx, dw, _column_sums(dy) if need_dbias else None


def _is_transposed(w) -> bool:
    """Whether a checked K x N weight is stored N x K."""
    s0, s1 = w.stride()
    # (a single column's elements may lie any way apart)
    return not (s1 == 1 and s0 >= w.shape[1]) and (w.shape[1] > 1 or s0 == 1 or w.shape[0] == 1)


class _ScaledLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, residual, grad_dtype):
        need_x, need_w = ctx.needs_input_grad[:2]
        xq, xt = _activations(x, torch.float8_e4m3fn, True, need_w)
        wq, wt = _weights(w, True, need_x)
        y = _product(*xq, wq[0].t(), wq[1].t(), bias, residual, x.dtype, None)
        ctx.plan = (_is_transposed(w), grad_dtype)
        ctx.save_for_backward(*(xt or (None, None)), *(wt or (None, None)))
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        _no_capture()
        need_x, need_w, need_b, need_r, _ = ctx.needs_input_grad
        dx = dw = db = None
        if need_x or need_w or need_b:
            xt, xts, wt, wts = ctx.saved_tensors
            dx, dw, db = _gradients(_rows(dy), (xt, xts), (wt, wts), *ctx.plan, need_x, need_w,
                                    need_b)
        return dx, dw, db, dy if need_r else None, None


def _check_training(x, w):
    """Both operands are tensors: checks them."""
    _matrix(x, "x")
    _weight(w, "w", x)


def scaled_linear(x, w, x_scales=None, w_scales=None, bias=None, residual=None, dtype=None,
                  out=None, grad_dtype=torch.float8_e4m3fn, stream=None):
    """x w + bias + residual on 8-bit operands, as a new M x N tensor or in ``out``.

    ``w`` is K x N: the transposed view of N x K values (float8_e4m3fn) with ``w_scales``, the
    transposed view of their scales; or a tensor of x's type, in either layout of
    ``linear``, which the call quantizes in blocks of 128 x 128.  ``x`` is M x K: values
    with ``x_scales`` of w_scales' type, or a tensor, which the call quantizes.
    ``dtype``, of the result, bias and residual, is x's by default, and bfloat16 where x is
    values; float32 sums come with float32 alone (see the module).  ``residual`` may be ``out``.

    Differentiable where both x and w are tensors; ``grad_dtype`` is what the result's
    gradient is quantized to, float8_e4m3fn or float8_e5m2.  ``out`` is refused where
    autograd records the call, and so are quantized weights.  ``stream`` as in ``linear``.
    """
    tensors = (x, w, x_scales, w_scales, bias, residual, out)
    _recorded_elsewhere(*tensors)
    if stream is not None:
        return _on(stream, lambda: scaled_linear(x, w, x_scales, w_scales, bias, residual, dtype,
                                                 out, grad_dtype), *tensors)
    if not isinstance(x, torch.Tensor) or not isinstance(w, torch.Tensor):
        raise TypeError("x and w must be torch.Tensors")
    if not x.is_cuda:
        raise TypeError("x must be a tensor on a GPU")
    given = x.dtype in FP8
    if given != (x_scales is not None):
        raise ValueError("x_scales goes with 8-bit x")
    if (w.dtype in FP8) != (w_scales is not None):
        raise ValueError("w_scales goes with 8-bit w")
    if dtype is None:
        dtype = torch.bfloat16 if given else x.dtype
    if dtype not in DTYPES:
        raise ValueError(f"dtype must be one of {', '.join(map(str, DTYPES))}; got {dtype!r}")
    _code(FP8, grad_dtype, "grad_dtype")
    wants = _wants_grad(*tensors)
    if w_scales is None:
        if given or dtype != x.dtype:
            raise ValueError("a w that the call quantizes goes with a tensor x and a result of "
                             "its type")
        _check_training(x, w)
        if wants:
            if out is not None:
                raise ValueError("out cannot be given where gradients are recorded")
            return _ScaledLinear.apply(x, w, bias, residual, grad_dtype)
        (wq, ws), _ = _weights(w, True, False)
        w, w_scales = wq.t(), ws.t()
    elif wants:
        raise ValueError("gradients cannot be recorded with quantized weights: give w as a "
                         "tensor, or use torch.no_grad()")
    y = _product(x, x_scales, w, w_scales, bias, residual, dtype, out)
    if out is not None:
        _written(out)
    return y


def scaled_linear_backward(dy, x, w, grad_dtype=torch.float8_e4m3fn, need_dx=True, need_dw=True,
                           need_dbias=False, stream=None):
    """(dx, dw, dbias) of ``scaled_linear`` for dy, the gradient of its result (that of the
    residual is dy itself); None for each not asked for.  x and w are the tensors of the
    forward call; dw has w's layout.  ``stream`` as in ``linear``."""
    _recorded_elsewhere(dy, x, w)
    if stream is not None:
        return _on(stream, lambda: scaled_linear_backward(dy, x, w, grad_dtype, need_dx, need_dw,
                                                          need_dbias), dy, x, w)
    _check_training(x, w)
    _matrix(dy, "dy", x)
    if dy.shape[0] != x.shape[0] or dy.shape[1] != w.shape[1]:
        raise ValueError(f"dy must be {x.shape[0]} x {w.shape[1]}")
    _code(FP8, grad_dtype, "grad_dtype")
    xt = _activations(x, torch.float8_e4m3fn, False, True)[1] if need_dw else None
    wt = _weights(w, False, True)[1] if need_dx else None
    return _gradients(dy, xt, wt, _is_transposed(w), grad_dtype, need_dx, need_dw, need_dbias)
