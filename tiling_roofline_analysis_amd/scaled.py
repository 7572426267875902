"""Matrices in 8-bit floating point with a scale for each block of 128, on torch tensors:
``quantize`` and products of what it makes.

A block is 128 consecutive elements along the axis that a product sums over, of one row
(activations, gradients) or of 128 rows (weights).  Its scale is float32 or, as the
matrix units of MI355X take it, float8_e8m0fnu, a power of two.  A matrix is a pair of
plain tensors: values (float8_e4m3fn or float8_e5m2, rows x columns filled up with zeros to
a multiple of 16) and scales (rows, or rows / 128 rounded up, x columns / 128 rounded up).
"""
from __future__ import annotations

import struct

import torch

from . import TRA_OK, TraError, load
from .fused import DTYPES, _matrix, _on, _recorded_elsewhere

# tra_fp8, tra_scale
FP8 = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}
SCALES = {torch.float32: 0, torch.float8_e8m0fnu: 1}
FORMS = ("rows", "columns", "both")
BLOCK = 128

# tra_quantize_args, field by field
_QUANTIZE = struct.Struct("@4i2qPqPqPqqPqPqq")


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


def _empty(rows, cols, block_rows, dtype, scale_dtype, device):
    """An 8-bit matrix: values, scales and the scales' strides.  Scales of rows lie next
    to each other for one block of columns: a product reads them so."""
    values = torch.empty((rows, _up(cols, 16) * 16), dtype=dtype, device=device)
    r, b = _up(rows, block_rows), _up(cols, BLOCK)
    if block_rows == 1:
        return values, torch.empty((b, r), dtype=scale_dtype, device=device).t(), 1, r
    return values, torch.empty((r, b), dtype=scale_dtype, device=device), b, 1


def _call(name, packed, device):
    if torch.cuda.current_device() == device.index:
        st = getattr(load(), name)(packed, torch._C._cuda_getCurrentRawStream(device.index))
    else:
        with torch.cuda.device(device):
            st = getattr(load(), name)(packed, torch._C._cuda_getCurrentRawStream(device.index))
    if st != TRA_OK:
        raise TraError(st, name)


def _quantize(x, block_rows, dtype, scale_dtype, rows, columns):
    """The forms asked for of a checked x: [values, scales] each."""
    ldx = _matrix(x, "x")
    M, K = x.shape
    fields, got = [], []
    for want, r, c in ((rows, M, K), (columns, K, M)):
        if not want:
            fields += [0, 0, 0, 0, 0]
            continue
        values, scales, ss_row, ss_block = _empty(r, c, block_rows, dtype, scale_dtype, x.device)
        fields += [values.data_ptr(), values.shape[1], scales.data_ptr(), ss_row, ss_block]
        got += [values, scales]
    _call("tra_quantize", _QUANTIZE.pack(DTYPES[x.dtype], FP8[dtype], SCALES[scale_dtype],
                                         block_rows, M, K, x.data_ptr(), ldx, *fields), x.device)
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
