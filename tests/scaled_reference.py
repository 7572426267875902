"""8-bit matrices with block scales in 64 bits, from the definition: the largest finite
magnitude, the least fitting scale, and each element's nearest value by search."""
from __future__ import annotations

import torch

FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
SCALES = {"f32": torch.float32, "e8m0": torch.float8_e8m0fnu}


def up(n, m):
    return -(-n // m)


def codes(fp8, device):
    """The type's finite values from zero up; their codes are 0, 1, .."""
    v = torch.arange(128, dtype=torch.uint8, device=device).view(FP8[fp8]).double()
    return v[torch.isfinite(v)]


def nearest(t, fp8):
    """Of t's two neighbours the nearer, of two as near the one with the even code; what
    is not finite as the type's own conversion has it."""
    table = codes(fp8, t.device)
    size = t.abs().contiguous()
    high = torch.searchsorted(table, size).clamp(max=table.numel() - 1)
    low = (high - 1).clamp(min=0)
    above, below = table[high] - size, size - table[low]
    code = torch.where((above < below) | ((above == below) & (high % 2 == 0)), high, low)
    got = torch.copysign(table[code], t)
    strange = torch.full_like(t, float("nan")) if fp8 == "e4m3" else t
    return torch.where(torch.isfinite(t), got, strange)


def scale_of(largest, fp8, scale):
    bound = largest / float(codes(fp8, largest.device)[-1])
    if scale == "f32":
        s = bound.float().double().clamp(min=2.0 ** -126)
    else:
        powers = torch.tensor([2.0 ** e for e in range(-127, 128)], dtype=torch.float64,
                              device=largest.device)
        s = powers[torch.searchsorted(powers, bound).clamp(max=254)]
    return torch.where(largest > 0, s, torch.ones_like(s))


def quantized(x, fp8="e4m3", scale="e8m0", block_rows=1):
    """(values, scales) of x in 64 bits, the values filled up to a multiple of 16."""
    M, K = x.shape
    MB, KB = up(M, block_rows), up(K, 128)
    x = torch.nn.functional.pad(x.detach().double(), (0, KB * 128 - K, 0, MB * block_rows - M))
    x = x.view(MB, block_rows, KB, 128)
    size = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))
    s = scale_of(size.amax((1, 3)), fp8, scale)
    q = nearest(x / s[:, None, :, None], fp8).view(MB * block_rows, KB * 128)
    return q[:M, :up(K, 16) * 16].contiguous(), s


def stands_for(values, scales, block_rows=None):
    """What values (any type) with scales stand for, in 64 bits."""
    M, K = values.shape
    s = scales.double()
    if block_rows is None:
        block_rows = 1 if s.shape[0] == M else 128
    s = s.repeat_interleave(block_rows, 0)[:M].repeat_interleave(128, 1)[:, :K]
    return values.double() * s


class Operand:
    """What values with scales stand for (v), and for each 8 neighbours of a row the largest
    magnitude that their matrix instruction may take one to have (g): a subnormal value
    counts as the least normal one."""

    def __init__(self, values, scales, block_rows=None, fp8=None):
        fp8 = fp8 or {t: n for n, t in FP8.items()}[values.dtype]
        self.v = stands_for(values, scales, block_rows)
        least = 2.0 ** -6 if fp8 == "e4m3" else 2.0 ** -14
        size = stands_for(values.double().abs().clamp(min=least), scales, block_rows)
        self.g = size.nan_to_num(0.0).view(size.shape[0], -1, 8).amax(2)


def product_bound(x, w, dtype):
    """x w^T in 64 bits and how far the kernels' sums may be off: K roundings or truncations
    of binary32, and with 16-bit results, 8 neighbouring products at a time, each cut off
    13 binary places below the largest one's exponent: 8 x 2^-13 of it."""
    z = x.v @ w.v.t()
    err = (x.v.shape[1] + 4) * 2.0 ** -23 * (x.v.abs() @ w.v.abs().t())
    if dtype != torch.float32:
        err = err + 8 * 2.0 ** -13 * (x.g @ w.g.t())
    return z, err
