"""The fused linear operators' activations and slopes by themselves, on the GPU: one
input times a weight of one, in binary32, so that the pre-activation is the input
and nothing but the activation's own error is left.

Tolerances count binary32 roundings (u = 2^-24 relative) and the units in the last
place of the hardware's exp2 and reciprocal (2^-23 each):
  gelu       |z| < 1: Phi = 1/2 + z R, R within 1.1 ULP (its fit 4.1e-8, the rounding of
             z^2, Horner) of itself, so Phi within 1.1 ULP |Phi - 1/2| + u Phi.
             Beyond: q = Phi(-|z|) = 2^-Q.  Q's Horner steps round by u times 4.2 Q at
             most (the sum of the intermediate results' sizes), exp2 by an ULP, and the
             fit with its coefficients rounded is within 1.25 times the least of
             3e-8 (1 - q) / q, 3e-8 / (|z| q) and 3e-4: q within
             q (ULP (1.46 Q + 1) + fit).  1 - q rounds once more.  Past 9, where
             q < 2^-62, it only has to stay that small.
             The products with z and of the slope add u each; the slope's exponential
             is within ULP (0.5 z^2 + 1).
  sigmoid    s within 2^-23 ((1 - s) (|z| + 1) + 1.5): the exponent's rounding, exp2,
             the sum, the reciprocal; gelu_tanh has (1 - s) (4 |a| + 1) for its
             argument a, whose four steps round; products add u each.
Below 2^-120 the hardware's exp2 and reciprocal flush: absolute 2^-120 (1 + |z|).
"""
from __future__ import annotations

import math

import pytest
import torch

import tiling_roofline_analysis_amd as tra
from test_gpu_linear import ACTS, act64

pytestmark = pytest.mark.gpu

U, ULP = 2.0 ** -24, 2.0 ** -23


def points():
    parts = [torch.linspace(-12, 12, 30001), torch.linspace(-0.1, 0.1, 4001),
             torch.linspace(0.99, 1.01, 2001), -torch.linspace(0.99, 1.01, 2001),
             torch.linspace(-60, 60, 3001), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 88.0, -88.0])]
    return torch.cat(parts).cuda()


def exact(z, act):
    """act(z), act'(z) in 64 bits.  gelu_tanh through 1 + tanh(a) = 2 sigmoid(2a):
    1 + tanh(a) itself is off by 2^-53 absolute, which is more than the value's
    tolerance where |z| > 6 (z = -7.2: 4e-16 of a value of 4e-16)."""
    if act != "gelu_tanh":
        return act64(z, act)
    c = 2 * math.sqrt(2 / math.pi)
    s, r = (torch.sigmoid(v * c * (z + 0.044715 * z ** 3)) for v in (1, -1))
    return z * s, s + z * s * r * c * (1 + 3 * 0.044715 * z * z)


def phi_error(z, cdf):
    a = z.abs()
    q = 0.5 * torch.erfc(a / math.sqrt(2))
    tiny = q.clamp(min=1e-300)
    fit = 1.25 * torch.minimum(3e-8 * (1 - q) / tiny, 3e-8 / (a * tiny)).clamp(max=3e-4)
    tail = q * (ULP * (1.46 * -torch.log2(tiny) + 1) + fit) + U * cdf * (z > 0)
    core = 1.1 * ULP * (cdf - 0.5).abs() + U * cdf
    return torch.where(a < 1, core, tail) + 2.0 ** -60 * (a > 9)


def tolerances(z, act):
    """How far act(z) and act'(z) may be from their values."""
    y, d = exact(z, act)
    flush = 2.0 ** -120 * (1 + z.abs())
    if act in ("none", "relu"):
        return 0 * z, 0 * z
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
        pdf = z.abs() * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        ep = phi_error(z, cdf)
        return (1.01 * (z.abs() * ep + U * y.abs()) + flush,
                1.01 * (ep + pdf * (ULP * (0.5 * z * z + 1) + 2 * U) + U * d.abs()) + flush)
    if act == "gelu_tanh":
        a = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        s = torch.sigmoid(a)
        es = s * ULP * ((1 - s) * (4 * a.abs() + 1) + 1.5)
        slope = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
        ey = z.abs() * es + U * y.abs()
        # s + y (1 - s) slope
        ed = es + slope * ((1 - s) * ey + y.abs() * (es + U * (1 - s))) + 6 * U * (s + d.abs())
        return 1.01 * ey + flush, 1.01 * ed + flush * slope
    s = torch.sigmoid(z)
    es = s * ULP * ((1 - s) * (z.abs() + 1) + 1.5)
    if act == "sigmoid":
        return 1.01 * es + flush, 1.01 * (es + U * (1 - s) * s + U * s) + flush
    ey = z.abs() * es + U * y.abs()
    return (1.01 * ey + flush,
            1.01 * (es + (1 - s) * ey + y.abs() * (es + U) + 3 * U * (s + d.abs())) + flush)


@pytest.mark.parametrize("act", ACTS)
def test_activation_and_slope(act):
    z = points()
    x, w = z[:, None], torch.ones(1, 1, device="cuda")
    kept = torch.empty_like(x)
    y = tra.linear(x, w, act=act, z=kept)
    assert torch.equal(kept, x)
    d = tra.linear_backward(torch.ones_like(x), x, w, kept, act)[0]
    want, slope = exact(z.double(), act)
    tol, dtol = tolerances(z.double(), act)
    for got, ref, t, what in ((y, want, tol, "value"), (d, slope, dtol, "slope")):
        err = (got[:, 0].double() - ref).abs()
        bad = ~(err <= t)
        worst = int((err - t).argmax())
        assert not bad.any(), (f"{act} {what}: {int(bad.sum())} off, worst at z = "
                               f"{float(z[worst])!r}: {float(err[worst]):.3g} where "
                               f"{float(t[worst]):.3g} is allowed")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("act", ACTS)
def test_activation_in_16_bits(act, dtype):
    z = points().to(dtype)
    y = tra.linear(z[:, None], torch.ones(1, 1, device="cuda", dtype=dtype), act=act)[:, 0]
    want = exact(z.double(), act)[0]
    tol = 1.01 * tolerances(z.double(), act)[0] + torch.finfo(dtype).eps / 2 * want.abs()
    tol = tol + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -130)
    assert ((y.double() - want).abs() <= 1.01 * tol).all()
