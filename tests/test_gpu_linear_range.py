"""Binary16 gradients whose dZ lies outside binary16's range, on the GPU against
64-bit products.

dZ, the gradient of the pre-activations, is an operand of dX and dW and is held in
binary16 times a power of two.  A term's rounding is at most 2^-11 of it, or 2^-25
of the largest |dZ|; the rest of the tolerance is that of the other gradient tests:
sums of binary32 terms, slopes within 2^-20 (1 + |z|), the result's own rounding.
"""
from __future__ import annotations

import pytest
import torch

import tiling_roofline_analysis_amd as tra
from test_gpu_linear import act64, within

pytestmark = pytest.mark.gpu

F16 = torch.float16


def normal(seed, *shape, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").mul_(scale)


def store_step(v):
    return 2.0 ** -11 * v.abs() + 2.0 ** -25


def check(x, ws, dzs, errs, dx, dws, what):
    """dx and dws for dzs known within errs, each rounded once more."""
    top = max(float(dz.abs().max()) for dz in dzs)
    rounded = [1.01 * (e + 2.0 ** -11 * dz.abs() + 2.0 ** -25 * top) for dz, e in zip(dzs, errs)]
    xd, wd = x.double(), [w.double() for w in ws]
    want = sum(dz @ w.t() for dz, w in zip(dzs, wd))
    tol = sum(r @ w.abs().t() for r, w in zip(rounded, wd))
    size = sum((dz.abs() + r) @ w.abs().t() for dz, r, w in zip(dzs, rounded, wd))
    tol = tol + len(ws) * dzs[0].shape[1] * 2.0 ** -23 * size
    assert float(want.abs().max()) < 65504 and float(want.abs().max()) > 1e-5, what
    within(dx, want, 1.01 * tol + 1.01 * store_step(want), what + " dx")
    for dw, dz, r in zip(dws, dzs, rounded):
        want = xd.t() @ dz
        tol = xd.abs().t() @ r + x.shape[0] * 2.0 ** -23 * (xd.abs().t() @ (dz.abs() + r))
        assert float(want.abs().max()) < 65504 and float(want.abs().max()) > 1e-5, what
        within(dw, want, 1.01 * tol + 1.01 * store_step(want), what + " dw")


# few rows and tiles, whole and split, one and many workgroups of the slope pass
SHAPES = [(3, 96, 64), (40, 96, 64), (130, 1100, 72), (600, 520, 2056)]

# size of dY and of the kept u, and that of x and the weights which brings the
# gradients back into range: a gate's dZ past 65504; of usual size; far below 2^-25
SIZES = {"large": (1e3, 100.0, 1e-3), "usual": (1e-2, 1.0, 1.0), "small": (1e-6, 1e-2, 1e3)}


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("size", list(SIZES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gated_gradients_of_any_size(shape, size, layout):
    M, N, K = shape
    sdy, su, sw = SIZES[size]
    x = normal(1, M, K, scale=sw).to(F16)
    ws = [normal(2 + i, *((K, N) if layout == "kn" else (N, K)), scale=sw).to(F16)
          for i in range(2)]
    ws = ws if layout == "kn" else [w.t() for w in ws]
    dy = normal(4, M, N, scale=sdy).to(F16)
    z = torch.cat([normal(5, M, N), normal(6, M, N, scale=su)], 1).contiguous()
    dx, dg, du = tra.gated_linear_backward(dy, x, *ws, z, "silu")
    a, d = act64(z[:, :N].double(), "silu")
    u, dyd = z[:, N:].double(), dy.double()
    e = 2.0 ** -20 * (1 + z[:, :N].double().abs())
    dzs = [dyd * u * d, dyd * a]
    errs = [(dyd * u).abs() * e + 2.0 ** -22 * dzs[0].abs(), dyd.abs() * e + 2.0 ** -22 * dzs[1].abs()]
    check(x, ws, dzs, errs, dx, (dg, du), f"{size} {layout}")


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gradients_of_saturated_units(shape):
    # slopes of 1e-6 and less in most columns: their dZ is far below the others'
    M, N, K = shape
    x, w = normal(1, M, K, scale=100.0).to(F16), normal(2, K, N, scale=10.0).to(F16)
    dy = normal(3, M, N, scale=1e-2).to(F16)
    z = normal(4, M, N)
    z[:, 3:] -= 14.0
    z[:, 2] *= 0.0
    dx, dw, db = tra.linear_backward(dy, x, w, z, "sigmoid", need_dbias=True)
    d = act64(z.double(), "sigmoid")[1]
    dz = dy.double() * d
    # the slope y (1 - y) is of y's size here, and so is its error
    err = 2.0 ** -19 * (1 + z.double().abs()) * dz.abs()
    check(x, [w], [dz], [err], dx, [dw], "saturated")
    want = dz.sum(0)
    within(db, want, 1.01 * (err.sum(0) + M * 2.0 ** -23 * dz.abs().sum(0)) + store_step(want), "db")
    # the saturated columns' gradients are there at all
    assert float(dw[:, 3:].abs().max()) > 0


@pytest.mark.parametrize("size", [1e-4, 1.0, 3e4])
def test_infinities_and_nan_keep_to_their_rows(size):
    # and do not take part in the choice of the scale
    M, N, K = 70, 200, 96
    x, w = normal(1, M, K, scale=1e-3).to(F16), normal(2, K, N, scale=1e-3).to(F16)
    dy, z = normal(3, M, N, scale=size).clamp_(-6e4, 6e4).to(F16), normal(4, M, N)
    want = tra.linear_backward(dy, x, w, z, "silu")[0]
    dy[5, 7] = float("inf")
    dy[9, 0] = float("nan")
    z[20, 3] = float("nan")
    got = tra.linear_backward(dy, x, w, z, "silu")[0]
    keep = [m for m in range(M) if m not in (5, 9, 20)]
    assert torch.equal(got[keep], want[keep])
    assert not torch.isfinite(got[5]).any()
    assert torch.isnan(got[9]).all() and torch.isnan(got[20]).all()


def test_zero_gradients_are_zero():
    M, N, K = 20, 96, 64
    x, w, z = normal(1, M, K).to(F16), normal(2, K, N).to(F16), normal(3, M, N)
    for t in tra.linear_backward(torch.zeros(M, N, device="cuda", dtype=F16), x, w, z, "gelu",
                                 need_dbias=True):
        assert not t.any()


def test_captured_gradients_follow_the_scale():
    # the scale is found anew by every replay: sizes that take the usual one, and
    # ones that write dZ again, in turn
    M, N, K = 40, 264, 136
    x, w, z = normal(1, M, K, scale=1e-2).to(F16), normal(2, K, N, scale=1e-2).to(F16), normal(3, M, N)
    dy = normal(4, M, N).to(F16)
    tra.linear_backward(dy, x, w, z, "silu")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = tra.linear_backward(dy, x, w, z, "silu")[:2]
    for i, size in enumerate((1.0, 1e4, 1e-5, 1.0, 3e4)):
        dy.copy_(normal(10 + i, M, N, scale=size).clamp_(-6e4, 6e4).to(F16))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = tra.linear_backward(dy, x, w, z, "silu")[:2]
        assert all(torch.equal(a, b) for a, b in zip(got, want)), size


# shapes whose fastest plan, with the stores of kept pre-activations counted, would
# be another
@pytest.mark.parametrize("case", [(193, 6280, 4264, "f32", "nk", 0), (1486, 272, 2256, "bf16", "kn", 0),
                                  (554, 720, 5936, "bf16", "kn", 1), (78, 6080, 7040, "bf16", "nk", 0),
                                  (9, 512, 1024, "f16", "nk", 1)], ids=str)
def test_the_same_bits_with_and_without_gradients(case):
    M, N, K, dtype, layout, gated = case
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": F16}[dtype]
    x = normal(1, M, K).to(dt)
    ws = [normal(2 + i, *((K, N) if layout == "kn" else (N, K)), scale=K ** -0.5).to(dt)
          for i in range(1 + gated)]
    ws = ws if layout == "kn" else [w.t() for w in ws]

    def call(t, **kw):
        return tra.gated_linear(*t, **kw) if gated else tra.linear(*t, act="silu", **kw)

    want = call([x, *ws])
    z = torch.empty(M, N * (1 + gated), device="cuda")
    assert torch.equal(call([x, *ws], z=z), want)
    assert torch.equal(call([t.detach().requires_grad_() for t in (x, *ws)]).detach(), want)
