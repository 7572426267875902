"""scaled_linear on the GPU against plain 64-bit products of what the operands stand for.

With S = sum |x||w| over what they stand for, a binary32 sum of K products is within
K 2^-23 S of the exact one, in any order (one rounding or truncation per step).  e8m0
scales add nothing; binary32 scales two roundings a block, 2^-23 S.  16-bit results come
from 8-bit matrix instructions, which cut products off (product_bound).  Bias and residual
are one rounding each, and a store half a step.  Small integers must come out exactly.
"""
from __future__ import annotations

import ctypes

import pytest
import torch

import tiling_roofline_analysis_amd as tra
from scaled_reference import FP8, SCALES, Operand, product_bound, quantized, stands_for, up
from test_gpu_linear import half_step, within

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available()


def test_the_instruction_adds_as_the_bounds_say():
    # eight neighbours: 2^16 and 2^(16 - d) come out whole to d = 13; not neighbours: always
    for far, kept in ((1, 13), (7, 13), (8, 23), (100, 23)):
        for d in range(24):
            a = 16 - d
            ea = min(a // 2, 8) if a > 0 else a // 2
            row = torch.zeros(1, 128, device="cuda")
            row[0, 0], row[0, far] = 2.0 ** 8, 2.0 ** ea
            col = torch.zeros(1, 128, device="cuda")
            col[0, 0], col[0, far] = 2.0 ** 8, 2.0 ** (a - ea)
            one = torch.ones(1, 1, device="cuda").to(SCALES["e8m0"])
            x, w = row.to(FP8["e4m3"]), col.to(FP8["e4m3"])
            # the difference to the largest alone, as a bfloat16 residual leaves it
            big = torch.full((1, 1), -2.0 ** 16, device="cuda", dtype=torch.bfloat16)
            y = tra.scaled_linear(x, w.t(), one, one.t(), residual=big)
            if d <= kept:
                assert float(y) == 2.0 ** a, (far, d)


def normal(M, K, dtype, seed=0, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    size = torch.randn(1, K, generator=gen, device="cuda").mul_(0.7).exp_()
    return torch.randn(M, K, generator=gen, device="cuda").mul_(size).mul_(scale).to(dtype)


def check(y, x, w, bias=None, residual=None, what="y"):
    """y against x w^T + bias + residual, x and w Operands."""
    z, err = product_bound(x, w, y.dtype)
    for t in (bias, residual):
        if t is not None:
            z = z + t.double()
            err = err + 2.0 ** -23 * (z.abs() + t.double().abs())
    within(y, z, err * 1.01 + half_step(z, y.dtype), what)


def weights(N, K, scale, block_rows=128, fp8="e4m3", seed=7):
    w = normal(N, K, torch.float32, seed, K ** -0.5)
    return tra.quantize(w, (block_rows, 128), FP8[fp8], SCALES[scale])


SIZES = [(1, 1, 1), (1, 16, 16), (2, 3, 5), (16, 64, 128), (17, 65, 144), (33, 130, 1000),
         (64, 64, 256), (65, 129, 127), (100, 300, 513), (130, 256, 4100), (257, 1000, 640),
         (700, 520, 2000), (1, 5000, 3000), (300, 1, 300), (515, 4104, 4088), (2000, 2049, 1531)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("scale", list(SCALES))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(size, scale, dtype):
    M, N, K = size
    dt = DTYPES[dtype]
    x, bias, residual = normal(M, K, dt), normal(1, N, dt, 2)[0], normal(M, N, dt, 3)
    w, ws = weights(N, K, scale)
    xq, xs = tra.quantize(x, scale_dtype=SCALES[scale])
    xv, wv = Operand(xq, xs), Operand(w, ws, 128)
    y = tra.scaled_linear(x, w.t(), None, ws.t())
    assert y.dtype == dt
    check(y, xv, wv)
    # quantized before or in the call: the same bits
    assert torch.equal(y, tra.scaled_linear(xq, w.t(), xs, ws.t(), dtype=dt))
    y = tra.scaled_linear(x, w.t(), None, ws.t(), bias, residual)
    check(y, xv, wv, bias, residual)


@pytest.mark.parametrize("size", [(5, 48, 300), (70, 200, 1100), (300, 640, 2064)], ids=str)
@pytest.mark.parametrize("fx,fw,scale,block_rows", [
    ("e4m3", "e4m3", "e8m0", 1), ("e4m3", "e4m3", "e8m0", 128), ("e5m2", "e4m3", "e8m0", 1),
    ("e5m2", "e4m3", "e8m0", 128), ("e4m3", "e5m2", "e8m0", 1), ("e4m3", "e5m2", "e8m0", 128),
    ("e4m3", "e4m3", "f32", 128), ("e5m2", "e4m3", "f32", 128)])
def test_formats(fx, fw, scale, block_rows, size):
    M, N, K = size
    x, xs = tra.quantize(normal(M, K, torch.float32), dtype=FP8[fx], scale_dtype=SCALES[scale])
    w, ws = weights(N, K, scale, block_rows, fw)
    for dt in DTYPES.values():
        y = tra.scaled_linear(x, w.t(), xs, ws.t(), dtype=dt)
        check(y, Operand(x, xs), Operand(w, ws, block_rows))


def ints(M, K, block_rows, scale, gen, fp8="e4m3", most=4):
    """Small integers in 8 bits, with scales that are small integers or powers of two."""
    v = torch.randint(-most, most + 1, (M, up(K, 16) * 16), generator=gen, device="cuda").float()
    v[:, K:] = 0
    shape = (up(M, block_rows), up(K, 128))
    if scale == "e8m0":
        s = 2.0 ** torch.randint(-1, 3, shape, generator=gen, device="cuda").float()
    else:
        s = torch.randint(1, 4, shape, generator=gen, device="cuda").float()
    return v.to(FP8[fp8]), s.to(SCALES[scale])


def exact(M, N, K, fx, fw, scale, block_rows, dt, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x, xs = ints(M, K, 1, scale, gen, fx)
    w, ws = ints(N, K, block_rows, scale, gen, fw)
    a, b = stands_for(x, xs, 1), stands_for(w, ws, block_rows)
    # a unit is 2^-2 at least, and no sum passes 2^22
    assert float(a.abs().max() * b.abs().max()) * K < 2 ** 22
    got = tra.scaled_linear(x, w.t(), xs, ws.t(), dtype=dt)
    assert torch.equal(got, (a @ b.t()).to(dt)), (M, N, K, fx, fw, scale, block_rows)


# the sizes reach every kernel, deep and shallow, split and whole (test_operators_cpu.py
# checks that they do)
from scaled_plans import CALLS, describe  # noqa: E402

FORMATS = [("e4m3", "e4m3", "e8m0", 1), ("e4m3", "e4m3", "e8m0", 128), ("e5m2", "e4m3", "e8m0", 128),
           ("e4m3", "e5m2", "e8m0", 1), ("e4m3", "e4m3", "f32", 128), ("e5m2", "e4m3", "f32", 128)]


@pytest.mark.parametrize("lib", ["product", "poison"])
@pytest.mark.parametrize("form", FORMATS, ids=str)
@pytest.mark.parametrize("call", CALLS, ids=str)
def test_integers_are_exact(call, form, lib, monkeypatch):
    if lib == "poison":
        import tiling_roofline_analysis_amd.fused as fused
        monkeypatch.setattr(fused, "load", POISON.load)
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        exact(*call, *form, dt)


@pytest.mark.parametrize("form", [("e5m2", "e4m3", "e8m0", 1), ("e4m3", "e5m2", "e8m0", 128)],
                         ids=str)
@pytest.mark.parametrize("call", CALLS, ids=str)
def test_integers_are_exact_in_binary32(call, form):
    # (binary32 results have kernels of their own for scales of one row and of 128)
    exact(*call, *form, torch.float32)


class POISON:
    lib = None

    @classmethod
    def load(cls):
        if cls.lib is None:
            cls.lib = tra.load_poisoned()
        return cls.lib


def test_all_pairs_of_values():
    # every finite value of both types against every one of e4m3fn: products one at a time
    for fx in FP8:
        a = torch.arange(256, dtype=torch.uint8, device="cuda").view(FP8[fx])
        a = a[torch.isfinite(a.float())]
        b = torch.arange(256, dtype=torch.uint8, device="cuda").view(FP8["e4m3"])
        b = b[torch.isfinite(b.float())]
        x = torch.zeros(a.numel(), 16, dtype=torch.uint8, device="cuda")
        w = torch.zeros(b.numel(), 16, dtype=torch.uint8, device="cuda")
        x[:, 3], w[:, 3] = a.view(torch.uint8), b.view(torch.uint8)
        x, w = x.view(FP8[fx]), w.view(FP8["e4m3"])
        for scale in SCALES:
            xs = torch.full((a.numel(), 1), 2.0, device="cuda").to(SCALES[scale])
            ws = torch.full((up(b.numel(), 128), 1), 0.25, device="cuda").to(SCALES[scale])
            y = tra.scaled_linear(x, w.t(), xs, ws.t(), dtype=torch.float32)
            assert torch.equal(y, 0.5 * a.float()[:, None] * b.float()[None])


def test_scales_of_all_sizes():
    # e8m0 over its range: sums in binary32's, subnormal results flushed or not
    x = torch.ones(256, 16, device="cuda").to(FP8["e4m3"])
    w = torch.ones(300, 16, device="cuda").to(FP8["e4m3"])
    bits = torch.arange(256, dtype=torch.uint8, device="cuda")
    xs = bits.view(SCALES["e8m0"])[:, None]
    ws = bits[torch.arange(300, device="cuda") % 256].view(SCALES["e8m0"])[:, None]
    y = tra.scaled_linear(x, w.t(), xs, ws.t(), dtype=torch.float32)
    want = 16 * xs.double() @ ws.double().t()
    normal_range = (want >= 2.0 ** -126) & (want < 2.0 ** 128)
    assert torch.equal(y[normal_range], want[normal_range].float())
    assert torch.isnan(y[255]).all() and torch.isnan(y[:, 255]).all()
    assert (y[want >= 2.0 ** 128] == float("inf")).all()
    low = want < 2.0 ** -126
    assert (y[low].double() <= want[low]).all()
    # binary32 scales over theirs
    xs = 2.0 ** torch.arange(-126, 128, device="cuda").float()[:, None]
    x = torch.ones(254, 16, device="cuda").to(FP8["e4m3"])
    ws = torch.tensor([[1.5], [2.0 ** -20], [2.0 ** 20]], device="cuda")
    y = tra.scaled_linear(x, w.t(), xs, ws.t(), dtype=torch.float32)
    want = 16 * xs.double() @ ws.double().repeat_interleave(128, 0)[:300].t()
    ok = (want >= 2.0 ** -100) & (want < 2.0 ** 124)
    assert torch.equal(y[ok], want[ok].float())


def test_strides_of_scales_and_values():
    M, N, K = 70, 300, 700
    x = normal(M, K, torch.bfloat16)
    for scale in SCALES:
        w, ws = weights(N, K, scale)
        xq, xs = tra.quantize(x, scale_dtype=SCALES[scale])
        want = tra.scaled_linear(xq, w.t(), xs, ws.t())
        # row-major and column-major scales, inside larger tensors
        for s in (xs.contiguous(), xs.t().contiguous().t()):
            for t in (ws.contiguous(), ws.t().contiguous().t()):
                assert torch.equal(tra.scaled_linear(xq, w.t(), s, t.t()), want)
        big = torch.zeros(M, 9, device="cuda", dtype=torch.uint8 if scale == "e8m0" else torch.float32)
        big = big.view(SCALES[scale])
        big[:, 2:2 + xs.shape[1]].copy_(xs)
        assert torch.equal(tra.scaled_linear(xq, w.t(), big[:, 2:2 + xs.shape[1]], ws.t()), want)
        wide = torch.full((M, 1024), 0x7f, device="cuda", dtype=torch.uint8).view(FP8["e4m3"])
        wide[:, 64:64 + xq.shape[1]].copy_(xq)
        wb = torch.full((N, 1024), 0x7f, device="cuda", dtype=torch.uint8).view(FP8["e4m3"])
        wb[:, 16:16 + w.shape[1]].copy_(w)
        got = tra.scaled_linear(wide[:, 64:64 + xq.shape[1]], wb[:, 16:16 + w.shape[1]].t(), xs,
                                ws.t())
        assert torch.equal(got, want)


@pytest.mark.parametrize("pad", [1, 8])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_padded_rows_are_left_alone(dtype, pad):
    dt = DTYPES[dtype]
    for M, N, K in ((5, 33, 200), (70, 200, 1100)):
        w, ws = weights(N, K, "e8m0")
        x = normal(M, K + pad, dt)[:, :K]
        r = normal(M, N + pad, dt, 5)[:, :N]
        buf = torch.full((M + 2, N + pad), 7.0, device="cuda", dtype=dt)
        y = tra.scaled_linear(x, w.t(), None, ws.t(), residual=r, out=buf[:M, :N])
        check(y, Operand(*tra.quantize(x)), Operand(w, ws, 128), None, r)
        assert (buf[:M, N:] == 7).all() and (buf[M:] == 7).all()


def test_residual_in_place():
    for M, N, K in ((1, 200, 300), (130, 192, 640)):
        w, ws = weights(N, K, "f32")
        x, r = normal(M, K, torch.bfloat16), normal(M, N, torch.bfloat16, 4)
        want = tra.scaled_linear(x, w.t(), None, ws.t(), residual=r)
        buf = r.clone()
        assert tra.scaled_linear(x, w.t(), None, ws.t(), residual=buf, out=buf) is buf
        assert torch.equal(buf, want)


@pytest.mark.parametrize("scale", list(SCALES))
def test_rows_past_32_bit_offsets(scale):
    # rows 5 GB into a buffer: x, its values, the result
    M, N, K, ld = 70000, 72, 144, 80000
    gen = torch.Generator(device="cuda").manual_seed(1)
    big = torch.zeros(M, ld, dtype=torch.uint8, device="cuda").view(FP8["e4m3"])
    x, xs = ints(M, K, 1, scale, gen)
    far = big[:, 79000 // 16 * 16:][:, :K]
    far.copy_(x)
    w, ws = ints(N, K, 128, scale, gen)
    want = tra.scaled_linear(x, w.t(), xs, ws.t())
    assert torch.equal(want, (stands_for(x, xs) @ stands_for(w, ws, 128).t()).bfloat16())
    assert torch.equal(tra.scaled_linear(far, w.t(), xs, ws.t()), want)
    del big, far
    buf = torch.zeros(M, 40000, dtype=torch.bfloat16, device="cuda")
    tra.scaled_linear(x, w.t(), xs, ws.t(), out=buf[:, 39000:39000 + N])
    assert torch.equal(buf[:, 39000:39000 + N], want)
    t = buf[:, 100:100 + K]
    t.copy_(x.float())
    assert torch.equal(tra.scaled_linear(t, w.t(), None, ws.t()),
                       tra.scaled_linear(t.contiguous(), w.t(), None, ws.t()))


def test_long_k():
    for scale in SCALES:
        x, (w, ws) = normal(20, 150000, torch.bfloat16), weights(24, 150000, scale)
        check(tra.scaled_linear(x, w.t(), None, ws.t()),
              Operand(*tra.quantize(x, scale_dtype=SCALES[scale])), Operand(w, ws, 128))


def test_nan_stays_in_its_row_and_column():
    for M, N, K in ((3, 40, 130), (70, 200, 1000)):
        for scale in SCALES:
            w, ws = weights(N, K, scale)
            x = normal(M, K, torch.bfloat16)
            want = tra.scaled_linear(x, w.t(), None, ws.t())
            x[1, K - 1] = float("nan")
            got = tra.scaled_linear(x, w.t(), None, ws.t())
            keep = torch.arange(M, device="cuda") != 1
            assert torch.equal(got[keep], want[keep]) and torch.isnan(got[1]).all()
            w.view(torch.uint8)[5, 0] = 0x7f
            got = tra.scaled_linear(x, w.t(), None, ws.t())
            assert torch.isnan(got[:, 5]).all()
            cols = torch.arange(N, device="cuda") != 5
            assert torch.equal(got[keep][:, cols], want[keep][:, cols])


@pytest.mark.parametrize("shape", [(0, 8, 8), (8, 0, 8), (8, 8, 0), (0, 0, 0)], ids=str)
def test_empty_sizes(shape):
    M, N, K = shape
    x = torch.ones(M, K, device="cuda").requires_grad_()
    w = torch.ones(N, K, device="cuda").requires_grad_()
    b = torch.full((N,), 2.0, device="cuda").requires_grad_()
    y = tra.scaled_linear(x, w.t(), bias=b)
    assert torch.equal(y, torch.full((M, N), 2.0, device="cuda"))
    dx, dw, db = torch.autograd.grad(y, (x, w, b), torch.ones_like(y))
    assert dx.shape == x.shape and dw.shape == w.shape and torch.equal(db, torch.full_like(db, M))
    assert not dx.any() or N > 0
    assert not dw.any() or M > 0


# --- training -------------------------------------------------------------------------

def q64(t, fp8="e4m3", block_rows=1):
    return Operand(*quantized(t, fp8, "e8m0", block_rows), block_rows, fp8)


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("grad", list(FP8))
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("size", [(1, 1, 1), (5, 17, 33), (70, 130, 200), (300, 260, 513),
                                  (129, 640, 256), (1000, 384, 512)], ids=str)
def test_training_step(size, dtype, grad, layout):
    M, N, K = size
    dt = DTYPES[dtype]
    x, b, r = normal(M, K, dt), normal(1, N, dt, 2)[0], normal(M, N, dt, 3)
    w = normal(N, K, dt, 7, K ** -0.5)
    w = w.t() if layout == "nk" else w.t().contiguous()
    dy = normal(M, N, dt, 5, 0.1)
    leaves = [t.detach().requires_grad_() for t in (x, w, b, r)]
    y = tra.scaled_linear(leaves[0], leaves[1], bias=leaves[2], residual=leaves[3],
                          grad_dtype=FP8[grad])
    wq = q64(w.t(), block_rows=128)
    check(y, q64(x), wq, b, r)
    dx, dw, db, dr = torch.autograd.grad(y, leaves, dy)
    check(dx, q64(dy, grad), q64(w, block_rows=128), what="dx")
    assert dw.stride() == w.stride() or 1 in w.shape
    check(dw.t(), q64(dy.t(), grad), q64(x.t()), what="dw")
    sums = dy.double().sum(0)
    tol = M * 2.0 ** -23 * dy.double().abs().sum(0)
    within(db, sums, tol + half_step(sums, dt), "db")
    assert torch.equal(dr, dy)
    # the passes by themselves
    with torch.no_grad():
        assert torch.equal(tra.scaled_linear(x, w, bias=b, residual=r), y)
    again = tra.scaled_linear_backward(dy, x, w, FP8[grad], need_dbias=True)
    assert all(torch.equal(a, c) for a, c in zip(again, (dx, dw, db)))


def test_gradients_are_those_of_the_unquantized_product_roughly():
    # against differences of x w: each operand's values are off by 2^-4 at most and by
    # 0.03 in the mean square (a uniform error of a step's half over the octave), two a
    # product, independent over long sums
    M, N, K = 512, 512, 512
    gen = torch.Generator(device="cuda").manual_seed(0)
    x, w, dy = (torch.randn(512, 512, generator=gen, device="cuda") for _ in range(3))
    leaves = [x.clone().requires_grad_(), w.clone().requires_grad_()]
    y = tra.scaled_linear(*leaves)
    dx, dw = torch.autograd.grad(y, leaves, dy)
    for got, want in ((y.detach(), x @ w), (dx, dy @ w.t()), (dw, x.t() @ dy)):
        assert float((got - want).norm() / want.norm()) < 2 ** 0.5 * 0.04
    # and a step along a direction, in the loss's own quantized product
    way = torch.randn(512, 512, generator=gen, device="cuda")
    slope = float(((((x + way) @ w) - (x @ w)).double() * dy.double()).sum())
    assert abs(float((dx.double() * way.double()).sum()) - slope) < 0.06 * float(
        dx.double().norm() * way.double().norm()) / 512 ** 0.5


def test_only_what_is_asked_for():
    x, w, dy = normal(40, 200, torch.bfloat16), normal(72, 200, torch.bfloat16, 1), normal(
        40, 72, torch.bfloat16, 2)
    b = torch.zeros(72, device="cuda", dtype=torch.bfloat16)
    r = torch.zeros(40, 72, device="cuda", dtype=torch.bfloat16)
    want = tra.scaled_linear_backward(dy, x, w.t(), need_dbias=True)
    for i in range(4):
        leaves = [t.detach().requires_grad_(j == i) for j, t in enumerate((x, w.t(), b, r))]
        y = tra.scaled_linear(leaves[0], leaves[1], bias=leaves[2], residual=leaves[3])
        (g,) = torch.autograd.grad(y, leaves[i], dy)
        assert torch.equal(g, want[i] if i < 3 else dy)


def test_expanded_gradients_and_saved_tensors_of_other_strides():
    x, w = normal(40, 200, torch.bfloat16), normal(72, 200, torch.bfloat16, 1)
    leaves = [x.requires_grad_(), w.requires_grad_()]
    y = tra.scaled_linear(leaves[0], leaves[1].t())
    full = torch.autograd.grad(y, leaves, torch.ones_like(y), retain_graph=True)
    assert all(torch.equal(a, f) for a, f in zip(torch.autograd.grad(y.sum(), leaves), full))
    with torch.autograd.graph.save_on_cpu():
        y = tra.scaled_linear(leaves[0], leaves[1].t())
        got = torch.autograd.grad(y, leaves, torch.ones_like(y))
    assert all(torch.equal(a, f) for a, f in zip(got, full))


# --- streams, graphs ---------------------------------------------------------------------

def test_same_bits_every_time():
    for M, N, K in ((1, 512, 8192), (60, 300, 4096), (700, 512, 2048)):
        x, (w, ws) = normal(M, K, torch.bfloat16), weights(N, K, "e8m0")
        first = tra.scaled_linear(x, w.t(), None, ws.t())
        for _ in range(3):
            assert torch.equal(tra.scaled_linear(x, w.t(), None, ws.t()), first)


def test_captured_step_replays():
    M, N, K = 40, 384, 1536
    x, w = normal(M, K, torch.bfloat16), normal(N, K, torch.bfloat16, 1, K ** -0.5)
    wq, ws = tra.quantize(w, (128, 128))

    def step():
        y = tra.scaled_linear(x, wq.t(), None, ws.t())
        z = tra.scaled_linear(x, w.t())
        return (y, z, *tra.scaled_linear_backward(z, x, w.t(), need_dbias=True))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(4):
        x.copy_(normal(M, K, torch.bfloat16, i))
        g.replay()
        tra.scaled_linear(x, wq.t(), None, ws.t())
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step())), i


def test_streams_side_by_side():
    # splits and quantized inputs: each call has its own workspace
    M, N, K = 24, 512, 8192
    w, ws = weights(N, K, "e8m0")
    xs = [normal(M, K, torch.bfloat16, i) for i in range(3)]
    want = [tra.scaled_linear(x, w.t(), None, ws.t()) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(4):
        got = [[tra.scaled_linear(x, w.t(), None, ws.t(), stream=s) for _ in range(8)]
               for x, s in zip(xs, streams)]
        torch.cuda.synchronize()
        for g, t in zip(got, want):
            assert all(torch.equal(y, t) for y in g)


def test_memory_dropped_after_a_call_on_a_stream():
    w, ws = weights(512, 2048, "e8m0")
    x = normal(64, 2048, torch.bfloat16)
    want = tra.scaled_linear(x, w.t(), None, ws.t()).clone()
    mine = [x.clone(), w.clone(), ws.clone()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    got = tra.scaled_linear(mine[0], mine[1].t(), None, mine[2].t(), stream=s)
    shapes = [(t.shape, t.dtype) for t in mine]
    del mine
    again = [torch.full(shape, 1, device="cuda", dtype=torch.uint8 if d.itemsize == 1 else d)
             for shape, d in shapes]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    del again


def test_autograd_is_refused_in_a_capture():
    # (a stand-in for the capture: nothing is recorded on the GPU)
    x, w = torch.ones(4, 32, device="cuda"), torch.ones(8, 32, device="cuda")
    real = torch.cuda.is_current_stream_capturing
    torch.cuda.is_current_stream_capturing = lambda: True
    try:
        with pytest.raises(RuntimeError, match="captured"):
            tra.scaled_linear(x, w.clone().requires_grad_().t())
        tra.scaled_linear(x, w.t())
    finally:
        torch.cuda.is_current_stream_capturing = real


def test_block_in_8_bits():
    # add_norm -> quantize -> scaled_linear -> add_norm, as a block runs, with gradients:
    # x + gate * down(up(norm(x + h)))
    M, D, F = 200, 264, 520
    dt = torch.bfloat16
    x, h = normal(M, D, dt), normal(M, D, dt, 1)
    wu, wd = normal(F, D, dt, 2, D ** -0.5), normal(D, F, dt, 3, F ** -0.5)
    g, gate = normal(1, D, dt, 4)[0], normal(1, D, dt, 5)[0]
    dy = normal(M, D, dt, 6)
    leaves = [t.detach().requires_grad_() for t in (x, h, wu, wd, g, gate)]

    def block(x, h, wu, wd, g, gate):
        r, y = tra.add_norm(x, h, weight=g)
        u = tra.scaled_linear(y, wu.t())
        out, _ = tra.add_norm(r, tra.scaled_linear(u, wd.t()), gate=gate, kind="none")
        return out

    out = block(*leaves)
    grads = torch.autograd.grad(out, leaves, dy)
    wide = [t.detach().double().requires_grad_() for t in leaves]
    r = wide[0] + wide[1]
    y = r / (r.square().mean(1, keepdim=True) + 1e-6).sqrt() * wide[4]
    want = r + wide[5] * ((y @ wide[2].t()) @ wide[3].t())
    wants = torch.autograd.grad(want, wide, dy.double())
    # each quantized operand is off by 0.03 of its size in the mean square (e4m3fn: half a
    # step is 2^-4 at most, uniform over the octave), independently: a chain of n products
    # has 2 n of them.  At most two products lie on the way to any of these: 4 x 0.04^2
    for got, ref in [(out, want), *zip(grads, wants)]:
        got, ref = got.detach().double(), ref.detach()
        assert float((got - ref).norm() / ref.norm()) <= (2 * 4 * 0.04 ** 2) ** 0.5
    # serving: the weights quantized once, the activations by themselves: the same bits
    with torch.no_grad():
        qu, qd = tra.quantize(wu, (128, 128)), tra.quantize(wd, (128, 128))
        r, y = tra.add_norm(x, h, weight=g)
        yq, ys = tra.quantize(y)
        u = tra.scaled_linear(yq, qu[0].t(), ys, qu[1].t())
        z = tra.scaled_linear(u, qd[0].t(), None, qd[1].t())
        assert torch.equal(tra.add_norm(r, z, gate=gate, kind="none")[0], out)


def test_refusals():
    x = torch.ones(8, 256, device="cuda", dtype=torch.bfloat16)
    w, ws = tra.quantize(torch.ones(64, 256, device="cuda"), (128, 128))
    r1, r1s = tra.quantize(torch.ones(64, 256, device="cuda"))
    wf, wfs = tra.quantize(torch.ones(64, 256, device="cuda"), scale_dtype=torch.float32)
    q, qs = tra.quantize(x)
    q5, q5s = tra.quantize(x, dtype=FP8["e5m2"])
    w5, w5s = tra.quantize(torch.ones(64, 256, device="cuda"), (128, 128), FP8["e5m2"])
    mm = tra.scaled_linear
    off = torch.zeros(64, 272, device="cuda", dtype=torch.uint8).view(FP8["e4m3"])
    for error, call in [
            (ValueError, lambda: mm(x, w.t())),                          # no scales
            (ValueError, lambda: mm(q, w.t(), None, ws.t())),
            (ValueError, lambda: mm(x, w.t(), qs, ws.t())),
            (ValueError, lambda: mm(q, w.t().float(), qs)),              # w to quantize, x values
            (ValueError, lambda: mm(x[:, :200], w.t(), None, ws.t())),
            (ValueError, lambda: mm(q[:, :128], w.t(), qs[:, :1], ws.t())),
            (ValueError, lambda: mm(q, w.t(), qs[:4], ws.t())),
            (ValueError, lambda: mm(q, w.t(), qs, ws.t()[:1])),
            (ValueError, lambda: mm(q, w.t(), qs.float(), ws.t())),      # two types of scales
            (ValueError, lambda: mm(x, wf.t(), None, wfs.t())),          # f32 scales of rows
            (ValueError, lambda: mm(q5, w5.t(), q5s, w5s.t())),          # both e5m2
            (ValueError, lambda: mm(x, w5.t(), None, w5s.t())),
            (ValueError, lambda: mm(x, w, None, ws)),                    # not the transposed view
            (ValueError, lambda: mm(x, off[:, 8:264].t(), None, ws.t())),    # off alignment
            (ValueError, lambda: mm(x, w.t(), None, ws.t(), dtype=torch.float64)),
            (TypeError, lambda: mm(x, w.t(), None, ws.t(), bias=torch.ones(64, device="cuda"))),
            (ValueError, lambda: mm(x, w.t(), None, ws.t(), residual=x[:, :8])),
            (ValueError, lambda: mm(x, w.t(), None, ws.t(), out=x[:4, :64])),
            (tra.TraError, lambda: mm(x, w.t(), None, ws.t(), out=x[:, :64])),
            (ValueError, lambda: mm(x.clone().requires_grad_(), w.t(), None, ws.t())),
            (TypeError, lambda: mm(x, torch.ones(256, 8, device="cuda"))),
            (ValueError, lambda: mm(x, torch.ones(256, 8, device="cuda", dtype=x.dtype),
                                    dtype=torch.float32)),
            (ValueError, lambda: mm(x, torch.ones(256, 8, device="cuda", dtype=x.dtype),
                                    grad_dtype=torch.float16)),
            (ValueError, lambda: mm(x.clone().requires_grad_(),
                                    torch.ones(256, 8, device="cuda", dtype=x.dtype),
                                    out=x[:, :8].contiguous())),
            (ValueError, lambda: tra.scaled_linear_backward(x, x, torch.ones(
                256, 8, device="cuda", dtype=x.dtype)))]:
        with pytest.raises(error):
            call()
    assert isinstance(describe(8, 64, 256, "e8m0"), str)
