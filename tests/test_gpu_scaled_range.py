"""scaled_linear where the product of two scales leaves binary32's range and the result need
not: sums of zero, small values under large scales, large values under small ones.

The definition is s_x s_w t for a block, t the sum of its values' products.  Its terms are taken
in 64 bits here.  In binary32 t s_x s_w is within two roundings, 2^-23 of itself, wherever it is
normal, and within half a unit of the least subnormal, 2^-150, where it is not; then come a
rounding for each block that is added and the store's half step (product_bound, and 2^-149 a
block).  Powers of two that neither overflow nor underflow must come out exactly.
"""
from __future__ import annotations

import pytest
import torch

import tiling_roofline_analysis_amd as tra
from scaled_plans import CALLS, describe
from scaled_reference import FP8, SCALES, Operand, product_bound, up
from test_gpu_linear import half_step, within

pytestmark = pytest.mark.gpu

# (M, N, K), scale, rows of a block of W, result: every kernel that multiplies by scales, or, of
# binary32 results, e8m0 ones; whole and split along K, ragged
ROUTES = [
    ((1, 33, 400), "scaled_few"), ((16, 500, 1300), "scaled_few"),
    ((73, 8900, 272), "scaled_tile"), ((19, 150, 2069), "scaled_tile"),
    ((300, 264, 1040), "scaled_tile"), ((1135, 273, 1425), "scaled_tile"),
    ((2527, 1619, 386), "any"), ((2000, 2049, 144), "any"),
]
FORMS = [("f32", 128, torch.float32), ("f32", 128, torch.bfloat16), ("e8m0", 128, torch.float32),
         ("e8m0", 128, torch.bfloat16), ("e8m0", 1, torch.bfloat16),
         ("e8m0", 1, torch.float32)]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available()


def powers(exponents, scale):
    # (exact, which pow need not be)
    t = torch.ldexp(torch.ones((), dtype=torch.float64, device="cuda"), exponents)
    return t.float().to(SCALES[scale])


def operands(M, N, K, block_rows):
    K = up(K, 16) * 16
    x = torch.zeros(M, K, device="cuda")
    w = torch.zeros(N, K, device="cuda")
    blocks = up(K, 128)
    return (x, w, torch.zeros(M, blocks, device="cuda", dtype=torch.int32),
            torch.zeros(up(N, block_rows), blocks, device="cuda", dtype=torch.int32))


def product(x, w, xs, ws, scale, dtype, **kw):
    return tra.scaled_linear(x.to(FP8["e4m3"]), w.to(FP8["e4m3"]).t(), powers(xs, scale),
                             powers(ws, scale).t(), dtype=dtype, **kw)


@pytest.mark.parametrize("scale,block_rows,dtype", FORMS, ids=str)
@pytest.mark.parametrize("size,kernel", ROUTES, ids=str)
def test_a_block_whose_sum_is_zero_adds_nothing(size, kernel, scale, block_rows, dtype):
    M, N, K = size
    if kernel != "any":
        dt = 0 if dtype is torch.float32 else 1
        assert kernel in describe(M, N, K, scale, dtype=dt, w_block_rows=block_rows)
    x, w, xs, ws = operands(M, N, K, block_rows)
    # block 0: 448 against +-448, whose sum is 0, with scales whose product is 2^140; the others
    # are of ones in their first 8 elements
    x[:, :128], w[:, :128:2], w[:, 1:128:2] = 448.0, 448.0, -448.0
    xs[:, 0], ws[:, 0] = 70, 70
    for b in range(1, xs.shape[1]):
        x[:, b * 128:b * 128 + 8], w[:, b * 128:b * 128 + 8] = 1.0, 1.0
    y = product(x, w, xs, ws, scale, dtype)
    assert torch.equal(y, torch.full_like(y, 8.0 * (xs.shape[1] - 1)))


@pytest.mark.parametrize("scale,block_rows,dtype", FORMS, ids=str)
@pytest.mark.parametrize("size,kernel", ROUTES, ids=str)
@pytest.mark.parametrize("value,ex,ew", [(448.0, -75, -75), (448.0, -126, -24), (448.0, -20, -126),
                                         (2.0 ** -9, 70, 60), (2.0 ** -9, 115, 14),
                                         (2.0 ** -9, 10, 119), (448.0, -110, 115),
                                         (448.0, 115, -110)], ids=str)
def test_products_of_scales_past_the_range(value, ex, ew, size, kernel, scale, block_rows, dtype):
    # 448 x 448 x 128 is 2^24.6: results from 2^-131.4 (a subnormal) on; 2^-18 x 2^130: 2^112
    M, N, K = size
    x, w, xs, ws = operands(M, N, K, block_rows)
    x[:, :128], w[:, :128] = value, value
    if value < 1:
        x[:, 1:128] = 0.0
    xs[:, 0], ws[:, 0] = ex, ew
    want = float((x[0, :128].double() * w[0, :128].double()).sum()) * 2.0 ** (ex + ew)
    y = product(x, w, xs, ws, scale, dtype)
    # (the power of two is exact; 128 x 448 x 448 has 19 bits, 8 of them stored in bfloat16; a
    # subnormal result keeps those above 2^-149, or, in bfloat16, 2^-133)
    least = 2.0 ** -149 if dtype is torch.float32 else 2.0 ** -133
    off = max(abs(want) * (2.0 ** -23 if dtype is torch.float32 else 2.0 ** -8), least)
    assert float((y.double() - want).abs().max()) <= off, (float(y[0, 0]), want)
    assert float(y.abs().min()) > 0


@pytest.mark.parametrize("scale,block_rows,dtype", FORMS, ids=str)
@pytest.mark.parametrize("size,kernel", ROUTES, ids=str)
def test_scales_of_any_exponent(size, kernel, scale, block_rows, dtype):
    # rows of x have blocks of all sizes; columns of w blocks that leave the results inside the
    # range with some of them and not with others, which are not compared
    M, N, K = size
    gen = torch.Generator(device="cuda").manual_seed(M + N)
    x, w, xs, ws = operands(M, N, K, block_rows)
    for t in (x, w):
        t[:, :K] = torch.randint(-8, 9, (t.shape[0], K), generator=gen, device="cuda").float()
    xs.random_(-126, 120, generator=gen)
    ws.random_(-126, 120, generator=gen)
    y = product(x, w, xs, ws, scale, dtype)
    xq, wq = x.to(FP8["e4m3"]), w.to(FP8["e4m3"])
    a, b = Operand(xq, powers(xs, scale), 1), Operand(wq, powers(ws, scale), block_rows)
    want, err = product_bound(a, b, dtype)
    # (no partial sum can pass 2^127)
    fits = a.v.abs() @ b.v.abs().t() < 2.0 ** 127
    assert fits.any() or size[0] == 1
    err = 1.01 * err + half_step(want, dtype) + 2.0 ** -149 * xs.shape[1]
    if dtype is torch.bfloat16:
        err = err + 2.0 ** -134
    within(y[fits], want[fits], err[fits], "y")


@pytest.mark.parametrize("block_rows,dtype", [(128, torch.bfloat16), (128, torch.float32)])
def test_scales_that_are_no_blocks(block_rows, dtype):
    # zero, subnormal, negative and infinite scales stand for what they are
    for M, N in ((5, 40), (70, 300), (2527, 1619)):
        x = torch.ones(M, 256, device="cuda").to(FP8["e4m3"])
        w = torch.ones(N, 256, device="cuda").to(FP8["e4m3"])
        ws = torch.ones(up(N, 128), 2, device="cuda")
        for s in (0.0, 2.0 ** -130, -3.0, float("inf"), float("nan")):
            xs = torch.ones(M, 2, device="cuda")
            xs[M // 2, 1] = s
            y = tra.scaled_linear(x, w.t(), xs, ws.t(), dtype=dtype)
            want = 128.0 + 128.0 * xs[:, 1:].double().expand(M, N)
            assert torch.equal(y.double(), want.to(dtype).double()) or (
                s != s and torch.isnan(y[M // 2]).all() and not torch.isnan(y[:M // 2]).any())


@pytest.mark.parametrize("scale,block_rows,dtype", FORMS, ids=str)
def test_rows_inside_the_range_keep_their_bits(scale, block_rows, dtype):
    # a row whose scales are near either end may have its waves take their sums the other way: the
    # other rows come out as without it
    for M, N, K in ((16, 64, 640), (150, 300, 1300), (2527, 1619, 386)):
        gen = torch.Generator(device="cuda").manual_seed(3)
        x, w, xs, ws = operands(M, N, K, block_rows)
        x[:, :K] = torch.randn(M, K, generator=gen, device="cuda")
        w[:, :K] = torch.randn(N, K, generator=gen, device="cuda")
        want = product(x, w, xs, ws, scale, dtype)
        ws[:, 1] = -3
        near = product(x, w, xs, ws, scale, dtype)
        rows = torch.arange(M, device="cuda") != M // 3
        for ex in (115, -126):
            xs[M // 3, 1] = ex
            far = product(x, w, xs, ws, scale, dtype)
            assert torch.equal(far[rows], near[rows]) and not torch.equal(near, want)
            assert torch.isfinite(far).all() and not torch.equal(far, near)


@pytest.mark.parametrize("scale,block_rows,dtype", FORMS, ids=str)
def test_nan_stays_in_its_row(scale, block_rows, dtype):
    # a row of NaN beside ordinary ones, and beside one whose scales leave the range
    for M, N, K in ((16, 64, 640), (150, 300, 1300), (2527, 1619, 386)):
        gen = torch.Generator(device="cuda").manual_seed(4)
        x, w, xs, ws = operands(M, N, K, block_rows)
        x[:, :K] = torch.randn(M, K, generator=gen, device="cuda")
        w[:, :K] = torch.randn(N, K, generator=gen, device="cuda")
        for ex in (0, 115):
            xs[M // 2 - 1, 1], ws[:, 1] = ex, -3
            x[M // 2, 7] = 1.0
            want = product(x, w, xs, ws, scale, dtype)
            x[M // 2, 7] = float("nan")
            got = product(x, w, xs, ws, scale, dtype)
            rows = torch.arange(M, device="cuda") != M // 2
            assert torch.equal(got[rows], want[rows]) and torch.isnan(got[M // 2]).all()
            assert torch.isfinite(want).all()


@pytest.mark.parametrize("scale,block_rows,dtype", FORMS, ids=str)
@pytest.mark.parametrize("call", CALLS, ids=str)
def test_every_kernel_instance(call, scale, block_rows, dtype):
    # whole and split, deep and shallow, all tile sizes: a block whose sum is 0 under scales of 2^140,
    # a row whose values are small under large scales, a row of NaN
    M, N, K = call
    x, w, xs, ws = operands(M, N, K, block_rows)
    x[:, :128], w[:, :128:2], w[:, 1:128:2] = 448.0, 448.0, -448.0
    xs[:, 0], ws[:, 0] = 70, 70
    for b in range(1, xs.shape[1]):
        x[:, b * 128:b * 128 + 8], w[:, b * 128:b * 128 + 8] = 1.0, 1.0
    want = torch.full((M, N), 8.0 * (xs.shape[1] - 1), device="cuda", dtype=dtype)
    if M > 2:
        # 2^-9 x 448 x 2^(30 + 70), which is 2^99.8, and exact
        x[M // 2, :128], x[M // 2, 0], xs[M // 2, 0] = 0.0, 2.0 ** -9, 30
        want[M // 2] = (2.0 ** -9 * 448.0 * 2.0 ** 100)
        x[M // 3, 1] = float("nan")
        want[M // 3] = float("nan")
    y = product(x, w, xs, ws, scale, dtype)
    assert torch.equal(y.isnan(), want.isnan())
    assert torch.equal(y.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))
