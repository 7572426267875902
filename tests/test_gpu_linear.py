"""The fused linear operators on the GPU against plain 64-bit products.

Tolerances are derived per element.  With S = sum |x||w| (+ |bias|):
  * a binary32 sum of K products is within K 2^-23 S of the exact one, in any
    order (one rounding or truncation per step);
  * the activations and their slopes are Lipschitz with constants below 1.2
    (gelu: 1.13 and 0.80; silu: 1.10 and 0.5), and evaluated within
    2^-20 (1 + |z|);
  * a store rounds by at most eps / 2 of the value (binary16: or half its
    smallest step, 2^-25), and so does dZ, which the products take in the
    element type.
Integer inputs with sums below 2^24 must come out exactly.
"""
from __future__ import annotations

import math

import pytest
import torch

import tiling_roofline_analysis_amd as tra
from tiling_roofline_analysis_amd import fused

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACTS = list(fused.ACTS)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available()


def act64(z, act):
    """act(z), act'(z) in 64 bits."""
    one = torch.ones_like(z)
    if act == "none":
        return z, one
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return (0.5 * z * (1 + t),
                0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z))
    s = torch.sigmoid(z)
    if act == "sigmoid":
        return s, s * (1 - s)
    return z * s, s * (1 + z * (1 - s))


def half_step(v, dtype):
    return torch.finfo(dtype).eps / 2 * v.abs() + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def product(x, w):
    """x @ w in 64 bits and the bound of a binary32 sum."""
    z = x.double() @ w.double()
    s = x.double().abs() @ w.double().abs()
    return z, x.shape[1] * 2.0 ** -23 * s


def within(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float(err.max()):.3g} where {float(tol[bad].min()):.3g} is allowed")


def weight(K, N, layout, dtype, gen, pad=0):
    shape = (K, N + pad) if layout == "kn" else (N, K + pad)
    t = torch.randn(shape, generator=gen, device="cuda").mul_(K ** -0.5).to(dtype)
    t = t[:, :shape[1] - pad] if pad else t
    return t if layout == "kn" else t.t()


def make(M, N, K, dtype, layout, seed=0, gated=False, pad=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K + pad, generator=gen, device="cuda").to(dtype)[:, :K]
    ws = [weight(K, N, layout, dtype, gen, pad) for _ in range(1 + gated)]
    b = torch.randn(N, generator=gen, device="cuda").mul_(0.5).to(dtype)
    r = torch.randn(M, N + pad, generator=gen, device="cuda").to(dtype)[:, :N]
    dy = torch.randn(M, N + pad, generator=gen, device="cuda").to(dtype)[:, :N]
    return x, ws, b, r, dy


def check_linear(x, w, b, r, act, y, z=None):
    z64, ez = product(x, w)
    if b is not None:
        z64 = z64 + b.double()
        ez = ez + 2.0 ** -23 * z64.abs() + 2.0 ** -23 * b.double().abs()
    y64 = act64(z64, act)[0]
    if r is not None:
        y64 = y64 + r.double()
    tol = 1.2 * ez + 2.0 ** -20 * (1 + z64.abs()) * (act != "none")
    tol = tol + 2.0 ** -23 * (y64.abs() + (0 if r is None else r.double().abs()))
    within(y, y64, tol * 1.01 + half_step(y64, y.dtype), "y")
    if z is not None:
        within(z, z64, ez + 2.0 ** -23 * z64.abs(), "z")


def check_gated(x, wg, wu, act, h):
    g, eg = product(x, wg)
    u, eu = product(x, wu)
    a = act64(g, act)[0]
    ea = 1.2 * eg + 2.0 ** -20 * (1 + g.abs())
    want = a * u
    tol = ea * u.abs() + a.abs() * eu + ea * eu + 2.0 ** -23 * want.abs()
    within(h, want, tol * 1.01 + half_step(want, h.dtype), "h")


def slope_error(dy, z, ez, act):
    """dz = dy act'(z) and how far it may be before its rounding."""
    d = act64(z, act)[1]
    err = 1.2 * ez + 2.0 ** -20 * (1 + z.abs())
    if act == "none":
        err = torch.zeros_like(z)
    if act == "relu":   # the side of zero is decided by the last bits
        err = (z.abs() <= ez).double()
    return dy * d, dy.abs() * err + 2.0 ** -22 * (dy * d).abs()


def check_grads(x, w, dz, edz, dtype, dx=None, dw=None, db=None):
    """Gradients of one weight for dz known within edz."""
    rounded = 1.01 * (edz + half_step(dz, dtype))
    wd, xd = w.double(), x.double()
    if dx is not None:
        want = dz @ wd.t()
        tol = rounded @ wd.abs().t() + dz.shape[1] * 2.0 ** -23 * ((dz.abs() + rounded) @ wd.abs().t())
        within(dx, want, 1.01 * tol + half_step(want, dtype) * 1.01, "dx")
    if dw is not None:
        want = xd.t() @ dz
        tol = xd.abs().t() @ rounded + dz.shape[0] * 2.0 ** -23 * (xd.abs().t() @ (dz.abs() + rounded))
        within(dw, want, 1.01 * tol + half_step(want, dtype) * 1.01, "dw")
    if db is not None:
        want = dz.sum(0)
        tol = edz.sum(0) + dz.shape[0] * 2.0 ** -23 * dz.abs().sum(0)
        within(db, want, 1.01 * tol + half_step(want, dtype) * 1.01, "dbias")


# one token, few, one tile and its neighbours, several tiles, long K, odd everything
SHAPES = [(1, 1, 1), (1, 512, 256), (2, 33, 65), (7, 300, 1000), (16, 256, 4096), (17, 64, 64),
          (33, 130, 127), (64, 128, 64), (65, 129, 257), (128, 256, 512), (129, 384, 96),
          (200, 1000, 72), (257, 255, 333), (300, 640, 1536), (1024, 768, 520)]


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear(shape, dtype, layout):
    M, N, K = shape
    dt = DTYPES[dtype]
    x, (w,), b, r, _ = make(M, N, K, dt, layout)
    check_linear(x, w, None, None, "none", tra.linear(x, w))
    act = ACTS[(M + N + K) % len(ACTS)]
    z = torch.full((M, N), float("nan"), device="cuda")
    y = tra.linear(x, w, bias=b, act=act, residual=r, z=z)
    check_linear(x, w, b, r, act, y, z)


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gated_linear(shape, dtype, layout):
    M, N, K = shape
    x, (wg, wu), _, _, _ = make(M, N, K, DTYPES[dtype], layout, gated=True)
    act = ACTS[(M + N + K) % len(ACTS)]
    check_gated(x, wg, wu, act, tra.gated_linear(x, wg, wu, act=act))


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_every_activation(dtype, act):
    dt = DTYPES[dtype]
    x, ws, b, r, dy = make(96, 200, 64, dt, "nk", seed=3, gated=True)
    x = x * 4      # pre-activations well into both tails
    check_linear(x, ws[0], b, r, act, tra.linear(x, ws[0], b, act, r))
    check_gated(x, ws[0], ws[1], act, tra.gated_linear(x, ws[0], ws[1], act))
    z = torch.empty(96, 200, device="cuda")
    tra.linear(x, ws[0], b, act, z=z)
    dx, dw, db = tra.linear_backward(dy, x, ws[0], z, act, need_dbias=True)
    z64, ez = product(x, ws[0])
    z64 = z64 + b.double()
    ez = ez + 2.0 ** -22 * (z64.abs() + b.double().abs())
    dz, edz = slope_error(dy.double(), z64, ez, act)
    check_grads(x, ws[0], dz, edz, dt, dx, dw, db)


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_linear_gradients(shape, dtype, layout):
    M, N, K = shape
    dt = DTYPES[dtype]
    x, (w,), b, r, dy = make(M, N, K, dt, layout)
    act = ACTS[(M + N + 2 * K) % len(ACTS)]
    leaves = [t.detach().requires_grad_() for t in (x, w, b, r)]
    y = tra.linear(leaves[0], leaves[1], leaves[2], act, leaves[3])
    check_linear(x, w, b, r, act, y.detach())
    dx, dw, db, dr = torch.autograd.grad(y, leaves, dy)
    z64, ez = product(x, w)
    z64 = z64 + b.double()
    ez = ez + 2.0 ** -22 * (z64.abs() + b.double().abs())
    dz, edz = slope_error(dy.double(), z64, ez, act)
    check_grads(x, w, dz, edz, dt, dx, dw, db)
    assert torch.equal(dr, dy)
    assert dw.shape == w.shape and (K == 1 or N == 1 or dw.stride() == w.stride())


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_gated_gradients(shape, dtype, layout):
    M, N, K = shape
    dt = DTYPES[dtype]
    x, (wg, wu), _, _, dy = make(M, N, K, dt, layout, gated=True)
    act = [a for a in ACTS if a != "relu"][(M + N + 2 * K) % (len(ACTS) - 1)]
    leaves = [t.detach().requires_grad_() for t in (x, wg, wu)]
    h = tra.gated_linear(leaves[0], leaves[1], leaves[2], act)
    check_gated(x, wg, wu, act, h.detach())
    dx, dg, du = torch.autograd.grad(h, leaves, dy)
    g, eg = product(x, wg)
    u, eu = product(x, wu)
    a, d = act64(g, act)
    e = 2.0 ** -20 * (1 + g.abs())
    d64 = dy.double()
    zg, zu = d64 * u * d, d64 * a
    eg_ = d64.abs() * ((1.2 * eg + e) * (u.abs() + eu) + eu * d.abs()) + 2.0 ** -22 * zg.abs()
    eu_ = d64.abs() * (1.2 * eg + e) + 2.0 ** -22 * zu.abs()
    check_grads(x, wg, zg, eg_, dt, dw=dg)
    check_grads(x, wu, zu, eu_, dt, dw=du)
    want = zg @ wg.double().t() + zu @ wu.double().t()
    rg, ru = eg_ + half_step(zg, dt), eu_ + half_step(zu, dt)
    tol = rg @ wg.double().abs().t() + ru @ wu.double().abs().t()
    tol = tol + 2 * N * 2.0 ** -23 * ((zg.abs() + rg) @ wg.double().abs().t() +
                                      (zu.abs() + ru) @ wu.double().abs().t())
    within(dx, want, 1.02 * tol + half_step(want, dt) * 1.01, "dx")


@pytest.mark.parametrize("op", ["linear", "gated_linear"])
def test_gradients_against_differences(op):
    # float32 directional differences: the step h loses about 2^-22 |f| / h to
    # rounding and h^2 |f'''| to curvature; with |f| below 40, h = 2^-6 and
    # third derivatives (along unit directions) below 40, 2e-2 bounds both.
    M, N, K = 12, 40, 24
    x, ws, b, _, dy = make(M, N, K, torch.float32, "nk", seed=5, gated=op == "gated_linear")
    leaves = [x, *ws] + ([b] if op == "linear" else [])

    def f(ts):
        y = (tra.linear(ts[0], ts[1], ts[2], "gelu_tanh") if op == "linear"
             else tra.gated_linear(ts[0], ts[1], ts[2], "silu"))
        return (y.double() * dy.double()).sum()

    req = [t.detach().requires_grad_() for t in leaves]
    y = (tra.linear(*req[:2], bias=req[2], act="gelu_tanh") if op == "linear"
         else tra.gated_linear(*req, act="silu"))
    grads = torch.autograd.grad(y, req, dy)
    gen = torch.Generator(device="cuda").manual_seed(9)
    for i, t in enumerate(leaves):
        v = torch.randn(t.shape, generator=gen, device="cuda")
        if t.dim() == 2 and t.stride(0) == 1:     # weights keep their layout
            v = v.t().contiguous().t()
        v = v / v.norm()
        h = 2.0 ** -6
        up = [u if j != i else u + h * v for j, u in enumerate(leaves)]
        dn = [u if j != i else u - h * v for j, u in enumerate(leaves)]
        num = (f(up) - f(dn)) / (2 * h)
        ana = (grads[i].double() * v.double()).sum()
        assert abs(float(num - ana)) <= 2e-2, (i, float(num), float(ana))


# --- exactness, edges and layout ---------------------------------------------------

def ints(shape, lo, hi, gen, dtype):
    return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda").to(dtype)


# every tile class, split and staging: sums of |x w| <= 9 over K stay below
# 2^24, and 64-bit integer sums rounded once are the answer
EXACT = [(1, 520, 4104), (5, 264, 96), (16, 1000, 264), (48, 200, 8), (64, 4096, 1024),
         (70, 136, 2056), (130, 264, 328), (256, 512, 64), (500, 1000, 120), (1000, 1032, 2048),
         (31, 77, 129), (255, 131, 515), (1, 1023, 2047), (3, 2049, 31), (2050, 2056, 136)]


@pytest.mark.parametrize("lib", ["product", "poison"])
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", EXACT, ids=str)
def test_integers_are_exact(shape, dtype, layout, lib, monkeypatch):
    check_integers(shape, dtype, layout, lib, monkeypatch)


def check_integers(shape, dtype, layout, lib, monkeypatch):
    if lib == "poison":
        # every kernel fills its LDS with NaN first
        poisoned = tra.load_poisoned()
        monkeypatch.setattr(fused, "load", lambda: poisoned)
    M, N, K = shape
    dt = DTYPES[dtype]
    gen = torch.Generator(device="cuda").manual_seed(M + N + K)
    x = ints((M, K), -3, 3, gen, dt)
    ws = [ints((K, N) if layout == "kn" else (N, K), -3, 3, gen, dt) for _ in range(2)]
    vs = ws if layout == "kn" else [w.t() for w in ws]
    b, r = ints((N,), -3, 3, gen, dt), ints((M, N), -3, 3, gen, dt)
    p, q = [x.double() @ v.double() for v in vs]
    z = torch.empty(M, N, device="cuda")
    y = tra.linear(x, vs[0], b, "relu", r, z=z)
    assert torch.equal(z.double(), p + b.double())
    assert torch.equal(y, ((p + b.double()).clamp(min=0) + r.double()).to(dt))
    z = torch.empty(M, 2 * N, device="cuda")
    h = tra.gated_linear(x, vs[0], vs[1], "relu", z=z)
    assert torch.equal(z.double(), torch.cat([p, q], 1))
    # the product of two binary32 integers rounds once more on its way to a
    # 16-bit type: in 32 bits first, as the kernel has it
    assert torch.equal(h, (p.clamp(min=0).float() * q.float()).to(dt))
    dy = ints((M, N), -2, 2, gen, dt)
    dx, dw, db = tra.linear_backward(dy, x, vs[0], need_dbias=True)
    assert torch.equal(dx, (dy.double() @ vs[0].double().t()).to(dt))
    assert torch.equal(dw, (x.double().t() @ dy.double()).to(dt))
    assert torch.equal(db, dy.double().sum(0).to(dt))
    # integer gates: relu of small kept values, so that dZ is exact in 16 bits
    kept = ints((M, 2 * N), -2, 2, gen, torch.float32)
    dx, dg, du = tra.gated_linear_backward(dy, x, vs[0], vs[1], kept, "relu")
    zg = dy.double() * kept[:, N:].double() * (kept[:, :N] > 0).double()
    zu = dy.double() * kept[:, :N].double().clamp(min=0)
    assert torch.equal(dx, (zg @ vs[0].double().t() + zu @ vs[1].double().t()).to(dt))
    assert torch.equal(dg, (x.double().t() @ zg).to(dt))
    assert torch.equal(du, (x.double().t() @ zu).to(dt))


# large products with ragged rows and a K tile that ends early, some of which the 256 x
# 256 kernel takes (test_gpu_linear_plans.py has every kernel, and checks that it has)
WIDE = [(4090, 4104, 520), (4090, 520, 4104), (515, 4104, 4088)]


@pytest.mark.parametrize("lib", ["product", "poison"])
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("shape", WIDE, ids=str)
def test_wide_integers_are_exact(shape, dtype, layout, lib, monkeypatch):
    check_integers(shape, dtype, layout, lib, monkeypatch)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("pad", [1, 8, 40])
@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_padded_rows_are_left_alone(layout, pad, dtype):
    dt = DTYPES[dtype]
    M, N, K = 70, 200, 136
    gen = torch.Generator(device="cuda").manual_seed(1)

    def buf(rows, cols):
        t = torch.full((rows + 2, cols + pad), float("nan"), device="cuda", dtype=dt)
        t[:rows, :cols] = torch.randn(rows, cols, generator=gen, device="cuda").to(dt)
        return t, t[:rows, :cols]

    (_, x), (_, r), (ob, out) = buf(M, K), buf(M, N), buf(M, N)
    _, w = buf(K, N) if layout == "kn" else buf(N, K)
    w = w if layout == "kn" else w.t()
    zb = torch.full((M + 1, N + pad), 7.0, device="cuda")
    y = tra.linear(x, w, act="silu", residual=r, out=out, z=zb[:M, :N])
    assert y is out
    check_linear(x, w, None, r, "silu", y, zb[:M, :N])
    assert torch.isnan(ob[:M, N:]).all() and torch.isnan(ob[M:]).all()
    assert (zb[:M, N:] == 7).all() and (zb[M:] == 7).all()


def test_packed_gate_and_up_weights():
    # one K x 2N (2N x K) parameter, as checkpoints often hold it
    x, _, _, _, _ = make(50, 8, 96, torch.bfloat16, "kn")
    gen = torch.Generator(device="cuda").manual_seed(2)
    kn = torch.randn(96, 2 * 128, generator=gen, device="cuda").mul_(0.1).bfloat16()
    for packed, split in ((kn, lambda t: (t[:, :128], t[:, 128:])),
                          (kn.t().contiguous(), lambda t: (t[:128].t(), t[128:].t()))):
        wg, wu = split(packed)
        check_gated(x, wg, wu, "silu", tra.gated_linear(x, wg, wu))
        p = packed.detach().requires_grad_()
        h = tra.gated_linear(x, *split(p))
        (dp,) = torch.autograd.grad(h, p, torch.ones_like(h))
        z = torch.empty(50, 256, device="cuda")
        tra.gated_linear(x, wg, wu, z=z)
        _, dg, du = tra.gated_linear_backward(torch.ones_like(h), x, wg, wu, z)
        want = torch.cat([dg, du], 1)
        assert torch.equal(dp if packed is kn else dp.t(), want)


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_rows_past_32_bit_offsets(dtype):
    # rows 5 GB (and more) into a buffer, for every operand that has rows
    dt = DTYPES[dtype]
    M, N, K, ld = 70000, 72, 64, 40000
    big = torch.empty(M, ld, device="cuda", dtype=dt)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, y = big[:, :K], big[:, 1024:1024 + N]
    x.copy_(ints((M, K), -3, 3, gen, dt))
    w = ints((K, N), -3, 3, gen, dt)
    tra.linear(x, w, out=y)
    want = (x.double() @ w.double()).to(dt)
    assert torch.equal(y, want)
    dx, dw, db = tra.linear_backward(y, x, w, need_dbias=True)
    assert torch.equal(dx, (want.double() @ w.double().t()).to(dt))
    del big, x, y


@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("shape", [(70, 96, 130), (33, 2, 3)], ids=str)
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_rows_of_megabytes(dtype, shape, layout):
    # rows so far apart that a tile's offsets pass 31 bits
    dt = DTYPES[dtype]
    M, N, K = shape
    gen = torch.Generator(device="cuda").manual_seed(7)
    big = torch.empty(256, (1 << 21) + 1, device="cuda", dtype=dt)

    def far(rows, cols, at):
        t = big[:rows, at:at + cols]
        t.copy_(ints((rows, cols), -3, 3, gen, dt))
        return t

    x, dy = far(M, K, 0), far(M, N, 1000)
    ws = [far(K, N, 2000 + 500 * i) if layout == "kn" else far(N, K, 2000 + 500 * i).t()
          for i in range(2)]
    p, q = [x.double() @ w.double() for w in ws]
    assert torch.equal(tra.linear(x, ws[0]), p.to(dt))
    assert torch.equal(tra.gated_linear(x, *ws, act="relu"),
                       (p.clamp(min=0).float() * q.float()).to(dt))
    dx, dw, _ = tra.linear_backward(dy, x, ws[0])
    assert torch.equal(dx, (dy.double() @ ws[0].double().t()).to(dt))
    assert torch.equal(dw, (x.double().t() @ dy.double()).to(dt))


def test_long_k():
    # long enough that no summation order keeps 16-bit products exact: the bound
    for dtype in DTYPES:
        x, (w,), b, r, dy = make(20, 24, 150000, DTYPES[dtype], "nk")
        check_linear(x, w, b, r, "silu", tra.linear(x, w, b, "silu", r))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", [(5, 96, 128), (90, 136, 264), (300, 512, 520)], ids=str)
def test_operands_off_alignment(shape, dtype):
    # every pointer one element past a 16-byte boundary, row lengths aligned
    M, N, K = shape
    dt = DTYPES[dtype]
    gen = torch.Generator(device="cuda").manual_seed(6)

    def off(rows, cols):
        t = torch.randn(rows, cols + 16, generator=gen, device="cuda").to(dt)
        return t[:, 1:cols + 1]

    for layout in ("kn", "nk"):
        x, r = off(M, K), off(M, N)
        w = off(K, N) if layout == "kn" else off(N, K).t()
        b = torch.randn(N + 1, generator=gen, device="cuda").to(dt)[1:]
        out = off(M, N)
        check_linear(x, w, b, r, "gelu", tra.linear(x, w, b, "gelu", r, out=out))
        dy = off(M, N)
        dx, dw, db = tra.linear_backward(dy, x, w, need_dbias=True)
        zero = torch.zeros(M, N, device="cuda", dtype=torch.float64)
        check_grads(x, w, dy.double(), zero, dt, dx, dw, db)


def test_residual_in_place():
    for dt in DTYPES.values():
        x, (w,), b, r, _ = make(130, 192, 64, dt, "nk")
        want = tra.linear(x, w, b, "gelu", r)
        buf = r.clone()
        assert tra.linear(x, w, b, "gelu", buf, out=buf) is buf
        assert torch.equal(buf, want)


@pytest.mark.parametrize("shape", [(0, 8, 8), (8, 0, 8), (8, 8, 0), (0, 0, 0), (1, 8, 0)], ids=str)
def test_empty_sizes(shape):
    M, N, K = shape
    x = torch.ones(M, K, device="cuda").requires_grad_()
    w = torch.ones(K, N, device="cuda").requires_grad_()
    b = torch.full((N,), 2.0, device="cuda").requires_grad_()
    y = tra.linear(x, w, b, "relu")
    assert torch.equal(y, torch.full((M, N), 2.0, device="cuda"))
    dx, dw, db = torch.autograd.grad(y, (x, w, b), torch.ones_like(y))
    assert dx.shape == x.shape and dw.shape == w.shape
    assert not dx.any() or N > 0
    assert torch.equal(dw, torch.zeros_like(dw)) or M > 0
    assert torch.equal(db, torch.full_like(db, float(M)))
    h = tra.gated_linear(x, w, w)
    assert torch.equal(h, torch.zeros(M, N, device="cuda"))
    for g in torch.autograd.grad(h, (x, w), torch.ones_like(h)):
        assert not g.any()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("shape", [(9, 70, 72), (150, 264, 200), (33, 65, 67)], ids=str)
def test_nan_and_inf_stay_in_their_rows(shape, dtype):
    M, N, K = shape
    dt = DTYPES[dtype]
    for layout in ("kn", "nk"):
        x, ws, b, r, _ = make(M, N, K, dt, layout, gated=True)
        want, hwant = tra.linear(x, ws[0], b, "none", r), tra.gated_linear(x, *ws)
        x = x.clone()
        x[3, K - 1] = float("nan")
        x[5, 0] = float("inf")
        got, h = tra.linear(x, ws[0], b, "none", r), tra.gated_linear(x, *ws)
        keep = torch.ones(M, dtype=torch.bool, device="cuda")
        keep[3] = keep[5] = False
        assert torch.equal(got[keep], want[keep]) and torch.equal(h[keep], hwant[keep])
        assert torch.isnan(got[3]).all() and torch.isnan(h[3]).all()
        assert not torch.isfinite(got[5]).any()
        ws[0] = ws[0].clone() if layout == "kn" else ws[0].t().clone().t()
        ws[0][:, 2] = float("nan")
        got = tra.linear(x, ws[0], b, "relu", r)
        assert torch.isnan(got[:, 2]).all()
        ok = torch.ones(N, dtype=torch.bool, device="cuda")
        ok[2] = False
        assert torch.isfinite(got[keep][:, ok]).all()


def test_same_bits_every_time():
    for M, N, K in ((4, 512, 8192), (60, 300, 4096), (700, 512, 2048)):
        x, ws, b, r, dy = make(M, N, K, torch.bfloat16, "kn", gated=True)
        first = tra.gated_linear(x, *ws)
        z = torch.empty(M, N, device="cuda")
        tra.linear(x, ws[0], b, "silu", z=z)
        grads = tra.linear_backward(dy, x, ws[0], z, "silu", need_dbias=True)
        for _ in range(3):
            assert torch.equal(tra.gated_linear(x, *ws), first)
            again = tra.linear_backward(dy, x, ws[0], z, "silu", need_dbias=True)
            assert all(torch.equal(a, g) for a, g in zip(again, grads))


@pytest.mark.parametrize("act", ACTS)
def test_huge_pre_activations_stay_finite(act):
    # values whose squares pass binary32: act and its slope are at their limits
    x = torch.tensor([[1e20], [-1e20], [3e38], [-3e38], [0.0]], device="cuda")
    w = torch.ones(1, 4, device="cuda")
    z = torch.empty(5, 4, device="cuda")
    y = tra.linear(x, w, act=act, z=z)
    want, slope = act64(x.double(), act if act != "gelu_tanh" else "gelu")
    assert torch.equal(y[:, 0], want[:, 0].float())
    dx, _, _ = tra.linear_backward(torch.ones(5, 4, device="cuda"), x, w, z, act)
    assert torch.equal(dx[:4], 4 * slope[:4].float())


# --- streams, graphs, autograd -------------------------------------------------------

def test_written_outputs_are_known_to_autograd():
    # a tensor saved for another gradient and then overwritten is an error, not a
    # wrong gradient
    x, (w,), b, r, _ = make(8, 16, 24, torch.float32, "kn")
    p = torch.ones(8, 16, device="cuda", requires_grad=True)
    saved = torch.randn(8, 16, device="cuda")
    loss = (p * saved).sum()
    tra.linear(x, w, out=saved)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    with pytest.raises(ValueError):
        tra.linear(x, w, out=torch.empty(8, 16, device="cuda", requires_grad=True))
    with pytest.raises(TypeError):
        tra.linear(x, w, z=True)


def test_another_stream():
    x, ws, b, r, _ = make(64, 256, 2048, torch.bfloat16, "nk", gated=True)
    want = tra.gated_linear(x, *ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a = tra.gated_linear(x, *ws, stream=s)
    with torch.cuda.stream(s):
        c = tra.gated_linear(x, *ws)
    s.synchronize()
    assert torch.equal(a, want) and torch.equal(c, want)


def test_captured_step_replays():
    # a forward and its gradients in one graph, a split among them; replayed
    # between other calls, on changing inputs
    M, N, K = 40, 384, 1536
    x, ws, b, r, dy = make(M, N, K, torch.bfloat16, "nk", gated=True)
    wd = torch.randn(N, K, device="cuda").mul_(0.05).bfloat16()

    def step():
        z = torch.empty(M, 2 * N, device="cuda")
        h = tra.gated_linear(x, *ws, z=z)
        y = tra.linear(h, wd, residual=x)
        dh, dwd, _ = tra.linear_backward(y, h, wd)
        return (y, dwd, *tra.gated_linear_backward(dh, x, *ws, z))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(4):
        x.copy_(torch.randn(M, K, device="cuda").bfloat16())
        g.replay()
        tra.linear(x, ws[0], b)          # other work between replays
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step()
        assert all(torch.equal(a, w) for a, w in zip(got, want)), i


def test_graphs_and_streams_side_by_side():
    # two captured graphs and an eager call, all with a split, on three streams at
    # once: each has its own workspace
    M, N, K = 24, 512, 8192
    x, ws, b, r, dy = make(M, N, K, torch.bfloat16, "kn", gated=True)
    xs = [x, x.flip(0).contiguous(), -x]
    want = [tra.gated_linear(t, *ws) for t in xs]
    assert want[0].isfinite().all() and not torch.equal(want[0], want[1])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for t in xs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([tra.gated_linear(t, *ws) for _ in range(8)])
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            eager = [tra.gated_linear(xs[2], *ws) for _ in range(8)]
        torch.cuda.synchronize()
        for got, w in zip([*outs, eager], want):
            assert all(torch.equal(y, w) for y in got)


def test_autograd_is_refused_in_a_capture():
    # (a stand-in for the capture: nothing is recorded on the GPU)
    x, (w,), b, _, _ = make(4, 8, 16, torch.float32, "kn")
    real = torch.cuda.is_current_stream_capturing
    torch.cuda.is_current_stream_capturing = lambda: True
    try:
        with pytest.raises(RuntimeError, match="captured"):
            tra.linear(x.detach().requires_grad_(), w)
        with pytest.raises(RuntimeError, match="captured"):
            tra.gated_linear(x, w, w.detach().clone().requires_grad_())
        tra.linear(x, w)
    finally:
        torch.cuda.is_current_stream_capturing = real


def test_block_of_both():
    # x + down(silu(gate x) * up x): the two operators in a row, with gradients
    M, F, K = 200, 520, 264
    dt = torch.bfloat16
    x, ws, _, _, _ = make(M, F, K, dt, "nk", seed=11, gated=True)
    gen = torch.Generator(device="cuda").manual_seed(12)
    wd = torch.randn(K, F, generator=gen, device="cuda").mul_(F ** -0.5).to(dt).t()
    dy = torch.randn(M, K, generator=gen, device="cuda").to(dt)
    leaves = [t.detach().requires_grad_() for t in (x, *ws, wd)]
    y = tra.linear(tra.gated_linear(*leaves[:3]), leaves[3], residual=leaves[0])
    grads = torch.autograd.grad(y, leaves, dy)
    wide = [t.detach().double().requires_grad_() for t in (x, *ws, wd)]
    g = wide[0] @ wide[1]
    y64 = (g * torch.sigmoid(g) * (wide[0] @ wide[2])) @ wide[3] + wide[0]
    grads64 = torch.autograd.grad(y64, wide, dy.double())
    # three roundings of relative size up to 2^-9 rms each (h or dh, dz, the
    # result), independent over long sums: 3 * 2^-9 in the norm is above each
    for got, want in [(y, y64), *zip(grads, grads64)]:
        got, want = got.detach().double(), want.detach()
        assert float((got - want).norm() / want.norm()) <= 3 * 2.0 ** -9


def test_expanded_and_transposed_output_gradients():
    x, (w,), b, _, _ = make(33, 48, 40, torch.float32, "kn")
    leaves = [t.detach().requires_grad_() for t in (x, w, b)]
    y = tra.linear(*leaves, act="silu")
    full = torch.autograd.grad(y, leaves, torch.ones_like(y), retain_graph=True)
    for got in (torch.autograd.grad(y.sum(), leaves, retain_graph=True),
                torch.autograd.grad(y.t().contiguous().sum(), leaves)):
        assert all(torch.equal(a, f) for a, f in zip(got, full))


@pytest.mark.parametrize("layout", ["kn", "nk"])
def test_saved_tensors_of_other_strides(layout):
    # hooks that hand back what was saved, contiguous: strides of the forward pass
    # no longer hold
    x, ws, b, r, dy = make(40, 48, 72, torch.bfloat16, layout, gated=True, pad=8)
    leaves = [t.detach().requires_grad_() for t in (x, *ws, b)]

    def grads():
        y = tra.linear(leaves[0], leaves[1], leaves[3], "silu")
        h = tra.gated_linear(*leaves[:3])
        return torch.autograd.grad((y, h), leaves, (dy, dy))

    want = grads()
    with torch.autograd.graph.save_on_cpu():
        got = grads()
    assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_one_row_of_any_stride():
    # a row whose own stride is shorter than it, as the transpose of a column has
    x, ws, b, _, _ = make(1, 48, 40, torch.float32, "kn", gated=True)
    col = torch.randn(48, 1, device="cuda")
    assert col.t().stride() == (1, 1)
    leaves = [t.detach().requires_grad_() for t in (x, *ws)]
    for y in (tra.linear(*leaves[:2], act="silu"), tra.gated_linear(*leaves)):
        got = torch.autograd.grad(y, leaves[0], col.t(), retain_graph=True)
        want = torch.autograd.grad(y, leaves[0], col.t().clone(
            memory_format=torch.contiguous_format).as_strided((1, 48), (48, 1)))
        assert torch.equal(got[0], want[0])
    z = torch.empty(1, 48, device="cuda")
    assert torch.equal(tra.linear(col[:40].t(), ws[0], z=z), tra.linear(col[:40].flatten()[None], ws[0]))
    tra.linear_backward(col.t(), x, ws[0], z, "silu")


def test_only_what_is_asked_for():
    x, (w,), b, _, dy = make(20, 24, 32, torch.float32, "kn")
    for i in range(3):
        leaves = [t.detach().requires_grad_(j == i) for j, t in enumerate((x, w, b))]
        y = tra.linear(*leaves, act="gelu")
        (g,) = torch.autograd.grad(y, leaves[i], dy)
        assert g.shape == leaves[i].shape
    y = tra.linear(x.detach().requires_grad_(), w, b)
    with pytest.raises(RuntimeError):
        (g,) = torch.autograd.grad(y.sum(), y.grad_fn.next_functions[0][0].variable,
                                   create_graph=True)
        g.sum().backward()


def test_refusals():
    x, ws, b, r, _ = make(8, 16, 24, torch.bfloat16, "kn", gated=True)
    w = ws[0]
    with pytest.raises(ValueError):
        tra.linear(x, w[:20])
    with pytest.raises(TypeError):
        tra.linear(x, w.float())
    with pytest.raises(TypeError):
        tra.linear(x.double(), w.double())
    with pytest.raises(TypeError):
        tra.linear(x[0], w)
    with pytest.raises(ValueError):
        tra.linear(x.t().contiguous().t(), w)        # x must be row-major
    with pytest.raises(ValueError):
        tra.linear(x, torch.empty(24, 16, 2, device="cuda", dtype=w.dtype)[..., 0])
    with pytest.raises(ValueError):
        tra.linear(x, w, bias=b[:-1])
    with pytest.raises(TypeError):
        tra.linear(x, w, bias=b.float())
    with pytest.raises(ValueError):
        tra.linear(x, w, residual=r[:4])
    with pytest.raises(ValueError):
        tra.linear(x, w, residual=r[:1].expand(8, 16))   # rows overlap
    with pytest.raises(ValueError):
        tra.linear(x, w, out=torch.empty(8, 17, device="cuda", dtype=x.dtype))
    with pytest.raises(tra.TraError):
        tra.linear(x, w, out=x[:, :16])              # the result over an input
    with pytest.raises(TypeError):
        tra.linear(x, w, z=torch.empty(8, 16, device="cuda", dtype=x.dtype))
    with pytest.raises(ValueError):
        tra.linear(x, w.detach().requires_grad_(), out=torch.empty_like(r))
    with pytest.raises(ValueError):
        tra.gated_linear(x, w, ws[1].t().contiguous().t())   # different strides
    with pytest.raises(ValueError):
        tra.linear_backward(r, x, w, None, "silu")
    with pytest.raises(ValueError):
        tra.linear_backward(r[:, :8], x, w)
