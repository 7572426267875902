"""norm and add_norm on the GPU against 64 bits, with the bounds of norm_reference.py."""
from __future__ import annotations

import pytest
import torch

import tiling_roofline_analysis_amd as tra
from norm_reference import reference

pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
NAMES = ("x", "h", "gate", "post_weight", "post_bias", "weight", "bias")
GRADS = ("x", "h", "gate", "post_weight", "post_bias", "weight", "bias")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available()


def make(M, D, dtype, params, has=NAMES, groups=1, pad=0, seed=0):
    """Tensors by name (one row of the vectors in "grouped" per sequence), dr and dy."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(rows, cols, to, scale=1.0, mean=0.0):
        t = torch.randn(rows, cols + pad, generator=gen, device="cuda").mul_(scale).add_(mean)
        return t.to(to)[:, :cols]

    t = {"x": normal(M, D, dtype, mean=0.3)}
    if "h" in has:
        t["h"] = normal(M, D, dtype, 0.5, -0.2)
    for name, scale, mean in (("gate", 0.3, 0.6), ("post_weight", 0.2, 1.0), ("post_bias", 0.1, 0),
                              ("weight", 0.2, 1.0), ("bias", 0.1, 0.0)):
        if name in has:
            # every second vector is shared by all sequences
            n = groups if name in ("gate", "weight", "bias") else 1
            v = normal(n, D, params, scale, mean)
            t[name] = v[0] if n == 1 else v
    return t, normal(M, D, dtype, 0.5), normal(M, D, dtype, 0.5)


def forward(t, kind, post, scale):
    if "h" not in t:
        return {"y": tra.norm(t["x"], t.get("weight"), t.get("bias"), kind)}
    args = {k: v for k, v in t.items() if k not in ("x", "h")}
    r, y = tra.add_norm(t["x"], t["h"], scale=scale, post=post, kind=kind, **args)
    return {"r": r} if y is None else {"r": r, "y": y}


def check(got, want, what=""):
    for name, t in got.items():
        near = want[name]
        tol = near.rounded(t.dtype)
        err = (t.double() - near.v).abs()
        bad = ~(err <= tol)
        assert not bad.any(), (f"{what} {name}: {int(bad.sum())} of {bad.numel()} off, worst "
                               f"{float((err / tol).max()):.3g} times what is allowed")


def check_all(M, D, dtype, params, kind, post, scale=1.0, has=NAMES, groups=1, pad=0):
    t, dr, dy = make(M, D, dtype, params, has, groups, pad, seed=M + D)
    if kind == "none":
        t.pop("weight", None), t.pop("bias", None)
    if post == "none":
        t.pop("post_weight", None), t.pop("post_bias", None)
    h = "h" in t
    use_dy = dy if kind != "none" else None
    want = reference(t, kind, post, scale, dr=dr if h else None, dy=use_dy)
    check(forward(t, kind, post, scale), want)
    leaves = {k: v.detach().requires_grad_() for k, v in t.items()}
    outs = forward(leaves, kind, post, scale)
    given = [dr if k == "r" else dy for k in outs]
    grads = torch.autograd.grad(list(outs.values()), list(leaves.values()), given)
    for (name, leaf), g in zip(leaves.items(), grads):
        assert g.shape == leaf.shape and g.dtype == leaf.dtype
    check({"d" + n: g for n, g in zip(leaves, grads)}, want)
    return t, outs, grads


SIZES = [(1, 1), (3, 2), (2, 7), (5, 8), (17, 63), (70, 64), (9, 128), (33, 129), (6, 511),
         (300, 512), (5, 513), (130, 2048), (3, 2049), (7, 4095), (66, 4096), (2, 5461), (3, 8192),
         (5, 8193), (70, 16384), (2, 20011)]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(size, dtype):
    for kind, post in (("rms", "rms"), ("layer", "layer")):
        check_all(*size, DTYPES[dtype], DTYPES[dtype], kind, post, scale=0.75)


@pytest.mark.parametrize("D", [40, 200, 1000, 3001, 9000])
@pytest.mark.parametrize("kind", ["none", "rms", "layer"])
@pytest.mark.parametrize("post", ["none", "rms", "layer"])
def test_kinds(kind, post, D):
    check_all(12, D, torch.bfloat16, torch.float32, kind, post)
    check_all(12, D, torch.float32, torch.float32, kind, post, has=("x", "h"))
    if kind != "none" and post == "none":
        check_all(12, D, torch.float16, torch.float16, kind, post, has=("x", "weight"))
        check_all(12, D, torch.float32, torch.float32, kind, post, has=("x",))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("D", [24, 100, 129, 500, 701, 2048, 2055, 4096, 4097, 6000, 8191])
def test_without_biases(D, dtype):
    # (their gradients' sums are left out of the kernels then)
    has = ("x", "h", "gate", "post_weight", "weight")
    for M in (1, 37, 600 if D < 3000 else 270):
        check_all(M, D, DTYPES[dtype], torch.float32, "rms", "rms", has=has)
    check_all(19, D, DTYPES[dtype], DTYPES[dtype], "layer", "layer", has=has)
    check_all(19, D, DTYPES[dtype], DTYPES[dtype], "layer", "none", has=("x", "h", "gate", "weight"))


@pytest.mark.parametrize("D", [72, 700, 2100, 8200])
@pytest.mark.parametrize("groups,rows", [(2, 1), (3, 5), (4, 70), (130, 2)])
def test_vectors_of_sequences(groups, rows, D):
    if groups * rows * D > 3e6:
        groups = 7
    check_all(groups * rows, D, torch.bfloat16, torch.bfloat16, "layer", "rms", groups=groups)
    check_all(groups * rows, D, torch.float32, torch.float32, "rms", "none", groups=groups)


@pytest.mark.parametrize("pad", [1, 3, 8])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_padded_rows_are_left_alone(dtype, pad):
    dt = DTYPES[dtype]
    for M, D in ((9, 77), (5, 1000), (3, 9001)):
        check_all(M, D, dt, torch.float32, "layer", "rms", pad=pad)
        t, _, _ = make(M, D, dt, dt, pad=pad)
        bufs = [torch.full((M + 1, D + pad), 7.0, device="cuda", dtype=dt) for _ in range(2)]
        r, y = tra.add_norm(t["x"], t["h"], r_out=bufs[0][:M, :D], out=bufs[1][:M, :D])
        want = tra.add_norm(t["x"], t["h"])
        for b, got, w in zip(bufs, (r, y), want):
            assert torch.equal(got, w)
            assert (b[:M, D:] == 7).all() and (b[M:] == 7).all()


def test_residual_stream_in_place():
    for M, D in ((5, 100), (3, 4096), (2, 9001)):
        t, _, _ = make(M, D, torch.bfloat16, torch.bfloat16)
        args = {k: v for k, v in t.items() if k not in ("x", "h")}
        want = tra.add_norm(t["x"], t["h"], post="rms", **args)
        x = t["x"].clone()
        r, y = tra.add_norm(x, t["h"], post="rms", r_out=x, **args)
        assert r is x and torch.equal(x, want[0]) and torch.equal(y, want[1])


def test_many_rows():
    # more rows than one round of workgroups takes
    check_all(70000, 64, torch.bfloat16, torch.float32, "rms", "rms")
    x = torch.randn((1 << 24) + 5, 8, device="cuda")
    y = tra.norm(x, kind="layer")
    want = x.double() - x.double().mean(1, keepdim=True)
    want = want / (want.square().mean(1, keepdim=True) + 1e-6).sqrt()
    assert float((y - want).abs().max()) < 1e-5


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_rows_past_32_bit_offsets(dtype):
    dt = DTYPES[dtype]
    M, D, ld = 70000, 72, 40000
    big = torch.empty(M, ld, device="cuda", dtype=dt)
    x, h, y = big[:, :D], big[:, 100:100 + D], big[:, 1024:1024 + D]
    x.copy_(torch.randn(M, D, device="cuda"))
    h.copy_(torch.randn(M, D, device="cuda"))
    small = x.clone(), h.clone()
    want = tra.add_norm(*small)
    got = tra.add_norm(x, h, out=y)
    assert got[1] is y and all(torch.equal(a, b) for a, b in zip(got, want))
    dx, dh, *_ = tra.add_norm_backward(h, y, x, h)
    wx, wh, *_ = tra.add_norm_backward(small[1], want[1], *small)
    assert torch.equal(dx, wx) and torch.equal(dh, wh)


def test_large_means_cost_a_layer_norm_no_digits():
    # a mean 2^10 times the deviation: squares about it, not their difference.  A value's
    # distance from the mean is exact to u 2^10 of the deviation here, and the mean to
    # steps_of(D) u 2^10; the bounds of check_all hold it to that
    for D in (64, 4096, 9000):
        t, dr, dy = make(20, D, torch.float32, torch.float32, has=("x",))
        t["x"] = t["x"] + 1024.0
        want = reference(t, "layer", dy=dy)
        check({"y": tra.norm(t["x"], kind="layer")}, want)
        check({"dx": tra.norm_backward(dy, t["x"], kind="layer")[0]}, want)


def test_constant_and_zero_rows():
    for D in (5, 600, 9000):
        x = torch.zeros(4, D, device="cuda")
        x[1] = 3.0
        for kind in ("rms", "layer"):
            y = tra.norm(x, kind=kind)
            dx = tra.norm_backward(torch.ones_like(x), x, kind=kind)[0]
            assert torch.isfinite(y).all() and torch.isfinite(dx).all()
            assert not y[0].any()
            if kind == "layer":
                # ones have no part that a layer norm of equal elements lets through; the mean
                # may be off by its roundings, which 1 / sqrt(eps) = 1000 multiplies
                assert float(y.abs().max()) <= 1000 * 3 * (40 + D // 1024) * 2.0 ** -24


@pytest.mark.parametrize("D", [9, 128, 700, 4096, 9001])
def test_nan_and_inf_stay_in_their_rows(D):
    t, dr, dy = make(40, D, torch.float32, torch.float32)
    args = {k: v for k, v in t.items() if k not in ("x", "h")}
    call = lambda x, h: tra.add_norm(x, h, post="rms", kind="layer", **args)  # noqa: E731
    back = lambda x, h: tra.add_norm_backward(dr, dy, x, h, post="rms", kind="layer",  # noqa: E731
                                              **args)[:2]
    want = (*call(t["x"], t["h"]), *back(t["x"], t["h"]))
    x, h = t["x"].clone(), t["h"].clone()
    x[3, D - 1] = float("nan")
    h[17, 0] = float("inf")
    x[39, D // 2] = -float("inf")
    got = (*call(x, h), *back(x, h))
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[[3, 17, 39]] = False
    for a, b in zip(got, want):
        assert torch.equal(a[keep], b[keep])
    assert torch.isnan(got[1][~keep]).all()


@pytest.mark.parametrize("D", [40, 300, 1500, 4000, 9000])
def test_an_infinity_in_the_last_row_is_counted_once(D):
    # (rows are taken several at a time; 0 times it would be NaN)
    t, dr, _ = make(5, D, torch.float32, torch.float32, has=("x", "h", "gate"))
    dr, h = dr.abs() + 1, t["h"].clone()
    h[4, 7] = float("inf")
    dx, dh, dgate = tra.add_norm_backward(dr, None, t["x"], h, t["gate"], kind="none")[:3]
    assert dgate[7] == float("inf")
    assert torch.isfinite(dgate[:7]).all() and torch.isfinite(dgate[8:]).all()
    assert torch.equal(dx, dr) and torch.equal(dh, dr * t["gate"])


@pytest.mark.parametrize("D", [5, 50, 2000, 5461, 9000, 17000])
@pytest.mark.parametrize("post", ["none", "layer"])
def test_an_unused_norm_has_gradients_of_zero(post, D):
    # whatever the rows hold: there is no 0 times an infinity
    t, dr, _ = make(6, D, torch.float32, torch.float32)
    h = t["h"].clone()
    h[2, 1] = float("inf")
    args = {k: v for k, v in t.items() if k not in ("x", "h")}
    if post == "none":
        args.pop("post_weight"), args.pop("post_bias")
    got = tra.add_norm_backward(dr, None, t["x"], h, post=post, kind="rms", **args)
    dweight, dbias = got[5:]
    assert not dweight.any() and not dbias.any()
    assert torch.equal(got[0], dr)


def test_missing_gradients_of_outputs():
    # either output may go unused
    for D in (50, 2000, 9000):
        t, dr, dy = make(10, D, torch.float32, torch.float32)
        leaves = {k: v.detach().requires_grad_() for k, v in t.items()}
        outs = forward(leaves, "rms", "layer", 0.5)
        for used, d in (("r", {"dr": dr}), ("y", {"dy": dy})):
            grads = torch.autograd.grad(outs[used], list(leaves.values()), dr if used == "r" else dy,
                                        retain_graph=True, allow_unused=True)
            want = reference(t, "rms", "layer", 0.5, **d)
            got = {"d" + n: g for n, g in zip(leaves, grads) if "d" + n in want}
            check(got, want, used)
            for n, g in zip(leaves, grads):
                if "d" + n not in want:
                    assert g is None or not g.any()


def test_only_what_is_asked_for():
    t, dr, dy = make(10, 300, torch.bfloat16, torch.float32)
    want = None
    for name in t:
        leaves = {k: v.detach().requires_grad_(k == name) for k, v in t.items()}
        outs = forward(leaves, "layer", "rms", 1.0)
        (g,) = torch.autograd.grad(list(outs.values()), leaves[name], [dr, dy])
        if want is None:
            full = {k: v.detach().requires_grad_() for k, v in t.items()}
            o = forward(full, "layer", "rms", 1.0)
            want = dict(zip(full, torch.autograd.grad(list(o.values()), list(full.values()),
                                                      [dr, dy])))
        assert torch.equal(g, want[name]), name


@pytest.mark.parametrize("D", [5, 700, 4097, 5461, 8192, 9000, 16384, 16392])
def test_rows_without_the_vectors_gradients(D):
    for post in ("none", "layer"):
        t, dr, dy = make(9, D, torch.float32, torch.float32)
        args = {k: v for k, v in t.items() if k not in ("x", "h")}
        if post == "none":
            args.pop("post_weight"), args.pop("post_bias")
        call = lambda **k: tra.add_norm_backward(  # noqa: E731
            dr, dy, t["x"], t["h"], scale=0.75, post=post, kind="layer", **args, **k)
        dx, dh = call()[:2]
        got = call(need_vectors=False)
        assert torch.equal(got[0], dx) and torch.equal(got[1], dh)
        assert all(g is None for g in got[2:])
        assert torch.equal(call(need_dh=False)[0], dx)
        assert torch.equal(call(need_dx=False, need_vectors=False)[1], dh)


def test_gradients_against_differences():
    gen = torch.Generator(device="cuda").manual_seed(3)
    t, dr, dy = make(4, 24, torch.float32, torch.float32, groups=2)
    args = dict(kind="layer", post="rms", scale=0.75)

    def loss(t):
        o = reference({k: v.double() for k, v in t.items()}, **args)
        return float((o["r"].v * dr.double()).sum() + (o["y"].v * dy.double()).sum())

    leaves = {k: v.detach().requires_grad_() for k, v in t.items()}
    outs = forward(leaves, **args)
    grads = torch.autograd.grad(list(outs.values()), list(leaves.values()), [dr, dy])
    for (name, leaf), g in zip(leaves.items(), grads):
        way = torch.randn(leaf.shape, generator=gen, device="cuda", dtype=torch.float64)
        # central differences: off by step^2 / 6 of the third derivative, here below 1e-6,
        # and 2^-53 of the loss over the step
        step = 1e-4
        up, down = ({**t, name: t[name].double() + s * step * way} for s in (1, -1))
        slope = (loss(up) - loss(down)) / (2 * step)
        assert abs(float((g.double() * way).sum()) - slope) < 1e-4 * max(1.0, abs(slope)), name


def test_empty_sizes():
    for M, D in ((0, 8), (4, 0), (0, 0)):
        x = torch.ones(M, D, device="cuda").requires_grad_()
        w = torch.ones(D, device="cuda").requires_grad_()
        r, y = tra.add_norm(x, x.detach(), gate=w, weight=w)
        assert r.shape == y.shape == (M, D)
        dx, dw = torch.autograd.grad((r, y), (x, w), (torch.ones_like(r), torch.ones_like(y)))
        assert dx.shape == (M, D) and dw.shape == (D,) and not dw.any()


def test_same_bits_every_time():
    for M, D in ((700, 128), (300, 1000), (515, 4096), (100, 9000)):
        t, dr, dy = make(M, D, torch.bfloat16, torch.float32)
        args = {k: v for k, v in t.items() if k not in ("x", "h")}
        first = (*tra.add_norm(t["x"], t["h"], post="rms", **args),
                 *tra.add_norm_backward(dr, dy, t["x"], t["h"], post="rms", **args))
        for _ in range(3):
            again = (*tra.add_norm(t["x"], t["h"], post="rms", **args),
                     *tra.add_norm_backward(dr, dy, t["x"], t["h"], post="rms", **args))
            assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_poisoned_lds(monkeypatch):
    import tiling_roofline_analysis_amd.fused as fused
    poisoned = tra.load_poisoned()
    cases = [(9, 100, "rms"), (40, 1000, "layer"), (7, 4096, "rms"), (5, 9001, "layer")]
    want = [check_all(M, D, torch.bfloat16, torch.float32, k, "rms") for M, D, k in cases]
    monkeypatch.setattr(fused, "load", lambda: poisoned)
    for (M, D, k), (_, outs, grads) in zip(cases, want):
        _, o, g = check_all(M, D, torch.bfloat16, torch.float32, k, "rms")
        assert all(torch.equal(o[n], outs[n]) for n in outs)
        assert all(torch.equal(a, b) for a, b in zip(g, grads))


# --- streams, graphs, autograd -------------------------------------------------------

def test_captured_step_replays():
    t, dr, dy = make(70, 1500, torch.bfloat16, torch.float32)
    args = {k: v for k, v in t.items() if k not in ("x", "h")}

    def step():
        r, y = tra.add_norm(t["x"], t["h"], post="rms", **args)
        return (r, y, *tra.add_norm_backward(r, y, t["x"], t["h"], post="rms", **args))

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(4):
        t["x"].copy_(torch.randn(70, 1500, device="cuda").bfloat16())
        g.replay()
        tra.norm(t["h"])                 # other work between replays
        torch.cuda.synchronize()
        got = [a.clone() for a in out]
        assert all(torch.equal(a, w) for a, w in zip(got, step())), i


def test_streams_side_by_side():
    ts = [make(200, 3000, torch.bfloat16, torch.float32, seed=i) for i in range(3)]

    def call(t, s=None):
        (t, dr, dy) = t
        args = {k: v for k, v in t.items() if k not in ("x", "h")}
        return (*tra.add_norm(t["x"], t["h"], post="rms", stream=s, **args),
                *tra.add_norm_backward(dr, dy, t["x"], t["h"], post="rms", stream=s, **args))

    want = [call(t) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ts]
    for _ in range(4):
        got = [call(t, s) for t, s in zip(ts, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_memory_dropped_after_a_call_on_a_stream():
    t, dr, dy = make(64, 500, torch.bfloat16, torch.float32)
    want = [a.clone() for a in tra.add_norm(t["x"], t["h"], weight=t["weight"])]
    mine = {k: v.clone() for k, v in t.items()}
    shapes = [(v.shape, v.dtype) for v in mine.values()]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
    got = tra.add_norm(mine["x"], mine["h"], weight=mine["weight"], stream=s)
    del mine
    again = [torch.full(shape, 7.0, device="cuda", dtype=dt) for shape, dt in shapes]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del again


def test_autograd_is_refused_in_a_capture():
    # (a stand-in for the capture: nothing is recorded on the GPU)
    x = torch.ones(4, 8, device="cuda")
    real = torch.cuda.is_current_stream_capturing
    torch.cuda.is_current_stream_capturing = lambda: True
    try:
        with pytest.raises(RuntimeError, match="captured"):
            tra.norm(x.clone().requires_grad_())
        with pytest.raises(RuntimeError, match="captured"):
            tra.add_norm(x, x, gate=torch.ones(8, device="cuda", requires_grad=True))
        tra.add_norm(x, x)
    finally:
        torch.cuda.is_current_stream_capturing = real


def test_expanded_and_transposed_output_gradients():
    t, dr, dy = make(33, 48, torch.float32, torch.float32)
    leaves = {k: v.detach().requires_grad_() for k, v in t.items()}
    r, y = forward(leaves, "rms", "rms", 1.0).values()
    at = list(leaves.values())
    full = torch.autograd.grad((r, y), at, (torch.ones_like(r), torch.ones_like(y)),
                               retain_graph=True)
    for got in (torch.autograd.grad(r.sum() + y.sum(), at, retain_graph=True),
                torch.autograd.grad(r.t().contiguous().sum() + y.sum(), at)):
        assert all(torch.equal(a, f) for a, f in zip(got, full))


def test_written_outputs_are_known_to_autograd():
    x = torch.randn(8, 16, device="cuda")
    p = torch.ones(8, 16, device="cuda", requires_grad=True)
    saved = torch.randn(8, 16, device="cuda")
    loss = (p * saved).sum()
    tra.norm(x, out=saved)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_refusals():
    x = torch.ones(8, 16, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(16, device="cuda", dtype=torch.bfloat16)
    for error, call in [
            (TypeError, lambda: tra.norm(x[0])),
            (TypeError, lambda: tra.norm(x.double())),
            (TypeError, lambda: tra.norm(x, w.double())),
            (TypeError, lambda: tra.norm(x, w, w.float())),
            (ValueError, lambda: tra.norm(x, w[:8])),
            (ValueError, lambda: tra.norm(x, w.expand(3, 16))),
            (ValueError, lambda: tra.norm(x, w.expand(4, 16))),
            (ValueError, lambda: tra.norm(x, kind="none")),
            (ValueError, lambda: tra.norm(x, kind="batch")),
            (ValueError, lambda: tra.norm(x.t().contiguous().t())),
            (ValueError, lambda: tra.norm(x[:1].expand(8, 16))),
            (TypeError, lambda: tra.add_norm(x, None)),
            (TypeError, lambda: tra.add_norm(x, x.float())),
            (ValueError, lambda: tra.add_norm(x, x[:4])),
            (ValueError, lambda: tra.add_norm(x, x, post_weight=w)),
            (ValueError, lambda: tra.add_norm(x, x, kind="none", weight=w)),
            (TypeError, lambda: tra.add_norm(x, x, scale=w)),
            (ValueError, lambda: tra.add_norm(x, x, gate=w.repeat(2, 1), weight=w.repeat(4, 1))),
            (tra.TraError, lambda: tra.add_norm(x, x, eps=-1.0)),
            (tra.TraError, lambda: tra.add_norm(x, x, eps=float("nan"))),
            (tra.TraError, lambda: tra.norm(x, out=x)),
            (tra.TraError, lambda: tra.add_norm(x, w.repeat(8, 1), out=x)),
            (ValueError, lambda: tra.norm(x, out=x[:4])),
            (ValueError, lambda: tra.norm(x.clone().requires_grad_(), out=torch.empty_like(x)))]:
        with pytest.raises(error):
            call()
