"""Every kernel instance of the fused linear operators, with every way of splitting it,
on integers, whose sums must come out exactly.

The rows of linear_plans.py; each checks that its operands lead to the plans that it
stands for.  Both builds: in the LDS-poison one every kernel fills its LDS with NaN
first.
"""
from __future__ import annotations

import pytest
import torch

import linear_plans as lp
import tiling_roofline_analysis_amd as tra
from test_gpu_linear import DTYPES, ints
from tiling_roofline_analysis_amd import fused

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def far_rows():
    """A buffer for rows 4 MB apart, for each type when it is wanted."""
    made = {}

    def get(dtype):
        if dtype not in made:
            made.clear()
            made[dtype] = torch.zeros(300, (1 << 22) // (4 if dtype == "f32" else 2) + 1,
                                      device="cuda", dtype=DTYPES[dtype])
        return made[dtype]

    yield get
    made.clear()


@pytest.mark.parametrize("lib", ["product", "poison"])
@pytest.mark.parametrize("row", lp.ROWS, ids=lambda r: "-".join(map(str, r)))
def test_integers_are_exact(row, lib, far_rows, monkeypatch):
    if lib == "poison":
        poisoned = tra.load_poisoned()
        monkeypatch.setattr(fused, "load", lambda: poisoned)
    M, N, K, dtype, layout, gated, pad, far = row
    dt = DTYPES[dtype]
    gen = torch.Generator(device="cuda").manual_seed(M + 3 * N + 7 * K)
    nk = layout == "nk"

    def matrix(rows, cols, size, column):
        ld = lp.pitch(cols, row)
        t = far_rows(dtype)[:, column:] if far else torch.empty(rows, ld, device="cuda", dtype=dt)
        t = t[:rows, :cols]
        t.copy_(ints((rows, cols), -size, size, gen, dt))
        return t

    x, dy = matrix(M, K, 3, 0), matrix(M, N, 2, 1024)
    stored = [matrix(*((N, K) if nk else (K, N)), 3, 2048 + 1024 * i) for i in range(1 + gated)]
    ws = [w.t() for w in stored] if nk else stored
    z = ints((M, N * (1 + gated)), -2, 2, gen, torch.float32)

    # the plans of these operands are the row's
    sizes = [M * N, M * K, N * K, N * K]
    outs = [torch.empty(n, device="cuda", dtype=dt) for n in sizes]
    at = dict(zip(("Y", "dX", "dW", "dW2"), (t.data_ptr() for t in outs)), X=x.data_ptr(),
              dY=dy.data_ptr(), W=ws[0].data_ptr(), W2=ws[-1].data_ptr(), Z=z.data_ptr())
    assert lp.plans(row, at) == lp.plans(row)
    del outs

    if gated:
        h = tra.gated_linear(x, *ws, act="relu")
        p, q = (x.double() @ w.double().contiguous() for w in ws)
        assert torch.equal(h, (p.clamp(min=0).float() * q.float()).to(dt))
        del p, q, h
        dx, *dws = tra.gated_linear_backward(dy, x, *ws, z, "relu")
        g, u = z[:, :N].double(), z[:, N:].double()
        dzs = [dy.double() * u * (g > 0), dy.double() * g.clamp(min=0)]
    else:
        y = tra.linear(x, ws[0], act="relu")
        assert torch.equal(y, (x.double() @ ws[0].double().contiguous()).clamp(min=0).to(dt))
        del y
        dx, *dws = tra.linear_backward(dy, x, ws[0])[:2]
        dzs = [dy.double()]
    want = sum(dz @ w.double().t().contiguous() for dz, w in zip(dzs, ws))
    assert torch.equal(dx, want.to(dt))
    xt = x.double().t().contiguous()
    for dw, dz in zip(dws, dzs):
        assert torch.equal(dw, (xt @ dz).to(dt))
