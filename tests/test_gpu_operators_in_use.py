"""quantize, scaled_linear, norm and add_norm as programs call them: from threads, under
saved-tensor hooks and checkpoints, with one tensor in several places, on views."""
from __future__ import annotations

import threading

import pytest
import torch
from torch.utils.checkpoint import checkpoint

import tiling_roofline_analysis_amd as tra

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available()


def normal(*shape, dtype=torch.bfloat16, seed=0, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda").mul_(scale).to(dtype)


def block(x, h, gate, g, w):
    """The join behind a block and the projection after it."""
    r, y = tra.add_norm(x, h, gate, post="rms", kind="layer", weight=g)
    return tra.scaled_linear(y, w.t(), residual=r)


def inputs(M=70, D=520, dtype=torch.bfloat16):
    t = [normal(M, D, dtype=dtype), normal(M, D, dtype=dtype, seed=1),
         normal(D, dtype=dtype, seed=2), normal(D, dtype=dtype, seed=3),
         normal(D, D, dtype=dtype, seed=4, scale=D ** -0.5)]
    return [v.requires_grad_() for v in t], normal(M, D, dtype=dtype, seed=5)


def step(leaves, dy, f=block):
    y = f(*leaves)
    return [y.detach(), *torch.autograd.grad(y, leaves, dy)]


def test_threads_side_by_side():
    cases = [inputs(M, D) for M, D in ((70, 520), (3, 4096), (300, 264), (1, 5000))]
    want = [step(*c) for c in cases]
    got = [None] * len(cases)

    def work(i):
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.default_stream())
        with torch.cuda.stream(stream):
            for _ in range(20):
                got[i] = step(*cases[i])
        stream.synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_saved_tensors_on_the_host_and_in_other_layouts():
    leaves, dy = inputs()
    want = step(leaves, dy)
    with torch.autograd.graph.save_on_cpu():
        got = step(leaves, dy)
    assert all(torch.equal(a, b) for a, b in zip(got, want))

    def padded(t):                # the same values, rows further apart
        if t.dim() != 2 or t.dtype is not torch.bfloat16:
            return t
        wide = t.new_zeros(t.shape[0], t.shape[1] + 24)
        wide[:, :t.shape[1]] = t
        return wide[:, :t.shape[1]]

    with torch.autograd.graph.saved_tensors_hooks(padded, lambda t: t):
        got = step(leaves, dy)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_checkpoint_gives_the_same_bits():
    leaves, dy = inputs(M=300)
    want = step(leaves, dy)
    got = step(leaves, dy, lambda *t: checkpoint(block, *t, use_reentrant=False))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_one_tensor_in_several_places():
    # x is h, and the gate is the weight: the gradients of the places add up
    for D in (300, 5000, 9000):
        x, g = normal(20, D, dtype=torch.float32), normal(D, dtype=torch.float32, seed=1)
        dr, dy = (normal(20, D, dtype=torch.float32, seed=s) for s in (2, 3))
        leaves = [x.clone().requires_grad_(), g.clone().requires_grad_()]
        out = tra.add_norm(leaves[0], leaves[0], leaves[1], post="rms", weight=leaves[1])
        got = torch.autograd.grad(out, leaves, (dr, dy))
        apart = [t.clone().requires_grad_() for t in (x, x, g, g)]
        out = tra.add_norm(apart[0], apart[1], apart[2], post="rms", weight=apart[3])
        dx, dh, dgate, dweight = torch.autograd.grad(out, apart, (dr, dy))
        assert torch.equal(got[0], dx + dh) and torch.equal(got[1], dgate + dweight)
    # x, the residual and, transposed, the weight of one product
    x = normal(264, 264, scale=0.1).requires_grad_()
    y = tra.scaled_linear(x, x.t(), residual=x)
    (got,) = torch.autograd.grad(y, x, torch.ones_like(y))
    a, b, c = (x.detach().clone().requires_grad_() for _ in range(3))
    z = tra.scaled_linear(a, b.t(), residual=c)
    parts = torch.autograd.grad(z, (a, b, c), torch.ones_like(z))
    assert torch.equal(y, z)
    # (the order in which autograd adds the three is its own: two roundings)
    want = sum(p.double() for p in parts)
    size = sum(p.double().abs() for p in parts)
    assert ((got.double() - want).abs() <= 2 * 2.0 ** -8 * 1.01 * size).all()


def test_single_rows_of_any_stride():
    K, N = 400, 130
    x = normal(7, 3, K)
    w, ws = tra.quantize(normal(N, K, scale=0.05), (128, 128))
    for row in (x[3, 1:2], x[2:3, 2], x[0].t().t()[1:2], x[5:6, 0].as_strided((1, K), (1, 1))):
        flat = row.reshape(1, K).clone()
        assert torch.equal(tra.scaled_linear(row, w.t(), None, ws.t()),
                           tra.scaled_linear(flat, w.t(), None, ws.t()))
        assert torch.equal(tra.norm(row), tra.norm(flat))
        for a, b in zip(tra.quantize(row, form="both"), tra.quantize(flat, form="both")):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        q, s = tra.quantize(flat)
        wide = torch.zeros(1, 3 * q.shape[1], dtype=torch.uint8, device="cuda")
        wide[:, q.shape[1]:2 * q.shape[1]] = q.view(torch.uint8)
        part = wide.view(q.dtype)[:, q.shape[1]:2 * q.shape[1]]
        assert torch.equal(tra.scaled_linear(part, w.t(), s, ws.t()),
                           tra.scaled_linear(q, w.t(), s, ws.t()))


def test_no_rows_of_several_sequences():
    g = normal(4, 96).requires_grad_()
    x = normal(0, 96).requires_grad_()
    h = normal(0, 96).requires_grad_()
    r, y = tra.add_norm(x, h, g, weight=g)
    assert r.shape == y.shape == (0, 96)
    grads = torch.autograd.grad((r, y), (x, h, g), (r.detach(), y.detach()))
    assert [t.shape for t in grads] == [(0, 96), (0, 96), (4, 96)]
    assert not grads[2].any()


def test_a_frozen_weight_and_a_frozen_input():
    leaves, dy = inputs()
    want = step(leaves, dy)
    for frozen in range(5):
        some = [t.detach().requires_grad_(i != frozen) for i, t in enumerate(leaves)]
        y = block(*some)
        kept = [t for t in some if t.requires_grad]
        got = torch.autograd.grad(y, kept, dy)
        others = [w for i, w in enumerate(want[1:]) if i != frozen]
        assert torch.equal(y, want[0])
        assert all(torch.equal(a, b) for a, b in zip(got, others))


def test_inference_mode_and_quantized_parameters():
    leaves, _ = inputs()
    q, s = tra.quantize(leaves[4].detach(), (128, 128))
    bias = normal(520, seed=7).requires_grad_()
    with pytest.raises(ValueError, match="quantized weights"):
        tra.scaled_linear(leaves[0].detach(), q.t(), None, s.t(), bias)
    with torch.no_grad():
        want = tra.scaled_linear(leaves[0], q.t(), None, s.t(), bias)
    with torch.inference_mode():
        got = tra.scaled_linear(leaves[0], q.t(), None, s.t(), bias)
        out = torch.empty_like(got)
        tra.scaled_linear(leaves[0], q.t(), None, s.t(), bias, out=out)
        r, y = tra.add_norm(leaves[0], leaves[1])
    assert torch.equal(got, want) and torch.equal(out, want)
    assert torch.equal(y, tra.add_norm(leaves[0].detach(), leaves[1].detach())[1])
