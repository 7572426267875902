"""The fused linear operators on a stream given by the caller: memory of tensors
dropped after the call, on the GPU.

A stream is kept busy by torch.cuda._sleep, and tensors of the same sizes as the
dropped ones are allocated and filled meanwhile: where the allocator hands out
memory that is still to be read, the results are those of the fill.
"""
from __future__ import annotations

import pytest
import torch

import tiling_roofline_analysis_amd as tra
from test_gpu_linear import make

pytestmark = pytest.mark.gpu

CYCLES = 100_000_000      # about 50 ms


def calls():
    x, ws, b, r, dy = make(64, 256, 192, torch.bfloat16, "kn", gated=True)
    z, zz = torch.randn(64, 256, device="cuda"), torch.randn(64, 512, device="cuda")
    return {
        "linear": (lambda t, s: (tra.linear(*t[:2], bias=t[2], residual=t[3], act="silu",
                                            stream=s),), [x, ws[0], b, r]),
        "linear z out": (lambda t, s: (tra.linear(*t[:2], z=t[2], out=t[3], stream=s),),
                         [x, ws[0], z, torch.empty_like(r)]),
        "gated": (lambda t, s: (tra.gated_linear(*t, stream=s),), [x, *ws]),
        "linear backward": (lambda t, s: tra.linear_backward(*t, "silu", need_dbias=True, stream=s),
                            [dy, x, ws[0], z]),
        "gated backward": (lambda t, s: tra.gated_linear_backward(*t, stream=s),
                           [dy, x, *ws, zz]),
    }


@pytest.mark.parametrize("name", ["linear", "linear z out", "gated", "linear backward",
                                  "gated backward"])
def test_inputs_dropped_after_the_call(name):
    call, tensors = calls()[name]
    want = [t.clone() for t in call(tensors, None)]
    mine = [t.clone() for t in tensors]
    shapes = [(t.shape, t.dtype) for t in mine]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(CYCLES)
    got = call(mine, s)
    del mine
    again = [torch.full(shape, 7.0, device="cuda", dtype=dt) for shape, dt in shapes]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del again


@pytest.mark.parametrize("name", ["linear", "gated", "linear backward", "gated backward"])
def test_results_dropped_while_read(name):
    call, tensors = calls()[name]
    want = [t.clone() for t in call(tensors, None)]
    torch.cuda.synchronize()
    s, current = torch.cuda.Stream(), torch.cuda.current_stream()
    got = call(tensors, s)
    current.wait_stream(s)
    torch.cuda._sleep(CYCLES)
    copies = [t.clone() for t in got]
    shapes = [(t.shape, t.dtype) for t in got]
    del got
    with torch.cuda.stream(s):
        again = [torch.full(shape, 7.0, device="cuda", dtype=dt) for shape, dt in shapes]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(copies, want))
    del again


def test_gradients_recorded_on_a_given_stream():
    x, ws, b, r, dy = make(64, 256, 192, torch.bfloat16, "nk", gated=True)
    leaves = [t.detach().requires_grad_() for t in (x, *ws, b)]

    def grads(s):
        y = tra.linear(*leaves[:2], bias=leaves[3], act="gelu", stream=s)
        h = tra.gated_linear(*leaves[:3], stream=s)
        if s is not None:
            torch.cuda.current_stream().wait_stream(s)
        return torch.autograd.grad((y, h), leaves, (dy, dy))

    want = grads(None)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = grads(s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_the_current_stream_by_name():
    x, (w,), b, _, _ = make(8, 16, 24, torch.float32, "kn")
    assert torch.equal(tra.linear(x, w, b, stream=torch.cuda.current_stream()),
                       tra.linear(x, w, b))


def test_refusals_on_a_stream():
    x, (w,), _, _, _ = make(8, 16, 24, torch.float32, "kn")
    s = torch.cuda.Stream()
    with pytest.raises(TypeError):
        tra.linear(x.cpu(), w.cpu(), stream=s)
    with pytest.raises(TypeError):
        tra.linear([1.0], w, stream=s)
    with pytest.raises(ValueError):
        tra.linear(x, w[:20], stream=s)
    with pytest.raises(TypeError):
        tra.linear(x, w, z=True, stream=s)
