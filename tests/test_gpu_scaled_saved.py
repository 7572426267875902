"""What scaled_linear saves for its backward pass, 8-bit values and scales, come back from
saved-tensor hooks in other layouts: the gradients keep their bits, or the pass refuses them."""
from __future__ import annotations

import pytest
import torch

import tiling_roofline_analysis_amd as tra

pytestmark = pytest.mark.gpu

FP8 = (torch.float8_e4m3fn, torch.float8_e5m2)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available()


def leaves_of(M, N, K, dtype, layout):
    gen = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, K, generator=gen, device="cuda").to(dtype).requires_grad_()
    w = torch.randn(N, K, generator=gen, device="cuda").mul_(K ** -0.5).to(dtype)
    w = w.requires_grad_() if layout == "nk" else w.t().contiguous().requires_grad_()
    return x, w, torch.randn(M, N, generator=gen, device="cuda").to(dtype)


def step(x, w, dy, pack=None):
    wt = w.t() if w.shape[1] == x.shape[1] and w.shape[0] == dy.shape[1] else w
    seen = []

    def hook(t):
        back = pack(t)
        seen.append((t.dtype, back.stride() != t.stride()))
        return back

    if pack is None:
        y = tra.scaled_linear(x, wt, grad_dtype=torch.float8_e5m2)
    else:
        with torch.autograd.graph.saved_tensors_hooks(hook, lambda t: t):
            y = tra.scaled_linear(x, wt, grad_dtype=torch.float8_e5m2)
    return torch.autograd.grad(y, (x, w), dy), seen


def within(t, rows, cols, at, ld):
    """t inside a larger tensor, `at` elements from its start, rows `ld` apart."""
    room = torch.zeros(at + rows * ld, dtype=torch.uint8 if t.element_size() == 1 else t.dtype,
                       device=t.device).view(t.dtype)
    return room[at:].as_strided((rows, cols), (ld, 1), at).copy_(t)


def wide(t):
    # rows of values stay 16-byte aligned
    return within(t, *t.shape, 32, t.shape[1] + 48)


def columns(t):
    return within(t.t(), t.shape[1], t.shape[0], 16, t.shape[0] + 16).t()


def scales_in_rows(t):
    return t if t.dtype in FP8 else wide(t)


def scales_in_columns(t):
    return t if t.dtype in FP8 else columns(t)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("layout", ["nk", "kn"])
@pytest.mark.parametrize("size", [(1, 40, 33), (40, 72, 200), (300, 264, 520)], ids=str)
def test_gradients_keep_their_bits(size, layout, dtype):
    x, w, dy = leaves_of(*size, dtype, layout)
    want, _ = step(x, w, dy)
    for pack in (wide, scales_in_rows, scales_in_columns):
        got, seen = step(x, w, dy, pack)
        assert {d for d, _ in seen} >= {torch.float8_e4m3fn, torch.float8_e8m0fnu}
        assert any(other for _, other in seen)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), pack.__name__


def test_layouts_that_the_kernels_do_not_take_are_refused():
    x, w, dy = leaves_of(40, 72, 200, torch.bfloat16, "nk")
    for pack, what in ((lambda t: columns(t) if t.dtype in FP8 else t, "row-major"),
                       (lambda t: within(t, *t.shape, 8, t.shape[1] + 16) if t.dtype in FP8 else t,
                        "16-byte aligned"),
                       (lambda t: within(t, *t.shape, 16, t.shape[1] + 8) if t.dtype in FP8 else t,
                        "16-byte aligned")):
        with pytest.raises(ValueError, match=what):
            step(x, w, dy, pack)
