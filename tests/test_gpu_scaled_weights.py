"""Weights of one column or one row in every layout that linear takes: scaled_linear takes them
too, with the same bits as a dense one."""
from __future__ import annotations

import pytest
import torch

import tiling_roofline_analysis_amd as tra

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available()


@pytest.mark.parametrize("K,N,strides", [
    (200, 1, (14, 7)), (200, 1, (3, 1)), (200, 1, (1, 1)), (200, 1, (1, 200)), (200, 1, (1, 7)),
    (1, 50, (7, 3)), (1, 50, (50, 1)), (1, 50, (1, 1)), (1, 1, (5, 7)), (1, 1, (0, 0)),
    (2, 1, (14, 7))], ids=str)
def test_single_rows_and_columns(K, N, strides):
    gen = torch.Generator(device="cuda").manual_seed(K)
    x = torch.randn(40, K, generator=gen, device="cuda").bfloat16().requires_grad_()
    dy = torch.randn(40, N, generator=gen, device="cuda").bfloat16()
    dense = torch.randn(K, N, generator=gen, device="cuda").bfloat16()
    w = torch.zeros(4096, device="cuda", dtype=torch.bfloat16).as_strided((K, N), strides)
    w.copy_(dense)
    assert w.stride() == strides and tra.linear(x, w).shape == (40, N)

    def step(w):
        w = w.detach().requires_grad_()
        y = tra.scaled_linear(x, w)
        return [y.detach(), *torch.autograd.grad(y, (x, w), dy),
                *tra.scaled_linear_backward(dy, x, w)[:2], tra.scaled_linear(x.detach(), w.detach())]

    for a, b in zip(step(w), step(dense)):
        assert torch.equal(a, b)
