"""Autograd over an empty batch with frozen weights: the gradient of the rows is an empty tensor."""
import pytest
import torch

import token_dispatch_grouped_route_amd as moe

pytestmark = pytest.mark.gpu


def rows_of_none(dtype=torch.bfloat16, *lead):
    return torch.empty(*lead, 0, 64, dtype=dtype, device="cuda").requires_grad_()


@pytest.mark.parametrize("act", [None, "gelu", "swiglu"])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_linear(act, out):
    w = torch.ones(64, 32, dtype=torch.bfloat16, device="cuda")
    bias = torch.ones(32, dtype=torch.bfloat16, device="cuda")
    for layout in (w, w.t().contiguous().t()):
        for b in (None, bias):
            x = rows_of_none(torch.bfloat16, 3)
            y = moe.linear(x, layout, b, act=act, out_dtype=out)
            assert y.shape == (3, 0, 16 if act == "swiglu" else 32) and y.dtype == out
            y.sum().backward()
            assert x.grad.shape == x.shape and x.grad.dtype == x.dtype
    # with a weight that learns, its gradient is zero
    x, w = rows_of_none(), w.clone().requires_grad_()
    moe.linear(x, w, bias, act=act).sum().backward()
    assert x.grad.shape == x.shape and w.grad.shape == w.shape and not w.grad.any()
