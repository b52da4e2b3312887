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


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_block_norm(kind, stream, post, pre):
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    gate = torch.ones(2, 64, dtype=torch.bfloat16, device="cuda")
    for learns in (False, True):
        x, b = rows_of_none(stream, 2), rows_of_none(torch.bfloat16, 2)
        v = [t.clone().requires_grad_(learns) if t is not None else None for t in (gate, w if post else None, w if pre else None)]
        r, n = moe.block_norm(x, b, v[0], post_weight=v[1], pre_weight=v[2], kind=kind, post=post, pre=pre)
        (r.sum().float() + (n.sum().float() if pre else 0)).backward()
        assert x.grad.shape == x.shape and x.grad.dtype == stream and b.grad.shape == b.shape
        for t in v:
            assert t is None or not learns or (t.grad.shape == t.shape and not t.grad.any())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_row_norm(dtype):
    w = torch.ones(64, dtype=dtype, device="cuda")
    for norm in (lambda x: moe.rms_norm(x, w), lambda x: moe.layer_norm(x, w, w), lambda x: moe.layer_norm(x)):
        x = rows_of_none(dtype)
        norm(x).sum().backward()
        assert x.grad.shape == x.shape and x.grad.dtype == dtype
