"""What the linear map keeps for its backward: x only where the weight learns."""
import pytest
import torch

import token_dispatch_grouped_route_amd as moe

pytestmark = pytest.mark.gpu


def kept(call):
    """The storages that autograd holds for the backward of call()."""
    held = []

    def pack(t):
        held.append(t.untyped_storage().data_ptr())
        return t

    with torch.autograd.graph.saved_tensors_hooks(pack, lambda t: t):
        y = call()
    return held, y


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("by_column", [False, True])
def test_x_is_kept_for_the_weight_alone(act, by_column):
    g = torch.Generator(device="cuda").manual_seed(5)
    make = lambda *shape: torch.randn(*shape, generator=g, device="cuda").bfloat16()
    x, w, bias = make(3, 7, 64), make(64, 48) / 8, make(48)
    w = w.t().contiguous().t() if by_column else w
    grads = {}
    for learns in (True, False):
        a, m, c = x.clone().requires_grad_(), w.clone(memory_format=torch.preserve_format).requires_grad_(learns), bias.clone().requires_grad_()
        held, y = kept(lambda: moe.linear(a, m, c, act=act))
        assert (a.untyped_storage().data_ptr() in held) == learns
        y.backward(torch.ones_like(y))
        grads[learns] = a.grad, c.grad
        assert (m.grad is not None) == learns
    assert all(torch.equal(p, q) for p, q in zip(*grads.values()))


def test_backward_without_x():
    g = torch.Generator(device="cuda").manual_seed(6)
    make = lambda *shape: torch.randn(*shape, generator=g, device="cuda").half()
    x, w, dy = make(70, 96), make(96, 40), make(70, 40)
    want = moe.linear_backward(dy, x, w, bias=True)
    got = moe.linear_backward(dy, None, w, bias=True, dw=False)
    assert got[1] is None and torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
    for call in (lambda: moe.linear_backward(dy, None, w), lambda: moe.linear_backward(dy, None, w.bfloat16(), dw=False), lambda: moe.linear_backward(dy[:, :39], None, w, dw=False),
                 lambda: moe.linear_backward(dy, None, w.cpu(), dw=False), lambda: moe.linear_backward(dy.float().double(), None, w, dw=False)):
        with pytest.raises(moe.MoeError):
            call()
