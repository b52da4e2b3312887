"""Row norm on the GPU where its promises are easiest to break: gradients in another type than x's, rows beyond
fp32's range, every geometry that a width selects.  u = 2^-24; the bounds are those of the row norm's other tests."""
import pytest
import torch

import token_dispatch_grouped_route_amd as moe
from test_gpu_norm import check_backward, check_forward, gen, rows_of

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_fp32_bias_without_a_weight_gets_an_fp32_gradient(dtype):
    """The bias's gradient is the column sum in the bias's own type, also where x's type could not hold it."""
    g = gen(21)
    rows, cols = 4001, 200
    x = rows_of(g, rows, cols, dtype)
    up = (30 + torch.randn(rows, cols, generator=g, device="cuda")).to(dtype)      # sums of about 120000
    bias = (0.1 * torch.randn(cols, generator=g, device="cuda")).requires_grad_()
    leaf = x.clone().requires_grad_()
    moe.layer_norm(leaf, None, bias).backward(up)
    want = up.double().sum(0)
    assert bias.grad.dtype == torch.float32
    assert ((bias.grad.double() - want).abs() <= (rows + 8) * U * up.double().abs().sum(0) + U * want.abs()).all()
    _, mean, rstd = moe.norm_forward(x, None, bias.detach())
    _, gw, gb = moe.norm_backward(up, x, None, mean, rstd, bias=torch.float32)
    assert gw is None and torch.equal(gb, bias.grad)
    assert moe.norm_backward(up, x, None, mean, rstd, bias=True)[2].dtype == dtype


def test_a_bias_type_of_its_own_is_refused_beside_a_weight():
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    _, mean, rstd = moe.norm_forward(x, w, w)
    for weight, kind in ((w, torch.float32), (w.float(), torch.bfloat16), (None, torch.float16), (None, torch.float64)):
        with pytest.raises(moe.MoeError):
            moe.norm_backward(x, x, weight, mean, rstd, bias=kind)
    assert moe.norm_backward(x, x, w, mean, rstd, bias=torch.bfloat16)[2].dtype == torch.bfloat16
