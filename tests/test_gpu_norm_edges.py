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


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("cols", [5, 1000, 7168])
def test_rows_out_of_range_are_nan_and_stay_alone(cols, kind):
    """Infinities, NaN and elements whose squares overflow make their own row NaN, forward and backward."""
    inf = float("inf")
    x = rows_of(gen(cols), 9, cols, torch.float32)
    x[1, 0], x[2, cols - 1], x[3, cols // 2] = inf, -inf, float("nan")
    x[4], x[4, ::2] = 1e25, -2e25
    x[5, 0] = 3e38
    x[6] = 0
    x[7] *= 1e15                       # large, with squares that fit
    bad = torch.zeros(9, dtype=torch.bool, device="cuda")
    bad[1:6] = True
    w = torch.full((cols,), 2.0, device="cuda")
    b = torch.full((cols,), 0.5, device="cuda") if kind == "layer" else None
    y, mean, rstd = moe.norm_forward(x, w, b, kind=kind)
    assert torch.isnan(y[bad]).all() and torch.isnan(rstd[bad]).all()
    check_forward(x[~bad].contiguous(), w, b, kind)
    assert torch.equal(y[~bad], moe.norm_forward(x[~bad].contiguous(), w, b, kind=kind)[0])
    dy = rows_of(gen(1), 9, cols, torch.float32)
    dx, _, _ = moe.norm_backward(dy, x, w, mean, rstd, kind=kind)
    assert torch.isnan(dx[bad]).all() and torch.isfinite(dx[~bad]).all()
    if kind == "rms":
        z = x.to(torch.bfloat16)
        assert torch.isnan(moe.norm_forward(z, kind=kind)[0][bad]).all()


# the first chunk counts (16 bytes of a row each) of every team and every number of chunks a thread takes
CHUNKS = [1] + [n for j in range(3, 13) for n in (2 ** j + 1, 3 * 2 ** (j - 1) + 1)] + [8192]


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("chunks,dtype", [(c, t) for t in (torch.bfloat16, torch.float16, torch.float32) for c in CHUNKS if c * 16 // t.itemsize <= 32768])
def test_every_geometry(chunks, kind, dtype):
    """Each (threads per row, chunks per thread) that a width selects, with several rows per team in the widest."""
    per = 16 // dtype.itemsize
    cols = chunks * per - (0 if chunks == 8192 else per // 2 - 1)
    rows = 600 if chunks > 1024 else 9
    g = gen(chunks)
    x, dy = rows_of(g, rows, cols, dtype), rows_of(g, rows, cols, dtype)
    w = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(dtype)
    b = (0.1 * torch.randn(cols, generator=g, device="cuda")).to(dtype) if kind == "layer" else None
    _, mean, rstd = check_forward(x, w, b, kind)
    check_backward(dy, x, w, mean, rstd, kind, kind == "layer")
