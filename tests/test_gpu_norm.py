"""Row norm (layer norm, RMS norm) on the GPU against its definition in 64 bits, with bounds counted
from the roundings the kernels make: u = 2^-24 per fp32 operation, half a step of the type per stored
value.  A thread adds at most 32 elements of a row and the team's sums are joined in at most 22 more
additions, so 64 u times the sum of the magnitudes covers every sum over a row."""
import pytest
import torch

import token_dispatch_grouped_route_amd as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
ROW = 64 * U
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


def half(dtype):
    return torch.finfo(dtype).eps / 2


def stored(v, dtype):
    """Rounding of a stored value: half a step relative, or half the smallest subnormal."""
    return half(dtype) * v.abs() + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def rows_of(g, rows, cols, dtype, offset=0.3):
    x = torch.randn(rows, cols, generator=g, device="cuda") * (0.5 + torch.rand(rows, 1, generator=g, device="cuda"))
    return (x + offset * torch.randn(rows, 1, generator=g, device="cuda")).to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ref_forward(x, w, b, eps, kind):
    x = x.double()
    mean = x.mean(-1, keepdim=True) if kind == "layer" else torch.zeros_like(x[..., :1])
    rstd = ((x - mean) ** 2).mean(-1, keepdim=True).add(eps).rsqrt()
    xh = (x - mean) * rstd
    w = w.double() if w is not None else torch.ones_like(xh[..., :1])
    b = b.double() if b is not None else torch.zeros_like(xh[..., :1])
    y = xh * w + b
    # mean off by ROW mean|x|; the centred squares and their sum by at most 50 u relative, so rstd by 30 u
    tol = w.abs() * (ROW * x.abs().mean(-1, keepdim=True) * rstd + ROW * xh.abs()) + 4 * U * ((xh * w).abs() + b.abs())
    return y, mean[..., 0], rstd[..., 0], tol


def check(got, want, tol, what):
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all(), what
    worst = (err / tol.clamp(min=1e-300)).max().item() if err.numel() else 0.0
    print("[parity] %-40s error / bound %.3g" % (what, worst))
    assert (err <= tol).all(), "%s: error / bound %.3g" % (what, worst)


def check_forward(x, w, b, kind, eps=1e-5, **kw):
    y, mean, rstd = moe.norm_forward(x, w, b, eps=eps, kind=kind, **kw)
    ry, rmean, rrstd, tol = ref_forward(x, w, b, eps, kind)
    what = "%s %s %s" % (kind, tuple(x.shape), x.dtype)
    check(y, ry, tol + stored(ry.abs() + tol, x.dtype), what + " y")
    if kind == "layer":
        check(mean, rmean, ROW * x.double().abs().mean(-1) + 1e-40, what + " mean")
    else:
        assert mean is None
    check(rstd, rrstd, ROW * rrstd, what + " rstd")
    return y, mean, rstd


def check_backward(dy, x, w, mean, rstd, kind, bias):
    dx, dw, db = moe.norm_backward(dy, x, w, mean, rstd, kind=kind, bias=bias)
    rows, cols = x.numel() // x.shape[-1], x.shape[-1]
    X, DY = x.double().reshape(-1, cols), dy.double().reshape(-1, cols)
    s = rstd.double().reshape(-1, 1)
    xh = (X - (mean.double().reshape(-1, 1) if mean is not None else 0.0)) * s
    g = DY * (w.double() if w is not None else 1.0)
    c0, c1 = (g * xh).mean(1, keepdim=True), g.mean(1, keepdim=True) * (kind == "layer")
    want = s * (g - c1 - xh * c0)
    # xh is 2 u off, g one; the two row means ROW of the mean magnitude; five more operations on the terms
    mag = g.abs() + c1.abs() + (xh * c0).abs()
    tol = s * (8 * U * mag + ROW * (kind == "layer") * g.abs().mean(1, keepdim=True) + 1.1 * ROW * xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    what = "%s %s %s" % (kind, tuple(x.shape), x.dtype)
    check(dx.reshape(-1, cols), want, tol + stored(want.abs() + tol, x.dtype), what + " dx")
    # a column's sum over the rows: at most one addition per row however they are split, three operations per term
    n = (rows + 8) * U
    if w is not None:
        want, tol = (DY * xh).sum(0), n * (DY * xh).abs().sum(0)
        check(dw, want, tol + stored(want.abs() + tol, w.dtype), what + " dw")
    else:
        assert dw is None
    if bias:
        want, tol = DY.sum(0), n * DY.abs().sum(0)
        wd = w.dtype if w is not None else x.dtype
        check(db, want, tol + stored(want.abs() + tol, wd), what + " db")
    else:
        assert db is None
    return dx, dw, db


# widths around every change of geometry (chunks of 8 or 4 elements; 64 .. 1024 threads), odd ones among them
SIZES = [(1, 1), (3, 2), (5, 7), (2, 8), (70, 63), (9, 512), (300, 513), (17, 1025), (33, 2048), (6, 2051), (21, 4097), (4, 5001),
         (40, 7168), (3, 8192), (2, 8200), (3, 16385), (2, 32768)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norm_forward_and_backward(rows, cols, kind, dtype):
    g = gen(rows * 40009 + cols)
    x, dy = rows_of(g, rows, cols, dtype), rows_of(g, rows, cols, dtype)
    wd = torch.float32 if cols % 2 else dtype
    w = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(wd)
    b = (0.1 * torch.randn(cols, generator=g, device="cuda")).to(wd) if kind == "layer" else None
    _, mean, rstd = check_forward(x, w, b, kind)
    check_backward(dy, x, w, mean, rstd, kind, kind == "layer")


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_without_weight_and_bias(kind):
    g = gen(3)
    x, dy = rows_of(g, 50, 300, torch.bfloat16), rows_of(g, 50, 300, torch.bfloat16)
    _, mean, rstd = check_forward(x, None, None, kind)
    check_backward(dy, x, None, mean, rstd, kind, False)


def test_weight_without_bias_and_bias_without_weight():
    g = gen(4)
    x, dy = rows_of(g, 50, 300, torch.float32), rows_of(g, 50, 300, torch.float32)
    w = torch.randn(300, generator=g, device="cuda")
    _, mean, rstd = check_forward(x, w, None, "layer")
    check_backward(dy, x, w, mean, rstd, "layer", False)
    check_forward(x, None, w, "layer")
    check_backward(dy, x, None, mean, rstd, "layer", True)


@pytest.mark.parametrize("rows", [9000, 70001])
def test_many_rows_per_team(rows):
    """More rows than teams, so every team walks several rows, the last ones unevenly."""
    g = gen(rows)
    x, dy = rows_of(g, rows, 264, torch.bfloat16), rows_of(g, rows, 264, torch.bfloat16)
    w = (1 + 0.2 * torch.randn(264, generator=g, device="cuda")).to(torch.bfloat16)
    b = torch.zeros_like(w)
    _, mean, rstd = check_forward(x, w, b, "layer")
    check_backward(dy, x, w, mean, rstd, "layer", True)


def test_many_long_rows():
    g = gen(8)
    x, dy = rows_of(g, 6200, 2304, torch.bfloat16), rows_of(g, 6200, 2304, torch.bfloat16)
    w = (1 + 0.2 * torch.randn(2304, generator=g, device="cuda")).to(torch.bfloat16)
    _, mean, rstd = check_forward(x, w, None, "rms")
    check_backward(dy, x, w, mean, rstd, "rms", False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [72, 1001, 4099])
def test_strided_and_unaligned_rows(cols, dtype):
    """Rows inside wider ones, starting off every vector boundary; what lies around them stays."""
    g = gen(cols)
    rows, lead = 37, 3
    wide_x, wide_dy = rows_of(g, rows, cols + 9, dtype), rows_of(g, rows, cols + 9, dtype)
    x, dy = wide_x[:, lead:lead + cols], wide_dy[:, 1:1 + cols]
    store = torch.full((rows + 2, cols + 5), 7.0, dtype=dtype, device="cuda")
    y = store[1:1 + rows, lead:lead + cols]
    base = torch.randn(cols + 1, generator=g, device="cuda").to(dtype)
    w = base[1:]   # one element off the allocation's alignment
    got, mean, rstd = check_forward(x, w, w, "layer", y=y)
    assert got.data_ptr() == y.data_ptr()
    around = torch.ones_like(store, dtype=torch.bool)
    around[1:1 + rows, lead:lead + cols] = False
    assert (store[around] == 7.0).all()
    check_backward(dy, x, w, mean, rstd, "layer", True)


def test_higher_dimensions_and_no_rows():
    g = gen(6)
    x = rows_of(g, 24, 200, torch.bfloat16).view(2, 3, 4, 200)
    y, mean, rstd = check_forward(x, None, None, "layer")
    assert y.shape == x.shape and mean.shape == rstd.shape == (2, 3, 4)
    e = torch.empty(0, 200, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(200, dtype=torch.bfloat16, device="cuda")
    y, mean, rstd = moe.norm_forward(e, w, w)
    assert y.shape == (0, 200) and mean.shape == (0,)
    dx, dw, db = moe.norm_backward(e, e, w, mean, rstd, bias=True)
    assert dx.shape == (0, 200) and (dw == 0).all() and (db == 0).all()


def test_special_rows():
    """A constant row (variance 0), a row far from zero, a tiny one, a zero one; NaN and inf stay in their rows."""
    x = torch.zeros(6, 1000, device="cuda")
    x[0] = 3.25
    x[1] = 4096 + torch.arange(1000, device="cuda") % 2
    x[2] = 1e-20 * torch.randn(1000, device="cuda", generator=gen(1))
    x[4, 5], x[5, 999] = float("nan"), float("inf")
    w, b = torch.full((1000,), 2.0, device="cuda"), torch.full((1000,), 0.5, device="cuda")
    y, mean, rstd = moe.norm_forward(x, w, b)
    assert (y[0] == 0.5).all() and (y[3] == 0.5).all() and mean[0] == 3.25
    check_forward(x[:4], w, b, "layer")
    assert torch.isfinite(y[:4]).all() and torch.isnan(y[4]).all() and not torch.isfinite(y[5]).any()
    dx, dw, db = moe.norm_backward(torch.ones_like(x)[:4], x[:4].contiguous(), w, mean[:4].contiguous(), rstd[:4].contiguous(), bias=True)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all() and (db == 4).all()


def test_large_row_offsets():
    """Row offsets past 2^31 elements: two rows far apart in one allocation."""
    base = torch.empty(2 ** 31 + 4096, dtype=torch.bfloat16, device="cuda")
    x = base.as_strided((2, 512), (2 ** 31 + 64, 1))
    x.copy_(rows_of(gen(2), 2, 512, torch.bfloat16))
    w = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    _, mean, rstd = check_forward(x, w, w, "layer")
    check_backward(x, x, w, mean, rstd, "layer", True)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_autograd_against_differences(kind):
    """Directional derivatives of the 64-bit definition by central differences; their truncation is
    estimated from two steps (it is four times as large at the double step)."""
    g = gen(11)
    rows, cols = 13, 333
    args = [rows_of(g, rows, cols, torch.float32), 1 + 0.3 * torch.randn(cols, generator=g, device="cuda")]
    args += [0.1 * torch.randn(cols, generator=g, device="cuda")] if kind == "layer" else []
    leaves = [a.clone().requires_grad_() for a in args]
    out = moe.layer_norm(*leaves) if kind == "layer" else moe.rms_norm(*leaves)
    up = torch.randn(rows, cols, generator=g, device="cuda")
    out.backward(up)

    def f(*a):
        return (ref_forward(a[0], a[1], a[2] if len(a) > 2 else None, 1e-5, kind)[0] * up.double()).sum().item()

    for i, leaf in enumerate(leaves):
        v = torch.randn(leaf.shape, generator=g, device="cuda").double()

        def d(h):
            hi, lo = [a.double() for a in args], [a.double() for a in args]
            hi[i], lo[i] = hi[i] + h * v, lo[i] - h * v
            return (f(*hi) - f(*lo)) / (2 * h)

        got = (leaf.grad.double() * v).sum().item()
        # each gradient element is within 256 u of the sums of magnitudes it is made of; those are at most
        # a few times the magnitudes of up, w and xh, which 8 covers at these sizes (|xh| and |up| below 5)
        slack = 256 * U * 8 * (leaf.grad.double().abs() * v.abs()).sum().item() + 256 * U * v.abs().sum().item() * 8
        assert abs(got - d(1e-4)) <= slack + abs(d(2e-4) - d(1e-4)), (kind, i)


def test_autograd_forms():
    """Expanded and transposed gradients, frozen inputs, leaves of different dtypes."""
    g = gen(12)
    x = rows_of(g, 20, 96, torch.bfloat16)
    w = torch.ones(96, device="cuda", requires_grad=True)
    a = x.clone().requires_grad_()
    moe.layer_norm(a, w).sum().backward()      # an expanded gradient
    assert a.grad.dtype == torch.bfloat16 and w.grad.dtype == torch.float32
    b = x.clone().requires_grad_()
    moe.layer_norm(b, w.detach()).backward(torch.ones(96, 20, dtype=torch.bfloat16, device="cuda").t())
    assert torch.equal(a.grad, b.grad)
    w2 = torch.ones(96, device="cuda", requires_grad=True)
    moe.layer_norm(x, w2).sum().backward()     # x frozen
    assert torch.equal(w.grad, w2.grad)
    gx, gw, gb = moe.norm_backward(x, x, w2.detach(), *moe.norm_forward(x, w2.detach())[1:], bias=True, dweight=False)
    assert gw is None and gx is not None and gb.dtype == torch.float32
    bias = torch.zeros(96, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    moe.layer_norm(x, None, bias).sum().backward()
    assert (bias.grad == 20).all()


def test_same_bits_on_every_run_streams_and_graph_replays():
    g = gen(13)
    x, dy = rows_of(g, 3000, 1408, torch.bfloat16), rows_of(g, 3000, 1408, torch.bfloat16)
    w = (1 + 0.2 * torch.randn(1408, generator=g, device="cuda")).to(torch.bfloat16)

    def both(stream=None):
        y, mean, rstd = moe.norm_forward(x, w, w, stream=stream)
        return [y, mean, rstd, *moe.norm_backward(dy, x, w, mean, rstd, bias=True, stream=stream)]

    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = both(side)
    side.synchronize()
    for a, b in zip(first, other):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = both()
    for n in range(3):
        x.copy_(rows_of(g, 3000, 1408, torch.bfloat16))
        for t in held:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(both(), held):
            assert torch.equal(a, b), n


def test_refusals():
    x = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    stats = torch.ones(4, device="cuda")
    for bad in (lambda: moe.norm_forward(x.cpu(), w), lambda: moe.norm_forward(x, w.cpu()), lambda: moe.norm_forward(x, w[:32]),
                lambda: moe.norm_forward(x, w.half()), lambda: moe.norm_forward(x, w, w.float()), lambda: moe.norm_forward(x.double()),
                lambda: moe.norm_forward(x, w, w, kind="rms"), lambda: moe.norm_forward(x, kind="batch"), lambda: moe.norm_forward(x, eps=-1.0),
                lambda: moe.norm_forward(x, eps=float("nan")), lambda: moe.norm_forward(x.t()), lambda: moe.norm_forward(x, y=x),
                lambda: moe.norm_forward(x[:, :0]), lambda: moe.norm_forward(x[:1].expand(4, 64)),
                lambda: moe.norm_forward(x, y=torch.empty(4, 63, dtype=x.dtype, device="cuda")),
                lambda: moe.norm_forward(torch.ones(1, 32769, device="cuda")),
                lambda: moe.norm_backward(x, x, w, None, stats), lambda: moe.norm_backward(x, x, w, stats[:3], stats),
                lambda: moe.norm_backward(x[:3], x, w, stats, stats), lambda: moe.norm_backward(x.float(), x, w, stats, stats),
                lambda: moe.norm_backward(x, x, w, None, stats, kind="rms", bias=True)):
        with pytest.raises(moe.MoeError):
            bad()
