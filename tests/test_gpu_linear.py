"""The linear map on the GPU, forward and backward, against 64-bit products of the same 16-bit inputs.

Bounds, u = 2^-24.  A product of reduction length K is summed in fp32: the matrix core adds 16 products to an
accumulator per instruction and its additions are counted at 2 u each, so an element is within
chain(K) sum |a b|, chain(K) = 2 u (K / 16 + 16 + 16) (the last 16 for the joined splits and the bias), of the exact sum.
Activations: expf, erff and the divisions are within a few ulp, counted as 16 u of the magnitudes they scale; the slope
of gelu and silu is below 1.13, so an error of z reaches y with that factor.  Stored values add half a step of their type.
The backward's dz is rounded to the operands' type before the products, which adds half a step of |dz| times |W| or |x|."""
import pytest
import torch

import token_dispatch_grouped_route_amd as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BOTH = [torch.bfloat16, torch.float16]
ACTS = [None, "relu", "gelu", "silu", "swiglu"]
SLOPE = 1.13   # the largest slope of gelu and silu


@pytest.fixture(autouse=True)
def _free_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def half(t):
    return torch.finfo(t).eps / 2


def stored(v, dtype):
    return half(dtype) * v + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps


def chain(K):
    return 2 * U * (K / 16 + 32)


def act64(z, act):
    F = torch.nn.functional
    if act == "swiglu":
        gate, up = z.chunk(2, -1)
        return F.silu(gate) * up
    return {None: lambda t: t, "relu": F.relu, "gelu": F.gelu, "silu": F.silu}[act](z)


def act_error(z, tol, act):
    """How far the activation of fp32 values within tol of z may be from that of z."""
    if act == "swiglu":
        (gate, up), (tg, tu) = z.chunk(2, -1), tol.chunk(2, -1)
        s = torch.nn.functional.silu(gate).abs()
        return SLOPE * tg * (up.abs() + tu) + s * tu + 16 * U * (gate.abs() * up.abs())
    return SLOPE * tol + (16 * U * z.abs() if act else 0)


def compare(what, got, want, tol):
    got, err = got.double(), (got.double() - want).abs()
    print("[parity] %s %s error / bound %.3g, error / rms %.3g" % (what, tuple(want.shape), (err / tol).nan_to_num().max(), err.max() / want.square().mean().sqrt()))
    assert torch.isfinite(got).all() and (err <= tol).all(), (what, (err / tol).nan_to_num().max())


def make(M, K, N, dtype, act, g, layout="kn", bias=None, residual=None):
    C = 2 * N if act == "swiglu" else N
    x = normal(g, M, K).to(dtype)
    w = (normal(g, K, C) / K ** 0.5).to(dtype)
    if layout == "nk":
        w = w.t().contiguous().t()
    return x, w, (0.3 * normal(g, C)).to(bias) if bias else None, normal(g, M, N).to(residual) if residual else None


def check_forward(x, w, bias, act, residual, out=None, **kw):
    dtype, K = x.dtype, x.shape[-1]
    out = out or dtype
    y, z = moe.linear_forward(x, w, bias, act=act, residual=residual, out_dtype=out, keep=True, **kw)
    assert y.dtype == out and (z is None) == (act is None)
    x64, w64 = x.double(), w.double()
    want, tol = x64 @ w64, chain(K) * (x64.abs() @ w64.abs())
    if bias is not None:
        want = want + bias.double()
        tol = tol + 2 * U * (want.abs() + bias.double().abs())
    if z is not None:
        compare("z", z, want, tol + stored(want.abs() + tol, dtype))
    a, tol = act64(want, act), act_error(want, tol, act)
    if residual is not None:
        a = a + residual.double()
        tol = tol + U * (a.abs() + tol)
    compare("y", y, a, tol + stored(a.abs() + tol, out))
    return y, z


# one row, a few, more than a tile; reductions shorter than a step, between steps and long enough to be split; columns
# that end inside a chunk, a wave's block and a tile
SIZES = [(1, 1, 1), (1, 64, 128), (1, 7168, 512), (2, 5, 3), (3, 33, 17), (4, 4096, 40), (16, 192, 72), (17, 1000, 130), (33, 96, 257), (48, 2048, 300), (64, 130, 64),
         (65, 640, 1000), (127, 63, 127), (128, 128, 128), (129, 65, 129), (200, 2560, 96), (257, 320, 264), (300, 72, 520), (1000, 24, 33), (2100, 136, 1096)]


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("M,K,N", SIZES)
def test_forward(M, K, N, layout, dtype):
    g = gen(M * 31 + K)
    x, w, _, _ = make(M, K, N, dtype, None, g, layout)
    check_forward(x, w, None, None, None)
    check_forward(x, w, None, None, None, out=torch.float32)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,K,N", [(1, 512, 96), (3, 2048, 31), (20, 200, 64), (130, 100, 65), (260, 1024, 128), (140, 4096, 33), (600, 64, 640)])
def test_epilogue(M, K, N, act, dtype):
    """Activation, bias in either type, residual in either type and z, with the weight in both layouts."""
    g = gen(M + N)
    for layout, bias, res in (("kn", dtype, dtype), ("nk", torch.float32, torch.float32), ("kn", None, torch.float32), ("nk", dtype, None)):
        x, w, b, r = make(M, K, N, dtype, act, g, layout, bias, res)
        check_forward(x, w, b, act, r, out=res)


def slope64(z, act, dy):
    z = z.double().requires_grad_()
    return torch.autograd.grad(act64(z, act), z, dy)[0]


def check_backward(dy, x, w, z, act, bias=None):
    dtype, (M, K), C = x.dtype, x.shape, w.shape[1]
    dx, dw, db = moe.linear_backward(dy, x, w, z, act, bias=bias or False)
    assert dx.dtype == dw.dtype == dtype and (dw.stride(0) < dw.stride(1)) == (w.stride(0) < w.stride(1)) and (db is None) == (bias is None)
    dy64 = dy.double()
    if act is None:
        dz, off = dy64, torch.zeros_like(dy64)
    else:
        dz = slope64(z, act, dy64)
        size = dy64.abs()
        if act == "swiglu":
            gate, up = z.double().chunk(2, 1)
            size = torch.cat((size * up.abs() * (1 + gate.abs()), size * gate.abs()), 1)
        else:
            size = size * (1 + z.double().abs())
        off = 16 * U * size
    raw = off
    if act is not None or dy.dtype != dtype:
        off = off + stored(dz.abs() + off, dtype)
    wa, xa = w.double().abs(), x.double().abs()
    tol = (off + chain(C) * (dz.abs() + off)) @ wa.t()
    want = dz @ w.double().t()
    compare("dx", dx, want, tol + stored(want.abs() + tol, dtype))
    tol = xa.t() @ (off + chain(M) * (dz.abs() + off))
    want = x.double().t() @ dz
    compare("dw", dw, want, tol + stored(want.abs() + tol, dtype))
    if bias:
        want, mag = dz.sum(0), dz.abs().sum(0)
        tol = raw.sum(0) + U * (M / 4 + 64) * mag   # a lane's rows, then the runs, in fp32
        compare("db", db, want, tol + stored(want.abs() + tol, bias))


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (1, 256, 64), (5, 33, 17), (64, 128, 128), (130, 200, 65), (300, 520, 264), (1003, 129, 71), (4100, 128, 40), (600, 1096, 640)])
def test_backward(M, K, N, layout, act, dtype):
    g = gen(M + 7 * K)
    for out, bias in ((dtype, torch.float32), (torch.float32, dtype)):
        x, w, _, _ = make(M, K, N, dtype, act, g, layout)
        C = w.shape[1]
        check_backward(normal(g, M, N).to(out), x, w, normal(g, M, C).mul(2).to(dtype) if act else None, act, bias)


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("layout", ["kn", "nk"])
@pytest.mark.parametrize("act", [None, "gelu", "swiglu"])
@pytest.mark.parametrize("M,K,N", [(700, 1001, 515), (300, 1537, 1032), (515, 1280, 777), (129, 4095, 260)])
def test_sizes_that_divide_into_no_chunks(M, K, N, act, layout, dtype):
    """Odd reductions, columns or both, large enough that the operands are copied with padded rows; between NaN."""
    g = gen(K + N)
    x, w, b, r = make(M, K, N, dtype, act, g, "kn", torch.float32, dtype)

    def framed(t):
        box = torch.full((t.shape[0] + 1, t.shape[1] + 3), float("nan"), dtype=t.dtype, device="cuda")
        inner = box[:-1, :-3]
        return inner.copy_(t)

    for x, w in ((x, w if layout == "kn" else w.t().contiguous().t()), (framed(x), framed(w) if layout == "kn" else framed(w.t()).t())):
        y, z = check_forward(x, w, b, act, r)
        assert torch.equal(y, moe.linear_forward(x, w, b, act, r)[0])
        check_backward(normal(g, M, N).to(dtype), x, w, z, act, dtype)


def test_backward_against_differences():
    """d sum(y v) along random directions of x, w, bias and residual, by central differences of the 64-bit formula at
    the run's own inputs: the sum of gradient times direction, within the gradients' rounding (bf16, 2^-9 each of a
    random sum, taken as its 2-norm times 8) and the difference's own error (its step squared)."""
    g = gen(3)
    M, K, N = 70, 96, 48
    for act in ACTS:
        x, w, b, r = make(M, K, N, torch.bfloat16, act, g, "kn", torch.float32, torch.float32)
        ins = [t.clone().requires_grad_() for t in (x, w, b, r)]
        y = moe.linear(*ins[:3], act=act, residual=ins[3], out_dtype=torch.float32)
        v = normal(g, M, N)
        grads = torch.autograd.grad(y, ins, v)
        f = lambda a, c, d, e: ((act64(a @ c + d, act) + e) * v.double()).sum()
        for i, (t, gr) in enumerate(zip(ins, grads)):
            d = normal(g, *t.shape).double()
            base = [s.detach().double() for s in ins]
            h = 1e-5
            step = lambda s: f(*[q + s * h * d if i == j else q for j, q in enumerate(base)])
            # relu's kink: elements within h of 0 are few and small; gelu and silu are smooth
            want, got = (step(1) - step(-1)) / (2 * h), (gr.double() * d).sum()
            tol = 8 * 2.0 ** -8 * (gr.double() * d).norm() + 1e-4 * (gr.double() * d).abs().max()
            assert (got - want).abs() <= tol, (act, i, got, want, tol)


@pytest.mark.parametrize("dtype", BOTH)
def test_strides_offsets_and_surroundings(dtype):
    """Leading dimensions, addresses off the 16 bytes, and NaN around every operand, which must neither be read into a
    result nor be overwritten."""
    g = gen(9)
    for M, K, N, pad, off in ((40, 72, 56, 8, 8), (40, 72, 56, 3, 1), (130, 200, 136, 16, 0), (129, 65, 33, 5, 3), (300, 136, 264, 8, 0), (7, 1024, 520, 24, 0), (2, 250, 90, 7, 1)):
        for layout in ("kn", "nk"):
            def framed(t):
                box = torch.full((t.shape[0] + 2, t.shape[1] + pad), float("nan"), dtype=t.dtype, device="cuda")
                box = box.view(-1)[off:off + (t.shape[0] + 1) * (t.shape[1] + pad)].view(t.shape[0] + 1, -1) if off else box
                inner = box[:t.shape[0], :t.shape[1]]
                inner.copy_(t)
                return inner, box
            x, w, _, r = make(M, K, N, dtype, None, g, "kn", residual=dtype)
            fx, fr = framed(x)[0], framed(r)[0]
            fw = framed(w)[0] if layout == "kn" else framed(w.t().contiguous())[0].t()
            fy, box = framed(torch.zeros(M, N, dtype=dtype, device="cuda"))
            check_forward(fx, fw, None, "silu", fr, y=fy)
            assert torch.equal(fy, moe.linear_forward(fx, fw, None, "silu", fr)[0])   # the same bits on every run
            around = box.clone()
            around[:M, :N] = float("nan")
            assert torch.isnan(around).all()
            fz, fdy = framed(normal(g, M, N).to(dtype))[0], framed(r)[0]
            check_backward(fdy, fx, fw, fz, "silu", torch.float32)


def test_in_place_residual_and_no_rows():
    g = gen(11)
    for M, K, N in ((1, 4096, 64), (50, 64, 100), (300, 512, 256)):
        x, w, b, r = make(M, K, N, torch.bfloat16, None, g, "kn", torch.bfloat16, torch.bfloat16)
        want = moe.linear_forward(x, w, b, residual=r)[0]
        out, _ = moe.linear_forward(x, w, b, residual=r, y=r)
        assert out is r and torch.equal(r, want)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, 32, dtype=torch.bfloat16, device="cuda")
    assert moe.linear_forward(x, w)[0].shape == (0, 32)
    dx, dw, db = moe.linear_backward(x[:, :32], x, w, bias=True)
    assert dx.shape == (0, 64) and not dw.any() and not db.any()


def test_rows_are_independent():
    """A row of NaN or infinity reaches its own row of y alone."""
    g = gen(12)
    for M, K, N in ((5, 256, 64), (40, 512, 64), (300, 192, 320)):
        x, w, b, _ = make(M, K, N, torch.bfloat16, None, g, "kn", torch.bfloat16)
        clean = moe.linear_forward(x, w, b, "relu")[0]
        for bad in (float("nan"), float("inf")):
            x2 = x.clone()
            x2[M // 2, K - 1] = bad
            y = moe.linear_forward(x2, w, b, "relu")[0]
            keep = torch.arange(M, device="cuda") != M // 2
            assert torch.equal(y[keep], clean[keep])
            assert not torch.isfinite(y[M // 2]).all()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", BOTH)
def test_each_gradient_alone(act, dtype):
    """Each gradient asked for by itself has the bits that it has among all three."""
    g = gen(15)
    for M, K, N in ((1, 64, 40), (37, 72, 24), (200, 256, 320)):
        x, w, b, _ = make(M, K, N, dtype, act, g, "kn", dtype)
        dy = normal(g, M, N).to(dtype)
        z = moe.linear_forward(x, w, b, act, keep=True)[1]
        whole = moe.linear_backward(dy, x, w, z, act, bias=True)
        for i, ask in enumerate((dict(dx=True, dw=False), dict(dx=False, dw=True), dict(dx=False, dw=False, bias=True))):
            got = moe.linear_backward(dy, x, w, z, act, **ask)
            assert torch.equal(got[i], whole[i]) and all(t is None for j, t in enumerate(got) if j != i)
    y = moe.linear(x, w, b.requires_grad_(), act=act)   # frozen weights, a trained bias
    y.backward(dy)
    assert torch.equal(b.grad, whole[2])


def test_leading_dimensions_of_x_and_autograd():
    g = gen(13)
    x = normal(g, 3, 7, 64).half().requires_grad_()
    w = (normal(g, 64, 96) / 8).half().requires_grad_()
    b = normal(g, 96).half().requires_grad_()
    r = normal(g, 3, 7, 48).half().requires_grad_()
    y = moe.linear(x, w, b, act="swiglu", residual=r)
    v = normal(g, 48).half()
    y.backward(v.expand(3, 7, 48))   # a gradient that autograd expanded
    z = moe.linear_forward(x, w, b, "swiglu", keep=True)[1]
    want = moe.linear_backward(v.expand(3, 7, 48).contiguous(), x.detach(), w.detach(), z, "swiglu", bias=True)
    for a, c in zip((x.grad, w.grad, b.grad), want):
        assert torch.equal(a, c)
    assert torch.equal(r.grad, v.expand(3, 7, 48))
    y2 = moe.linear(x.detach(), w.detach().requires_grad_(), out_dtype=torch.float32)
    assert y2.dtype == torch.float32 and y2.requires_grad


def test_other_stream_and_graph():
    """On a side stream, and captured and replayed with other inputs and eager work between the replays: the eager
    bits every time (a split reduction, a large one and a backward)."""
    g = gen(14)
    cases = []
    for M, K, N, act in ((2, 4096, 128, "swiglu"), (60, 2048, 256, None), (700, 320, 512, "gelu")):
        x, w, b, r = make(M, K, N, torch.bfloat16, act, g, "kn", torch.bfloat16, torch.bfloat16)
        cases.append((x, w, b, r, act, normal(g, M, N).bfloat16()))

    def step():
        out = []
        for x, w, b, r, act, dy in cases:
            y, z = moe.linear_forward(x, w, b, act, r, keep=True)
            out += [y, *moe.linear_backward(dy, x, w, z, act, bias=True)]
        return out

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
        x, w, b, r, act, _ = cases[0]
    other = moe.linear_forward(x, w, b, act, r, stream=side)[0]
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(other, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for n in range(3):
        for c in cases:
            c[0].copy_(normal(g, *c[0].shape))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in held]
        assert all(torch.equal(a, b) for a, b in zip(kept, step())), n


def test_refusals():
    x, w = torch.ones(4, 64, dtype=torch.bfloat16, device="cuda"), torch.ones(64, 32, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: moe.linear_forward(x.float(), w.float()), lambda: moe.linear_forward(x, w.half()), lambda: moe.linear_forward(x, w[:32]),
                 lambda: moe.linear_forward(x, w, act="tanh"), lambda: moe.linear_forward(x, w[:, :31], act="swiglu"),
                 lambda: moe.linear_forward(x, w, torch.ones(31, dtype=torch.bfloat16, device="cuda")), lambda: moe.linear_forward(x, w, residual=x),
                 lambda: moe.linear_forward(x, w, out_dtype=torch.float16), lambda: moe.linear_forward(x, w[:, ::2]), lambda: moe.linear_forward(x.t(), w),
                 lambda: moe.linear_forward(x, w.cpu()), lambda: moe.linear_forward(x, w, y=x), lambda: moe.linear_forward(torch.ones(4, 8192, dtype=torch.bfloat16, device="cuda"), torch.ones(8192, 32, dtype=torch.bfloat16, device="cuda"), ws=torch.empty(8, dtype=torch.uint8, device="cuda")),
                 lambda: moe.linear_backward(x, x, w), lambda: moe.linear_backward(x[:, :32], x, w, act="gelu"), lambda: moe.linear_backward(x[:, :32].cpu(), x, w)):
        with pytest.raises(moe.MoeError):
            call()
