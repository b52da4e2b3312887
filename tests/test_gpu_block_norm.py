"""The block norm on the GPU, forward and backward, against its formulas in 64 bits.

Bounds, u = 2^-24: a sum over a row is formed in fp32 from at most 64 elements a thread, then over lanes and waves, and its
magnitudes are counted with S = 140 u for sums, their means and what follows from them; single operations with u each
(E = 8 u for a handful).  Errors are carried through the formulas to first order, elementwise.  A sum over the rows goes
through at most R / 16 + 64 additions.  Stored values add half a step of their type."""
import itertools

import pytest
import torch

import token_dispatch_grouped_route_amd as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
S, E = 140 * U, 8 * U
DTYPES = [torch.bfloat16, torch.float16, torch.float32]
NAMES = ("dx", "db", "dgate", "dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias")


@pytest.fixture(autouse=True)
def _free_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def stored(v, dtype):
    fi = torch.finfo(dtype)
    return fi.eps / 2 * v + fi.smallest_normal * fi.eps


def compare(what, got, want, tol):
    err = (got.double() - want).abs()
    print("[parity] %s %s error / bound %.3g" % (what, tuple(want.shape), (err / tol).nan_to_num().max()))
    assert torch.isfinite(got).all() and (err <= tol).all(), (what, (err / tol).nan_to_num().max())


class Case:
    def __init__(self, rows, cols, dtype, seed, kind="rms", stream=None, vectors=None, post=True, pre=True, gate=1, bias=True, x_scale=1.0, scale=1.0, bare=False):
        g = gen(seed)
        self.kind, self.post_on, self.pre_on, self.x_scale, self.scale = kind, post, pre, x_scale, scale
        vd, st = vectors or dtype, stream or dtype
        sized = lambda: normal(g, rows, cols) * (0.5 + 2 * torch.rand(rows, 1, generator=g, device="cuda")) + 0.3 * normal(g, rows, 1)
        self.x, self.b = sized().to(st), sized().to(dtype)
        vec = lambda on: (None if bare else (1 + 0.2 * normal(g, cols)).to(vd), (0.3 * normal(g, cols)).to(vd) if kind == "layer" and bias else None) if on else None
        self.post, self.pre = vec(post), vec(pre)
        self.gate = (0.5 + 0.3 * normal(g, *((cols,) if gate == 1 else (gate, cols)))).to(vd) if gate else None
        self.dr, self.dn = normal(g, rows, cols).to(st), normal(g, rows, cols).to(dtype) if pre else None
        self.how = {"kind": kind, "post": self.post, "gate": self.gate, "pre": self.pre, "x_scale": x_scale, "scale": scale}

    def gates(self):
        if self.gate is None:
            return torch.ones(1, 1, dtype=torch.float64, device="cuda")
        g = self.gate.double()
        return g if g.dim() == 1 else g.repeat_interleave(len(self.x) // len(g), 0)

    def forward(self, eps=1e-5):
        return moe.block_norm_forward(self.x, self.b, eps=eps, **self.how)


def wide(wb):
    return [t.double() if t is not None else d for t, d in zip(wb, (1.0, 0.0))]


def norm64(v, ev, kind, eps):
    """N(v), its mean and rstd, and bounds on their errors, from v known within ev."""
    mean = v.mean(1, keepdim=True) if kind == "layer" else torch.zeros(len(v), 1, dtype=torch.float64, device=v.device)
    em = (ev.mean(1, keepdim=True) + S * v.abs().mean(1, keepdim=True)) if kind == "layer" else torch.zeros_like(mean)
    c = v - mean
    var = (c * c).mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    ec = ev + em + U * v.abs()
    er = 0.5 * rstd ** 3 * ((2 * c.abs() * ec + ec * ec).mean(1, keepdim=True) + S * var) + E * rstd
    return c * rstd, mean, rstd, ec * rstd + c.abs() * er + E * (c * rstd).abs(), em + E * mean.abs(), er


def check_forward(c, got, eps=1e-5):
    r, n, stats = got
    b, x = c.b.double(), c.x.double()
    p, ep = b, torch.zeros_like(b)
    if c.post is not None:
        w, bias = wide(c.post)
        h, mean, rstd, eh, em, er = norm64(b, ep, c.kind, eps)
        p = h * w + bias
        ep = eh * (w if isinstance(w, float) else w.abs()) + E * (p.abs() + (h * w).abs())
        compare("post_rstd", stats[1], rstd[:, 0], er[:, 0] + U * rstd[:, 0])
        if c.kind == "layer":
            compare("post_mean", stats[0], mean[:, 0], em[:, 0] + 1e-30)
    u = c.scale * c.gates() * p
    want = c.x_scale * x + u
    er_ = (c.scale * c.gates()).abs() * ep + E * (u.abs() + (c.x_scale * x).abs())
    assert r.dtype == c.x.dtype and (n is None) == (c.pre is None)
    compare("r", r, want, er_ + stored(want.abs() + er_, r.dtype))
    if c.pre is not None:
        w, bias = wide(c.pre)
        h, mean, rstd, eh, em, er = norm64(want, er_, c.kind, eps)
        n64 = h * w + bias
        en = eh * (w if isinstance(w, float) else w.abs()) + E * (n64.abs() + (h * w).abs())
        assert n.dtype == c.b.dtype
        compare("n", n, n64, en + stored(n64.abs() + en, n.dtype))
        compare("pre_rstd", stats[3], rstd[:, 0], er[:, 0] + U * rstd[:, 0])
        if c.kind == "layer":
            compare("pre_mean", stats[2], mean[:, 0], em[:, 0] + 1e-30)
    for t, there in zip(stats, (c.post is not None and c.kind == "layer", c.post is not None, c.pre is not None and c.kind == "layer", c.pre is not None)):
        assert (t is not None) == there


def back64(g, eg, h, rstd, kind):
    """N'(g) and its bound, from g known within eg."""
    mean = lambda v: v.mean(1, keepdim=True)
    m0 = mean(g) if kind == "layer" else torch.zeros(len(g), 1, dtype=torch.float64, device=g.device)
    e0 = mean(eg) + S * mean(g.abs()) if kind == "layer" else m0
    m1, e1 = mean(g * h), mean(eg * h.abs()) + S * mean((g * h).abs())
    out = rstd * (g - m0 - h * m1)
    return out, rstd * (eg + e0 + h.abs() * e1) + E * rstd * (g.abs() + m0.abs() + (h * m1).abs())


def check_backward(c, r, stats, dr, dn, want=None, got=None):
    rows, cols = c.b.shape
    got = got or moe.block_norm_backward(dr, dn, r, c.b, stats, **c.how, **({"want": want} if want else {}))
    got = dict(zip(NAMES, got))
    col = lambda t: t.double()[:, None] if t is not None else torch.zeros(rows, 1, dtype=torch.float64, device="cuda")
    over = (rows / 16 + 64) * U
    expect = {}
    t = dr.double() if dr is not None else torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
    et = torch.zeros_like(t)
    if c.pre is not None:
        d = dn.double() if dn is not None else torch.zeros_like(t)
        w, bias = wide(c.pre)
        h, rstd = (r.double() - col(stats[2])) * col(stats[3]), col(stats[3])
        g = d * w
        back, eb = back64(g, U * g.abs(), h, rstd, c.kind)
        t, et = t + back, eb + E * (t.abs() + back.abs())
        if c.pre[0] is not None:
            expect["dpre_weight"] = (d * h).sum(0), (over + E) * (d * h).abs().sum(0)
        if c.pre[1] is not None:
            expect["dpre_bias"] = d.sum(0), over * d.abs().sum(0)
    expect["dx"] = c.x_scale * t, abs(c.x_scale) * et + E * (c.x_scale * t).abs()
    p = h = c.b.double()
    if c.post is not None:
        w, bias = wide(c.post)
        rstd = col(stats[1])
        h = (p - col(stats[0])) * rstd
        p = h * w + bias
    t, et = c.scale * t, abs(c.scale) * et + E * (c.scale * t).abs()
    gates = c.gates()
    if c.gate is not None:
        shape = (max(1, len(c.gate) if c.gate.dim() == 2 else 1), -1, cols)
        mag = et * p.abs() + E * t.abs() * (p.abs() + h.abs()) + over * (t * p).abs()
        expect["dgate"] = (t * p).view(shape).sum(1).view(c.gate.shape), mag.view(shape).sum(1).view(c.gate.shape)
    dp, edp = t * gates, et * gates.abs() + E * (t * gates).abs()
    if c.post is not None:
        if c.post[0] is not None:
            expect["dpost_weight"] = (dp * h).sum(0), (edp * h.abs() + (over + E) * (dp * h).abs()).sum(0)
        if c.post[1] is not None:
            expect["dpost_bias"] = dp.sum(0), (edp + over * dp.abs()).sum(0)
        # the post norm's means are formed from sums of the parts of t, whose magnitudes are counted one by one
        parts = torch.zeros_like(t)
        if dr is not None:
            parts = parts + dr.double().abs()
        if c.pre is not None and dn is not None:
            d, w2 = dn.double(), wide(c.pre)[0]
            h2, r2 = (r.double() - col(stats[2])) * col(stats[3]), col(stats[3])
            g = d * w2
            m0 = g.mean(1, keepdim=True).abs() if c.kind == "layer" else 0.0
            parts = parts + r2 * (g.abs() + m0 + h2.abs() * (g * h2).mean(1, keepdim=True).abs())
        parts = parts * (c.scale * gates).abs()
        aw = w if isinstance(w, float) else w.abs()
        extra = S * ((parts * aw).mean(1, keepdim=True) + h.abs() * (parts * aw * h.abs()).mean(1, keepdim=True))
        db, edb = back64(dp * w, edp * aw + E * (dp * w).abs(), h, rstd, c.kind)
        expect["db"] = db, edb + rstd * extra
    else:
        expect["db"] = dp, edp
    for name in NAMES:
        there = name in expect and (want is None or name[1:] in want)
        assert (got[name] is not None) == there, name
        if there:
            v, tol = expect[name]
            compare(name, got[name], v, tol + stored(v.abs() + tol, got[name].dtype))


def run(c):
    f = c.forward()
    check_forward(c, f)
    check_backward(c, f[0], f[2], c.dr, c.dn)
    return f


SIZES = [(1, 1), (1, 7168), (2, 8), (3, 33), (5, 128), (7, 129), (70, 600), (9, 1024), (40, 400), (16, 512), (17, 513), (63, 1000), (33, 2048), (9, 2049), (20, 4095), (12, 5001), (6, 8192), (11, 8200), (5, 12289), (4, 16384),
         (3, 20000), (2, 32768), (1500, 96), (4100, 200)]


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_sizes(rows, cols, dtype, kind):
    run(Case(rows, cols, dtype, rows + cols, kind))


@pytest.mark.parametrize("dtype,stream,vectors", [(torch.bfloat16, torch.float32, None), (torch.bfloat16, None, torch.float32), (torch.float16, torch.float32, torch.float32),
                                                  (torch.float16, torch.float32, torch.float16)])
@pytest.mark.parametrize("rows,cols", [(1, 64), (40, 1000), (37, 7168), (9, 16384), (3, 20001)])
def test_types(rows, cols, dtype, stream, vectors):
    for kind in ("rms", "layer"):
        run(Case(rows, cols, dtype, rows, kind, stream, vectors, x_scale=1.7, scale=-0.3))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(24, 320), (130, 3000)])
def test_parts(rows, cols, dtype):
    """Every choice of norms, gate, weights and biases."""
    for post, pre, gate, bare, kind, bias in itertools.product((0, 1), (0, 1), (0, 1), (0, 1), ("rms", "layer"), (0, 1)):
        run(Case(rows, cols, dtype, 7, kind, None, None, bool(post), bool(pre), gate, bool(bias), bare=bool(bare)))


@pytest.mark.parametrize("rows,gate", [(12, 12), (12, 4), (1, 1), (60, 3), (1003, 17), (900, 300), (2000, 2), (4096, 4096), (4096, 64), (3000, 5)])
def test_gates(rows, gate):
    for cols, dtype, stream in ((264, torch.bfloat16, None), (700, torch.float32, None), (8200, torch.float16, torch.float32)):
        if rows * cols < 12e6:
            c = Case(rows, cols, dtype, rows + gate, "layer", stream, gate=2)   # a gate of its own shape follows
            c.gate = (0.5 + 0.3 * normal(gen(gate), gate, cols)).to(dtype)
            c.how["gate"] = c.gate
            run(c)


def test_one_gradient_alone():
    """dr or dn alone, and each gradient without the others: what is asked for does not change it."""
    for dtype, rows, cols in ((torch.bfloat16, 50, 1200), (torch.float32, 21, 9000)):
        c = Case(rows, cols, dtype, 3, "layer", gate=1)
        r, _, stats = c.forward()
        check_backward(c, r, stats, c.dr, None)
        check_backward(c, r, stats, None, c.dn)
        every = dict(zip(NAMES, moe.block_norm_backward(c.dr, c.dn, r, c.b, stats, **c.how)))
        for name in NAMES:
            one = moe.block_norm_backward(c.dr, c.dn, r, c.b, stats, want=(name[1:],), **c.how)
            for n, t in zip(NAMES, one):
                assert (t is not None) == (n == name)
                if t is not None:
                    assert torch.equal(t, every[n]), n


def test_autograd_against_differences():
    """Directional derivatives of sum(r v) + sum(n u) by central differences of the 64-bit formula, fp32 throughout: within
    fp32's rounding of the gradients (counted at 1e-5 of the sum of magnitudes) and the difference's own error."""
    g = gen(5)
    R, C, G = 12, 96, 3
    for kind, bias in (("rms", False), ("layer", True)):
        leaves = {"x": normal(g, R, C), "b": normal(g, R, C), "gate": normal(g, G, C), "post_weight": normal(g, C), "post_bias": normal(g, C) if bias else None,
                  "pre_weight": normal(g, C), "pre_bias": normal(g, C) if bias else None}
        leaves = {k: t.requires_grad_() if t is not None else None for k, t in leaves.items()}
        v, u = normal(g, R, C), normal(g, R, C)
        r, n = moe.block_norm(**leaves, kind=kind, x_scale=0.8, scale=1.3)
        there = [k for k, t in leaves.items() if t is not None]
        grads = torch.autograd.grad([r, n], [leaves[k] for k in there], [v, u])

        def f(d):
            def norm(t, w, c):
                m = t.mean(1, keepdim=True) if kind == "layer" else 0.0
                return (t - m) * ((t - m).square().mean(1, keepdim=True) + 1e-5).rsqrt() * w + (c if c is not None else 0.0)
            p = norm(d["b"], d["post_weight"], d["post_bias"])
            r = 0.8 * d["x"] + 1.3 * d["gate"].repeat_interleave(R // G, 0) * p
            return (r * v.double()).sum() + (norm(r, d["pre_weight"], d["pre_bias"]) * u.double()).sum()

        base = {k: t.detach().double() if t is not None else None for k, t in leaves.items()}
        for k, gr in zip(there, grads):
            d = normal(g, *gr.shape).double()
            h = 1e-5
            diff = (f({**base, k: base[k] + h * d}) - f({**base, k: base[k] - h * d})) / (2 * h)
            assert (diff - (gr.double() * d).sum()).abs() <= 1e-5 * (gr.double() * d).abs().sum() + 1e-6 * diff.abs() + 1e-6, (kind, k)


def test_strides_surroundings_and_in_place():
    g = gen(8)
    for dtype, stream, rows, cols, pad, off in ((torch.bfloat16, torch.bfloat16, 30, 500, 3, 1), (torch.float16, torch.float32, 41, 1032, 8, 8), (torch.float32, torch.float32, 7, 9001, 2, 1)):
        c = Case(rows, cols, dtype, 4, "layer", stream, gate=1)
        want = c.forward()
        framed = lambda t: torch.full((t.shape[0] + 2, cols + pad), float("nan"), dtype=t.dtype, device="cuda").view(-1)[off:off + (rows + 1) * (cols + pad)].view(rows + 1, -1)
        x, b, r, n, dr, dn = (framed(t) for t in (c.x, c.b, c.x, c.b, c.dr, c.dn))
        for box, t in ((x, c.x), (b, c.b), (dr, c.dr), (dn, c.dn)):
            box[:rows, :cols] = t
        inner = lambda box: box[:rows, :cols]
        moe.block_norm_forward(inner(x), inner(b), r=inner(r), n=inner(n), **c.how)
        for box, t in ((r, want[0]), (n, want[1])):
            assert torch.equal(inner(box), t)
            box = box.clone()
            inner(box).fill_(float("nan"))
            assert torch.isnan(box).all()
        for a, e in zip(moe.block_norm_backward(inner(dr), inner(dn), inner(r), inner(b), want[2], **c.how), moe.block_norm_backward(c.dr, c.dn, want[0], c.b, want[2], **c.how)):
            assert torch.equal(a, e)
        moe.block_norm_forward(inner(x), c.b, r=inner(x), **c.how)   # in place
        assert torch.equal(inner(x), want[0])


def test_rows_are_independent_and_not_finite_ones_show():
    for dtype, cols in ((torch.bfloat16, 600), (torch.float32, 5000)):
        c = Case(9, cols, dtype, 6, "rms", gate=1)
        r, n, stats = c.forward()
        clean = moe.block_norm_backward(c.dr, c.dn, r, c.b, stats, **c.how)
        keep = torch.arange(9, device="cuda") != 4
        for bad in (float("nan"), float("inf"), -float("inf")):
            b = c.b.clone()
            b[4, cols - 1] = bad
            r2, n2, stats2 = moe.block_norm_forward(c.x, b, **c.how)
            assert torch.equal(r2[keep], r[keep]) and torch.equal(n2[keep], n[keep])
            assert torch.isnan(r2[4]).all() and torch.isnan(n2[4]).all() and torch.isnan(stats2[1][4])
            g = moe.block_norm_backward(c.dr, c.dn, r2, b, stats2, **c.how)
            assert torch.equal(g[0][keep], clean[0][keep]) and torch.equal(g[1][keep], clean[1][keep])
            assert torch.isnan(g[1][4]).all()


def test_no_rows():
    x = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    r, n, stats = moe.block_norm_forward(x, x, kind="layer", post=(w, w), gate=w[None].expand(2, 64).contiguous(), pre=(w, w))
    assert r.shape == n.shape == (0, 64)
    g = moe.block_norm_backward(x, x, r, x, stats, kind="layer", post=(w, w), gate=w[None].expand(2, 64).contiguous(), pre=(w, w))
    assert g[0].shape == (0, 64) and g[2].shape == (2, 64) and not any(t.any() for t in g[2:])


def test_other_stream_and_graph():
    c, d = Case(70, 900, torch.bfloat16, 2, "rms", torch.float32, gate=1), Case(70, 9000, torch.bfloat16, 2, "layer", gate=2)

    def step():
        out = []
        for k in (c, d):
            r, n, stats = k.forward()
            out += [r, n, *(t for t in moe.block_norm_backward(k.dr, k.dn, r, k.b, stats, **k.how) if t is not None)]
        return out

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for n in range(3):
        c.x.normal_(generator=gen(n))
        d.dn.normal_(generator=gen(n + 9))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in held]
        assert all(torch.equal(a, b) for a, b in zip(kept, step())), n


def test_refusals():
    x = torch.ones(6, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    f = moe.block_norm_forward
    for call in (lambda: f(x, x.half()), lambda: f(x.half(), x), lambda: f(x, x[:5]), lambda: f(x, x, kind="rms", post=(w, w)), lambda: f(x, x, kind="max", post=(w, None)),
                 lambda: f(x, x, post=(w[:60], None)), lambda: f(x, x, post=(w, None), pre=(w.float(), None)), lambda: f(x, x, gate=x[:4]), lambda: f(x, x, gate=w[None, None]),
                 lambda: f(x, x, post=w), lambda: f(x, x, n=x), lambda: f(x, x.t()), lambda: f(x, x.cpu()), lambda: f(x, x, r=x), lambda: f(x, x, gate=w.cpu())):
        with pytest.raises(moe.MoeError):
            call()
    b = x.clone()
    r, n, stats = f(x, b, post=(w, None), pre=(w, None))
    g = lambda dr, dn, **kw: moe.block_norm_backward(dr, dn, r, b, stats, **{"post": (w, None), "pre": (w, None), **kw})
    for call in (lambda: g(None, None), lambda: g(x.float(), x), lambda: g(x[:3], x), lambda: g(x, x, pre=None), lambda: g(x, x, want=("weight",)), lambda: g(x, x, gate=w[:3])):
        with pytest.raises(moe.MoeError):
            call()
