"""4-bit products on the GPU: quantisation (integer results, equal), the linear map and the expert
layer against 64-bit products of the same codes.

Bound, u = 2^-24: a group's sum is formed as sum (16 + q) x - (16 + z) sum x, each in fp32 chains of at
most 128 products; the matrix core's additions are counted at 2 u each.  With the sums over groups,
waves and zero-point terms (K / group + 24 more), every output is within
(2 * 136 + K / group + 24) u * sum s (32 + q + z) |x| of the exact product, before its own rounding."""
import numpy as np
import pytest
import torch

import moe_workloads as mw
import token_dispatch_grouped_route_amd as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BOTH = [torch.bfloat16, torch.float16]


@pytest.fixture(autouse=True)
def _free_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def random_w4(g, lead, N, K, group, dtype, zeros):
    codes = torch.randint(0, 256, lead + (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((0.5 + torch.rand(lead + (N, K // group), generator=g, device="cuda")) / (4.6 * K ** 0.5)).to(dtype)
    z = torch.randint(0, 16, lead + (N, K // group), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    return codes, scales, z


def decode(codes, scales, zeros):
    """(weights, s (32 + q + z)) in 64 bits, [..., N, K]."""
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).double()
    rep = q.shape[-1] // scales.shape[-1]
    z = zeros.double().repeat_interleave(rep, -1) if zeros is not None else torch.full_like(q, 8.0)
    s = scales.double().repeat_interleave(rep, -1)
    return (q - z) * s, s * (32 + q + z)


def product(x, w, mag, groups):
    """x @ w^T and its bound."""
    return x @ w.transpose(-1, -2), (2 * 136 + groups + 24) * U * (x.abs() @ mag.transpose(-1, -2))


def stored(v, dtype):
    fi = torch.finfo(dtype)
    return fi.eps / 2 * v + fi.smallest_normal * fi.eps


def check_linear(x, w4, y=None, **kw):
    got = moe.w4_linear(x, *w4, y=y, **kw)
    want, tol = product(x.double(), *decode(*w4), w4[1].shape[-1])
    tol = tol + stored(want.abs() + tol, x.dtype)
    err = (got.double() - want).abs()
    rms = want.square().mean().sqrt()
    print("[parity] linear %s %s error / bound %.3g, error / rms %.3g" % (tuple(x.shape), tuple(w4[0].shape), (err / tol).max(), err.max() / rms))
    assert torch.isfinite(got).all() and (err <= tol).all(), (err / tol).max()
    return got


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,N,K,group", [(1, 1, 32, 32), (1, 100, 256, 128), (2, 17, 96, 32), (3, 64, 160, 32), (16, 33, 192, 64), (17, 130, 1024, 128), (5, 48, 4096, 256),
                                         (33, 31, 512, 64), (64, 256, 1408, 128), (65, 40, 640, 32), (130, 20, 320, 64), (1, 4096, 7168, 128), (7, 50, 32768, 32),
                                         (20, 10000, 256, 64), (3, 11000, 128, 32), (70, 5000, 384, 128), (2, 33000, 64, 32), (2, 33000, 32768, 32)])
def test_linear(M, N, K, group, zeros, dtype):
    g = gen(M * 1000 + N)
    check_linear(torch.randn(M, K, generator=g, device="cuda").to(dtype), random_w4(g, (), N, K, group, dtype, zeros))


def test_every_code_and_zero_point():
    """Unit scales and one-hot activations return code - zero exactly."""
    K, N = 256, 64
    codes = torch.arange(N * K // 2, device="cuda").to(torch.uint8).view(N, K // 2)
    z = (torch.arange(N * 8, device="cuda") % 16).to(torch.uint8).view(N, 8)
    w4 = (codes, torch.ones(N, 8, dtype=torch.bfloat16, device="cuda"), z)
    y = moe.w4_linear(torch.eye(K, dtype=torch.bfloat16, device="cuda"), *w4)
    assert torch.equal(y.double().t(), decode(*w4)[0])


@pytest.mark.parametrize("dtype", BOTH)
def test_linear_strided(dtype):
    g = gen(5)
    wide = torch.randn(20, 560, generator=g, device="cuda").to(dtype)
    store = torch.full((22, 75), 3.0, dtype=dtype, device="cuda")
    w4 = random_w4(g, (), 67, 512, 64, dtype, True)
    check_linear(wide[:, 16:528], w4, y=store[1:21, 5:72])
    around = torch.ones_like(store, dtype=torch.bool)
    around[1:21, 5:72] = False
    assert (store[around] == 3.0).all()
    assert torch.equal(moe.w4_linear(wide[:, 16:528].reshape(4, 5, 512), *w4).view(20, 67), store[1:21, 5:72])


def test_linear_without_rows_and_with_extreme_activations():
    g = gen(6)
    w4 = random_w4(g, (), 40, 256, 32, torch.bfloat16, True)
    assert moe.w4_linear(torch.empty(0, 256, dtype=torch.bfloat16, device="cuda"), *w4).shape == (0, 40)
    x = torch.randn(20, 256, generator=g, device="cuda").to(torch.bfloat16)
    x[3] *= 1e30
    x[4] *= 1e-30
    x[5] = 0
    x[6] = 5.0      # the zero-point terms cancel most
    y = check_linear(x, w4)
    assert (y[5] == 0).all()
    x[7, 9], x[8, 200] = float("nan"), float("inf")
    bad = moe.w4_linear(x, *w4)
    assert not torch.isfinite(bad[7:9]).any()
    rest = [i for i in range(20) if i not in (7, 8)]
    assert torch.equal(bad[rest], y[rest])      # a row's values do not reach the others


@pytest.mark.parametrize("wdtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_equals_its_definition(zeros, dtype, wdtype):
    E, K, N, group = 2, 256, 70, 64
    w = torch.randn(E, K, N, generator=gen(1), device="cuda")
    w[0, :64, 3] = 0
    w[0, 64:128, 4] = w[0, 64:128, 4].abs()
    w[1, :64, 5] = -w[1, :64, 5].abs()
    w[1, 0, 6] = 100.0
    w = (0.05 * w).to(wdtype)
    codes, scales, points = moe.w4_quantize(w, group, zeros, dtype)
    v = w.float().cpu().transpose(1, 2).reshape(E, N, K // group, group).numpy()
    lo, hi = np.minimum(v.min(-1), 0), np.maximum(v.max(-1), 0)
    s = torch.from_numpy((hi - lo) / np.float32(15) if zeros else np.maximum(hi, -lo) / np.float32(7)).to(dtype)
    assert torch.equal(scales.cpu(), s)
    s = s.float().numpy()
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(s > 0, np.minimum(np.rint(-lo / s), 15), 0) if zeros else np.full_like(s, 8)
        q = np.where(s[..., None] > 0, np.clip(np.rint(v / s[..., None]) + z[..., None], 0, 15), z[..., None])
    if zeros:
        assert np.array_equal(points.cpu().numpy(), z.astype(np.uint8))
    else:
        assert points is None
    q = q.astype(np.uint8).reshape(E, N, K)
    assert np.array_equal(codes.cpu().numpy(), q[..., 0::2] | (q[..., 1::2] << 4))
    # a weight is half a step of its group from its code; the scale's rounding adds at most 15 half steps of its type
    back = decode(codes, scales, points)[0].cpu()
    step = torch.from_numpy(s).double().repeat_interleave(group, -1)
    assert ((back - torch.from_numpy(v.reshape(E, N, K)).double()).abs() <= step * (0.5 + 17 * torch.finfo(dtype).eps) + 1e-12).all()


# ------------------------------------------------------------------------------------------------
# expert layer
# ------------------------------------------------------------------------------------------------
def reference_experts(s, x, idx, tw, w1, w2):
    """y and its bound in 64 bits."""
    dt, x = x.dtype, x.double()
    y, tol = torch.zeros(s.T, s.H, dtype=torch.float64, device="cuda"), torch.zeros(s.T, s.H, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(y)
    for e in range(s.EL):
        t, j = torch.nonzero(idx == s.e_lo + e, as_tuple=True)
        if not len(t):
            continue
        one, two = ([p[e] if p is not None else None for p in w] for w in (w1, w2))
        h, dh = product(x[t], *decode(*one), one[1].shape[-1])
        g, u, dg, du = h[:, :s.I], h[:, s.I:], dh[:, :s.I], dh[:, s.I:]
        sg = torch.sigmoid(g)
        a = g * sg * u
        # |silu'| <= 1.1; the sigmoid's exponential is (2.5 |g| + 4) u off, the products and the sum 4 u
        da = 1.1 * dg * (u.abs() + du) + (g * sg).abs() * du + (2.5 * g.abs() + 12) * U * a.abs()
        da = da + stored(a.abs() + da, dt)
        w, mag = decode(*two)
        o, do = product(a, w, mag, two[1].shape[-1])
        do = do + da @ w.abs().t() + (2 * 136 + two[1].shape[-1] + 24) * U * (da @ mag.t())
        f = tw[t, j].double()[:, None]
        y.index_add_(0, t, f * o)
        tol.index_add_(0, t, f.abs() * do)
        size.index_add_(0, t, (f * o).abs())
    tol = tol + (s.k + 2) * U * size
    return y, tol + stored(y.abs() + tol, dt)


def experts_inputs(T, H, I, E, EL, k, group, dtype, zeros, e_lo=0, seed=0, spread=1.0):
    g = gen(seed)
    s = moe.make_shape(T, H, I, E, EL, k, block_m=64, e_lo=e_lo)
    x = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    idx, tw = moe.route_topk(spread * torch.randn(1, E, generator=g, device="cuda") + torch.randn(T, E, generator=g, device="cuda"), k)
    return s, x, idx, tw, random_w4(g, (EL,), 2 * I, H, group, dtype, zeros), random_w4(g, (EL,), H, I, group, dtype, zeros)


def check_experts(s, x, idx, tw, w1, w2, ws=None):
    ws = moe.w4_alloc_workspace(s) if ws is None else ws
    ws.fill_(255)   # NaN in every type: rows that no pair writes must not be read
    y = torch.full((s.T + 2, s.H), 5.0, dtype=x.dtype, device="cuda")
    moe.forward_w4(s, x, idx, tw, w1, w2, ws, y=y[1:-1])
    assert (y[0] == 5.0).all() and (y[-1] == 5.0).all()
    y = y[1:-1]
    want, tol = reference_experts(s, x, idx, tw, w1, w2)
    err = (y.double() - want).abs()
    rms = want.square().mean().sqrt().item()
    print("[parity] experts %r error / bound %.3g, error / rms %.3g" % (s, (err / tol).max(), err.max() / max(rms, 1e-30)))
    assert torch.isfinite(y).all() and (err <= tol).all(), (err / tol).max()
    return y


@pytest.mark.parametrize("dtype", BOTH)
@pytest.mark.parametrize("T,H,I,E,EL,k,group,zeros,e_lo", [
    (1, 256, 128, 8, 8, 2, 128, False, 0),      # fewer pairs than experts
    (1, 384, 256, 64, 8, 6, 32, True, 16),      # most pairs elsewhere
    (3, 256, 384, 16, 16, 4, 64, True, 0),
    (4, 128, 128, 8, 8, 2, 32, False, 0),       # as many pairs as experts
    (5, 128, 128, 8, 8, 2, 64, False, 0),       # more
    (40, 512, 256, 8, 8, 4, 128, True, 0),      # several 16-row passes per expert
    (100, 256, 128, 1, 1, 1, 128, False, 0),    # one expert
    (33, 256, 128, 300, 200, 8, 32, False, 50),
    (130, 1152, 128, 4, 2, 3, 128, True, 1),
    (3, 256, 128, 40, 20, 17, 32, True, 5),     # more slots than a workgroup takes at once
    (2, 640, 2048, 12, 9, 9, 32, False, 3),
    (1, 128, 2176, 8, 8, 2, 128, True, 0),      # the shortest and longest K on either side of the token kernel
    (20, 512, 128, 160, 160, 8, 64, True, 0),   # by pair, with more waves than are resident
])
def test_experts(T, H, I, E, EL, k, group, zeros, e_lo, dtype):
    check_experts(*experts_inputs(T, H, I, E, EL, k, group, dtype, zeros, e_lo, seed=T))


def test_experts_at_the_pair_limit():
    s, x, idx, tw, w1, w2 = experts_inputs(512, 256, 128, 16, 16, 8, 64, torch.bfloat16, True)
    check_experts(s, x, idx, tw, w1, w2)
    idx.fill_(3)      # every pair on one expert, every id eight times in its token
    check_experts(s, x, idx, tw, w1, w2)


@pytest.mark.parametrize("few", [True, False])
def test_experts_ids_elsewhere_repeated_and_invalid(few):
    T = 2 if few else 9
    s, x, idx, tw, w1, w2 = experts_inputs(T, 256, 128, 32, 8, 3, 64, torch.bfloat16, True, e_lo=8)
    idx[0] = torch.tensor([9, 9, 15])          # the same expert twice
    idx[1] = torch.tensor([-1, 32, 2 ** 30])   # outside the routing
    y = check_experts(s, x, idx, tw, w1, w2)
    assert (y[1] == 0).all()
    idx.fill_(0)                                # nothing local
    assert (check_experts(s, x, idx, tw, w1, w2) == 0).all()


def test_experts_without_tokens():
    s, x, idx, tw, w1, w2 = experts_inputs(1, 256, 128, 8, 8, 2, 64, torch.bfloat16, False)
    s.T = 0
    y = moe.forward_w4(s, x[:0], idx[:0], tw[:0], w1, w2, moe.w4_alloc_workspace(s))
    assert y.shape == (0, 256)


def test_tokens_do_not_reach_each_other():
    """A token's output keeps its bits when the other tokens change, to NaN too, in both grids."""
    for T in (3, 24):
        s, x, idx, tw, w1, w2 = experts_inputs(T, 512, 256, 16, 16, 4, 64, torch.bfloat16, True)
        ws = moe.w4_alloc_workspace(s)
        y = moe.forward_w4(s, x, idx, tw, w1, w2, ws)
        for fill in (1.0, float("nan")):
            z = torch.full_like(x, fill)
            z[1] = x[1]
            assert torch.equal(moe.forward_w4(s, z, idx, tw, w1, w2, ws)[1], y[1])


@pytest.mark.parametrize("T", [1, 20])
@pytest.mark.parametrize("H,I", [(32768, 128), (128, 32768)])
def test_experts_with_the_longest_reductions(H, I, T):
    """As many scales as fit no workgroup of several teams."""
    check_experts(*experts_inputs(T, H, I, 4, 2, 2, 32, torch.bfloat16, True))


def test_large_weight_offsets():
    """Experts whose codes start past 2^31 bytes."""
    H, I, EL = 4096, 4096, 140
    assert (EL - 1) * 2 * I * H // 2 > 2 ** 31
    s = moe.make_shape(2, H, I, EL, EL, 2, block_m=64)
    g = gen(3)
    x = torch.randn(2, H, generator=g, device="cuda").to(torch.bfloat16)
    w1, w2 = random_w4(g, (EL,), 2 * I, H, 128, torch.bfloat16, True), random_w4(g, (EL,), H, I, 128, torch.bfloat16, True)
    idx = torch.tensor([[EL - 1, 0], [EL - 2, EL - 1]], dtype=torch.int32, device="cuda")
    check_experts(s, x, idx, torch.rand(2, 2, generator=g, device="cuda"), w1, w2)


def test_same_bits_streams_and_two_captured_graphs():
    """Two graphs that share a workspace, replayed in turn with eager work between."""
    s, x, idx, tw, w1, w2 = experts_inputs(12, 512, 256, 16, 16, 4, 64, torch.bfloat16, True)
    s2, x2, idx2, tw2, *_ = experts_inputs(3, 512, 256, 16, 16, 4, 64, torch.bfloat16, True, seed=9)
    ws = moe.w4_alloc_workspace(s)
    eager = lambda n=0: (moe.forward_w4(s, x, idx, tw, w1, w2, ws).clone(), moe.forward_w4(s2, x2, idx2, tw2, w1, w2, ws).clone(), moe.w4_linear(x, *[t[0] for t in w1]))
    first = eager()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = moe.forward_w4(s, x, idx, tw, w1, w2, ws, stream=side)
    side.synchronize()
    assert torch.equal(other, first[0])
    graphs, held = [], []
    for args in ((s, x, idx, tw), (s2, x2, idx2, tw2)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append((moe.forward_w4(*args, w1, w2, ws), moe.w4_linear(args[1], *[t[0] for t in w1])))
        graphs.append(graph)
    for n in range(3):
        x.copy_(torch.randn(12, 512, generator=gen(20 + n), device="cuda").to(torch.bfloat16))
        for h in held:
            for t in h:
                t.fill_(float("nan"))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        y, y2, lin = eager()
        torch.cuda.synchronize()
        assert torch.equal(held[0][0], y) and torch.equal(held[1][0], y2) and torch.equal(held[0][1], lin), n


def test_quantized_layer_end_to_end():
    """norm -> router -> expert layer on quantised weights, as a decode step runs them, against the bf16
    forward on the decoded weights (one rounding of them to bf16 apart)."""
    w = mw.Workload("w4_block", T=6, H=256, I=128, E=8, EL=8, k=2)
    d = mw.inputs(w, 4)
    as_bf16 = lambda a: torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16).cuda()
    gate = torch.randn(256, 8, generator=gen(1), device="cuda") / 16
    h = moe.rms_norm(as_bf16(d["x"]), torch.ones(256, device="cuda"))
    idx, tw = moe.route_topk(h.float() @ gate, 2)
    w1, w2 = moe.w4_quantize(as_bf16(d["W1"]), 64, True), moe.w4_quantize(as_bf16(d["W2"]), 64, True)
    s = moe.make_shape(6, 256, 128, 8, 8, 2, block_m=64)
    y = check_experts(s, h, idx, tw, w1, w2)
    W1, W2 = (decode(*t)[0].transpose(1, 2).to(torch.bfloat16).contiguous() for t in (w1, w2))
    w1p, w2p = moe.alloc_packed(s)
    moe.pack_weights(s, W1, W2, w1p, w2p)
    full = torch.empty_like(y)
    moe.forward(s, h, idx, tw, w1p, w2p, moe.alloc_workspace(s), full)
    # weights, activations and outputs each rounded to bf16 on one side or the other
    rms = full.double().square().mean().sqrt()
    assert (full.double() - y.double()).square().mean().sqrt() <= 4 * 2 ** -8 * rms


def test_refusals():
    g = gen(1)
    x = torch.randn(4, 256, generator=g, device="cuda").to(torch.bfloat16)
    c, s, z = random_w4(g, (), 32, 256, 64, torch.bfloat16, True)
    for bad in (lambda: moe.w4_linear(x.cpu(), c, s), lambda: moe.w4_linear(x.float(), c, s), lambda: moe.w4_linear(x, c[:, :64], s), lambda: moe.w4_linear(x, c, s.half()),
                lambda: moe.w4_linear(x, c, s[:, :3]), lambda: moe.w4_linear(x, c, s, z[:, :2]), lambda: moe.w4_linear(x, c, s[:31]), lambda: moe.w4_linear(x[:, :128], c, s),
                lambda: moe.w4_linear(x.t(), c, s), lambda: moe.w4_linear(x, c.view(1, 32, 128), s), lambda: moe.w4_linear(x, c, s, y=torch.empty(4, 31, dtype=x.dtype, device="cuda")),
                lambda: moe.w4_linear(torch.zeros(4, 264, dtype=x.dtype, device="cuda")[:, 1:257], c, s),
                lambda: moe.w4_quantize(x, 48), lambda: moe.w4_quantize(x, 0), lambda: moe.w4_quantize(x.t(), 32), lambda: moe.w4_quantize(x[0], 32),
                lambda: moe.w4_quantize(torch.zeros(128, 8, device="cuda"), 64, dtype=torch.float32)):
        with pytest.raises(moe.MoeError):
            bad()
    sh, x, idx, tw, w1, w2 = experts_inputs(4, 256, 128, 8, 8, 2, 64, torch.bfloat16, True)
    ws = moe.w4_alloc_workspace(sh)
    other = random_w4(g, (8,), 256, 128, 32, torch.bfloat16, True)
    for bad in (lambda: moe.forward_w4(sh, x[:3], idx, tw, w1, w2, ws), lambda: moe.forward_w4(sh, x, idx.long(), tw, w1, w2, ws), lambda: moe.forward_w4(sh, x, idx, tw[:, :1], w1, w2, ws),
                lambda: moe.forward_w4(sh, x, idx, tw, w2, w1, ws), lambda: moe.forward_w4(sh, x, idx, tw, w1, other, ws), lambda: moe.forward_w4(sh, x, idx, tw, w1, w2, ws[:256]),
                lambda: moe.forward_w4(sh, x.float(), idx, tw, w1, w2, ws), lambda: moe.forward_w4(sh, x, idx, tw, w1, w2, ws.cpu()),
                lambda: moe.forward_w4(sh, x, idx, tw, w1, w2, ws, y=torch.empty(3, 256, dtype=x.dtype, device="cuda"))):
        with pytest.raises(moe.MoeError):
            bad()
