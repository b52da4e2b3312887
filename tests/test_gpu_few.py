"""The expert layer for few tokens (moe_forward_few) against 64-bit products of the same bf16 weights, and beside the layer's
other forms.

Bound, u = 2^-24: a product of reduction length K is summed in fp32, 16 products per matrix instruction, additions counted at
2 u each: within chain(K) sum |a b|, chain(K) = 2 u (K / 16 + 16 + 16) (the last 16 for the waves' sums).  silu(gate) up
carries the errors of gate and up (slope at most 1.1) and 16 u of its own, then half a step of bf16; these go through |W2|
and the routing weights, with chain(I) and k additions more, and the output adds its rounding."""
import pytest
import torch

import token_dispatch_grouped_route_amd as moe

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(autouse=True)
def _free_memory():
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def chain(K):
    return 2 * U * (K / 16 + 32)


class Layer:
    def __init__(self, T, H, I, E, EL, k, e_lo=0, seed=0, idx=None, block_m=64):
        g = gen(seed + T + H)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.shape = moe.make_shape(T, H, I, E, EL, k, block_m=block_m, e_lo=e_lo)
        self.x = rand(T, H).bfloat16()
        self.idx = torch.sort(rand(T, E), 1, descending=True).indices[:, :k].int().contiguous() if idx is None else idx
        self.w = torch.rand(T, k, generator=g, device="cuda")
        self.W1, self.W2 = (rand(EL, H, 2 * I) / H ** 0.5).bfloat16(), (rand(EL, I, H) / I ** 0.5).bfloat16()
        self.pack()
        self.ws = moe.few_alloc_workspace(self.shape)

    def pack(self):
        self.w1p, self.w2p = moe.alloc_packed(self.shape)
        moe.pack_weights(self.shape, self.W1, self.W2, self.w1p, self.w2p)

    def run(self, **kw):
        return moe.forward_few(self.shape, self.x, self.idx, self.w, self.w1p, self.w2p, self.ws, **kw)

    def check(self):
        s, y = self.shape, self.run()
        want = torch.zeros(s.T, s.H, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(want)
        for e in range(s.EL):
            t, j = torch.nonzero(self.idx == s.e_lo + e, as_tuple=True)
            if not len(t):
                continue
            x, w1, w2 = self.x[t].double(), self.W1[e].double(), self.W2[e].double()
            h, eh = x @ w1, chain(s.H) * (x.abs() @ w1.abs())
            (gate, up), (eg, eu) = h.chunk(2, 1), eh.chunk(2, 1)
            sg = torch.nn.functional.silu(gate)
            a = sg * up
            ea = 1.1 * eg * (up.abs() + eu) + sg.abs() * eu + 16 * U * (gate * up).abs()
            ea = ea + HALF * (a.abs() + ea)
            p = self.w[t, j].double()[:, None]
            want.index_add_(0, t, p * (a @ w2))
            tol.index_add_(0, t, p * ((ea + (chain(s.I) + 34 * U) * (a.abs() + ea)) @ w2.abs()))
        tol = tol + HALF * (want.abs() + tol) + 1e-38
        err = (y.double() - want).abs()
        print("[parity] few %r error / bound %.3g, error / rms %.3g" % (s, (err / tol).max() if s.T else 0, err.max() / want.square().mean().sqrt() if s.T else 0))
        assert torch.isfinite(y).all() and (err <= tol).all(), (err / tol).max()
        return y


@pytest.mark.parametrize("T,H,I,E,EL,k,e_lo", [
    (1, 128, 128, 1, 1, 1, 0), (1, 256, 128, 8, 8, 2, 0), (1, 2048, 1408, 64, 64, 6, 0), (3, 384, 256, 16, 4, 4, 5), (7, 128, 384, 8, 3, 3, 2), (16, 1024, 640, 32, 8, 8, 24),
    (40, 256, 256, 4, 4, 2, 0), (64, 512, 384, 8, 8, 4, 0), (100, 640, 128, 3, 3, 1, 0), (129, 256, 384, 5, 2, 3, 1), (512, 128, 256, 16, 16, 8, 0), (4096, 128, 128, 9, 5, 1, 2), (128, 256, 128, 40, 33, 32, 3)])
def test_sizes(T, H, I, E, EL, k, e_lo):
    Layer(T, H, I, E, EL, k, e_lo).check()


@pytest.mark.parametrize("T", [1, 20])
@pytest.mark.parametrize("H,I", [(32768, 128), (128, 32768)])
def test_longest_reductions(H, I, T):
    Layer(T, H, I, 4, 2, 2).check()


def test_counts_around_the_row_tiles():
    """One expert with every number of pairs around 8, 32 and 64, another with the rest."""
    for n in (1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 97):
        T = n + 3
        idx = torch.ones(T, 1, dtype=torch.int32, device="cuda")
        idx[:n] = 0
        Layer(T, 256, 128, 2, 2, 1, idx=idx[torch.randperm(T, generator=gen(n), device="cuda")].contiguous()).check()


def test_odd_routing():
    """Ids that no GPU has, that other GPUs have, the same expert twice in a token, tokens without a local pair: with fewer
    pairs than experts and with more."""
    for EL, T in ((40, 6), (3, 50)):
        E = EL + 4
        g = gen(EL)
        idx = torch.randint(-2, E + 3, (T, 4), generator=g, device="cuda", dtype=torch.int32)
        idx[0] = -1
        idx[1] = 2
        idx[2] = torch.tensor([2, 5, 2, 2 ** 31 - 1], dtype=torch.int32)
        y = Layer(T, 256, 256, E, EL, 4, e_lo=2, idx=idx).check()
        assert not y[0].any()


def test_beside_the_other_forms():
    """moe_forward on the same packed weights: both round the activation and y to bf16, so they differ by those roundings
    of slightly different fp32 sums (at most one step of y where two round apart, plus the activation's through W2)."""
    for T in (1, 5, 48):
        l = Layer(T, 512, 256, 16, 16, 4)
        y, full = l.run(), torch.empty(T, 512, dtype=torch.bfloat16, device="cuda")
        moe.forward(l.shape, l.x, l.idx, l.w, l.w1p, l.w2p, moe.alloc_workspace(l.shape), full)
        rms = full.double().square().mean().sqrt()
        assert (full.double() - y.double()).square().mean().sqrt() <= HALF * rms


def test_no_tokens():
    l = Layer(0, 256, 128, 4, 4, 2, idx=torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert l.run().shape == (0, 256)


def test_tokens_do_not_reach_each_other():
    for T in (3, 24, 150):
        l = Layer(T, 512, 256, 16, 16, 4)
        y = l.run()
        for fill in (1.0, float("nan"), float("inf")):
            z = torch.full_like(l.x, fill)
            z[1] = l.x[1]
            l.x, keep = z, l.x
            assert torch.equal(l.run()[1], y[1])
            l.x = keep


def test_bad_weights_of_other_experts_are_not_read_into_a_result():
    """NaN weights of experts that no token chose, and non-local slots."""
    l = Layer(6, 256, 256, 12, 8, 2, e_lo=2)
    y = l.run()
    used = set(l.idx.flatten().tolist())
    for e in range(8):
        if e + 2 not in used:
            l.W1[e], l.W2[e] = float("nan"), float("nan")
    l.pack()
    assert torch.equal(l.run(), y)


def test_large_weight_offsets():
    """Experts whose weights start past 2^32 bytes."""
    H, I, EL = 4096, 2048, 140
    l = Layer(2, H, I, EL, EL, 2, idx=torch.tensor([[EL - 1, 0], [EL - 2, EL - 1]], dtype=torch.int32, device="cuda"))
    assert (EL - 1) * 4 * I * H > 2 ** 32
    l.check()


def test_streams_and_two_captured_graphs():
    """Two graphs that share a workspace, replayed in turn with eager work between; a side stream."""
    a, b = Layer(12, 512, 256, 16, 16, 4), Layer(3, 512, 256, 16, 16, 4, seed=9)
    b.ws = a.ws
    first = a.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = a.run(stream=side)
    side.synchronize()
    assert torch.equal(other, first)
    graphs, held = [], []
    for l in (a, b):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held.append(l.run())
        graphs.append(graph)
    for n in range(3):
        a.x.copy_(torch.randn(12, 512, generator=gen(n), device="cuda"))
        for t, graph in zip(held, graphs):
            t.fill_(float("nan"))
            graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in held]
        assert torch.equal(kept[0], a.run()) and torch.equal(kept[1], b.run())


def test_refusals():
    l = Layer(4, 256, 128, 8, 8, 2)
    f = lambda **kw: moe.forward_few(**{**dict(shape=l.shape, x=l.x, topk_idx=l.idx, topk_w=l.w, w1p=l.w1p, w2p=l.w2p, ws=l.ws), **kw})
    for bad in (dict(x=l.x[:3]), dict(x=l.x.half()), dict(topk_idx=l.idx.long()), dict(topk_w=l.w[:, :1]), dict(w1p=l.w2p), dict(ws=l.ws[:256]), dict(ws=l.ws.cpu()), dict(w2p=l.w2p.cpu()),
                dict(y=torch.empty(3, 256, dtype=torch.bfloat16, device="cuda")), dict(shape=moe.make_shape(4, 256, 128, 8, 8, 2, block_m=64, train=True))):
        with pytest.raises(moe.MoeError):
            f(**bad)
