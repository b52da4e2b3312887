"""The dense operators of a block as they are used together: the seam before the expert layer (block_norm), the gate product
(linear), the router, the expert layer, a shared expert added to its result (two linears) and the seam after it; as a training
step against the formulas in 64 bits, and as a decode step (forward_few) captured into a graph.

The reference is differentiated in 64 bits at the run's own rounded values and choice of experts.  A gradient passes at most six
roundings to bf16 on its way (of s, of the shared expert's dz, da and dn, of the sum of dn's three parts, its own), each at most
2^-8 of a value, and the expert layer's backward, held to TOL of the rms by its own tests.  Matrices of independent normal entries
of these shapes stretch a gradient and an error of it alike, within a factor of 2 in the 2-norm; so an error is within
2 (6 2^-8 + TOL) of the gradient in the 2-norm.  The gate's has twice that: the router's d(logits) is a difference of two
terms that carry it."""
import pytest
import torch

import token_dispatch_grouped_route_amd as moe

pytestmark = pytest.mark.gpu
TOL = 2e-2
BOUND = 2 * (6 * 2.0 ** -8 + TOL)
EPS = 1e-5


def rms64(v, w):
    return v / (v.square().mean(1, keepdim=True) + EPS).sqrt() * w


def experts64(n, idx, tw, W1, W2):
    y = torch.zeros(n.shape, dtype=torch.float64, device=n.device)
    for e in range(W1.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        gate, up = (n[t] @ W1[e]).chunk(2, 1)
        y = y.index_add(0, t, tw[t, j][:, None] * ((torch.nn.functional.silu(gate) * up) @ W2[e]))
    return y


class Block:
    def __init__(self, T, H, I, E, k, shared, train):
        g = torch.Generator(device="cuda").manual_seed(T + H)
        normal = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.shape = moe.make_shape(T, H, I, E, E, k, block_m=64, train=train)
        self.x, self.b = normal(T, H), normal(T, H).bfloat16()
        self.gate = normal(H)
        self.w1, self.w2, self.w3 = (1 + 0.2 * normal(H) for _ in range(3))
        self.route = (normal(H, E) / H ** 0.5).bfloat16()
        self.up, self.down = (normal(H, 2 * shared) / H ** 0.5).bfloat16(), (normal(shared, H) / shared ** 0.5).bfloat16()
        self.W1, self.W2 = (normal(E, H, 2 * I) / H ** 0.5).bfloat16(), (normal(E, I, H) / I ** 0.5).bfloat16()
        self.W1p, self.W2p = moe.alloc_packed(self.shape)
        moe.pack_weights(self.shape, self.W1, self.W2, self.W1p, self.W2p)
        self.v1, self.v2 = normal(T, H), normal(T, H).bfloat16()


NAMES = ("x", "b", "gate", "w1", "w2", "w3", "route", "up", "down")


@pytest.mark.parametrize("T,H,I,E,k,shared", [(96, 256, 128, 8, 2, 192), (301, 384, 256, 6, 3, 136)])
def test_training_step(T, H, I, E, k, shared):
    c = Block(T, H, I, E, k, shared, True)
    ws = moe.alloc_workspace(c.shape)
    leaves = {n: getattr(c, n).clone().requires_grad_() for n in NAMES}
    L = lambda n: leaves[n]
    r, n = moe.block_norm(L("x"), L("b"), L("gate"), L("w1"), None, L("w2"), eps=EPS)
    idx, tw = moe.router(moe.linear(n, L("route"), out_dtype=torch.float32), k)
    y = moe.moe_layer(n, idx, tw, c.W1p, c.W2p, c.shape, ws)
    a = moe.linear(n, L("up"), act="swiglu")
    s = moe.linear(a, L("down"), residual=y)
    r2, n2 = moe.block_norm(r, s, pre_weight=L("w3"), post=False, eps=EPS)
    got = torch.autograd.grad((r2, n2), [leaves[q] for q in NAMES], (c.v1, c.v2))

    d = {q: getattr(c, q).double().requires_grad_() for q in NAMES}
    at = lambda v, run: v + (run.detach().double() - v).detach()   # the run's value, this formula's gradient
    R = at(d["x"] + d["gate"] * rms64(d["b"], d["w1"]), r)
    N = at(rms64(R, d["w2"]), n)
    logits = (N @ d["route"]).gather(1, idx.long())
    W = at(torch.softmax(logits, 1), tw)
    Y = at(experts64(N, idx, W, c.W1.double(), c.W2.double()), y)
    A = N @ d["up"]
    A = at(torch.nn.functional.silu(A[:, :shared]) * A[:, shared:], a)
    R2 = R + at(A @ d["down"] + Y, s)
    want = torch.autograd.grad((R2, rms64(at(R2, r2), d["w3"])), [d[q] for q in NAMES], (c.v1.double(), c.v2.double()))
    for q, u, v in zip(NAMES, got, want):
        err = ((u.double() - v).norm() / v.norm()).item()
        print("[parity] %s error / bound %.3g" % (q, err / BOUND))
        assert err <= BOUND * (2 if q == "route" else 1), (q, err)


@pytest.mark.parametrize("T", [1, 5, 48])
def test_decode_step_in_a_graph(T):
    """Eager against the formulas at the run's own roundings, then captured and replayed with other inputs."""
    H, I, E, k, shared = 512, 256, 16, 4, 264
    c = Block(T, H, I, E, k, shared, False)
    ws = moe.few_alloc_workspace(c.shape)

    def step():
        r, n, _ = moe.block_norm_forward(c.x, c.b, post=(c.w1, None), gate=c.gate, pre=(c.w2, None), eps=EPS)
        idx, tw = moe.route_topk(moe.linear_forward(n, c.route, out_dtype=torch.float32)[0], k)[:2]
        y = moe.forward_few(c.shape, n, idx, tw, c.W1p, c.W2p, ws)
        s = moe.linear_forward(moe.linear_forward(n, c.up, act="swiglu")[0], c.down, residual=y, y=y)[0]
        r2, n2, _ = moe.block_norm_forward(r, s, pre=(c.w3, None), eps=EPS)
        return r, n, idx, tw, s, r2, n2

    r, n, idx, tw, s, r2, n2 = step()
    N = n.double()
    A = N @ c.up.double()
    S = experts64(N, idx, tw.double(), c.W1.double(), c.W2.double()) + (torch.nn.functional.silu(A[:, :shared]) * A[:, shared:]) @ c.down.double()
    # roundings to bf16: of both hidden activations, of y and of s; each at most 2^-8 of a value
    assert (s.double() - S).norm() <= 2 * 4 * 2.0 ** -8 * S.norm()
    R2 = r.double() + s.double()
    assert (n2.double() - rms64(R2, c.w3.double())).abs().max() <= 2.0 ** -7 * rms64(R2, c.w3.double()).abs().max()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    g = torch.Generator(device="cuda").manual_seed(1)
    for _ in range(3):
        c.x.copy_(torch.randn(T, H, generator=g, device="cuda"))
        c.b.copy_(torch.randn(T, H, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in held]
        assert all(torch.equal(u, v) for u, v in zip(kept, step()))
