"""The operators as a training step uses them together: rms_norm -> gate product -> router -> moe_layer and
back, against the formulas in 64 bits, and captured into a graph.

The reference takes the run's own rounded h (bf16) and its own choice of experts, and is otherwise
differentiated in 64 bits.  Bounds on the gradients, from those that each part is held to:
  dh (bf16) is the sum of the layer's dx, within TOL rms plus its rounding, of the gate product's part, rounded
  to bf16, and of their sum's rounding.  The gate product's part carries d(topk_w)'s TOL rms through the
  router, |d logits error| <= 2 p TOL rms(d topk_w), and through |gate|.
  The norm's backward is rstd (g - xh mean(g xh)) with g = dh w, whose matrix has a 2-norm of at most
  rstd max |w|, so a row's error has at most that times the 2-norm of dh's bound, plus dx's rounding.
"""
import numpy as np
import pytest
import torch

import moe_workloads as mw
import token_dispatch_grouped_route_amd as moe
from gpu_helpers import bf16_dev, check_bf16, f64_host, layer, unpacked

pytestmark = pytest.mark.gpu
TOL = 2e-2   # of the expert layer, relative to the rms
HALF = torch.finfo(torch.bfloat16).eps / 2


def f64(u16):
    return bf16_dev(u16).double().cpu()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("w", [mw.Workload("block_share", T=301, H=384, I=256, E=10, EL=5, k=3, e_lo=2, backward=True),
                               mw.Workload("block_all", T=64, H=256, I=128, E=8, EL=8, k=2, backward=True)], ids=lambda w: w.name)
def test_training_step(w, score):
    d = mw.inputs(w, 23)
    ns = layer(w, d, 64, train=True)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = ns.x.clone().requires_grad_()
    nw = (1 + 0.2 * torch.randn(w.H, generator=g, device="cuda")).requires_grad_()
    gate = (torch.randn(w.H, w.E, generator=g, device="cuda") / w.H ** 0.5).requires_grad_()
    W1p, W2p = ns.W1p.clone().requires_grad_(), ns.W2p.clone().requires_grad_()

    h = moe.rms_norm(x, nw)
    idx, tw = moe.router(h.float() @ gate, w.k, score=score)
    y = moe.moe_layer(h, idx, tw, W1p, W2p, ns.shape, ns.ws)
    y.backward(ns.dy)
    torch.cuda.synchronize()

    x64, nw64, gate64 = (t.detach().double().cpu().requires_grad_() for t in (x, nw, gate))
    W1, W2 = f64(d["W1"]).requires_grad_(), f64(d["W2"]).requires_grad_()
    rstd = 1 / (x64.square().mean(1, keepdim=True) + 1e-5).sqrt()
    h64 = x64 * rstd * nw64
    h64 = h64 + (h.detach().double().cpu() - h64).detach()
    to_layer, to_gate = h64 * 1, h64 * 1
    chosen = idx.cpu().long()
    l = (to_gate @ gate64).gather(1, chosen)
    p = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l) / torch.sigmoid(l).sum(1, keepdim=True)
    ref = torch.zeros(w.T, w.H, dtype=torch.float64)
    for e in range(w.EL):
        t, j = (chosen == w.e_lo + e).nonzero(as_tuple=True)
        a = to_layer[t] @ W1[e]
        a = torch.nn.functional.silu(a[:, :w.I]) * a[:, w.I:]
        ref = ref.index_add(0, t, p[t, j, None] * (a @ W2[e]))
    parts = torch.autograd.grad(ref, (to_layer, to_gate, p, x64, nw64, gate64, W1, W2), f64(d["dy"]))
    dh_layer, dh_gate, dp, dx, dnw, dgate, dW1, dW2 = (t.detach() for t in parts)

    check_bf16(f64_host(y.detach()), ref.detach().numpy(), TOL, "y")
    got1, got2 = unpacked(ns, W1p.grad, W2p.grad)
    check_bf16(got1, dW1.numpy(), TOL, "dW1")
    check_bf16(got2, dW2.numpy(), TOL, "dW2")
    dl = torch.zeros(w.T, w.E, dtype=torch.float64).scatter_add_(1, chosen, 2 * TOL * dp.square().mean().sqrt() * p.detach())
    off = dl @ gate64.detach().abs().t()
    off = 1.02 * (off + TOL * dh_layer.square().mean().sqrt() + HALF * (dh_layer.abs() + dh_gate.abs() + (dh_layer + dh_gate).abs()))
    xh = (x64 * rstd).detach()

    err = x.grad.double().cpu() - dx
    bound = rstd.detach()[:, 0] * nw64.detach().abs().max() * off.norm(dim=1) + HALF * dx.norm(dim=1)
    assert (err.norm(dim=1) <= bound).all(), (err.norm(dim=1) / bound).max()
    small = 1e-5   # fp32 sums over the tokens and the row's statistics
    err, bound = (nw.grad.double().cpu() - dnw).abs(), (xh.abs() * off).sum(0) + small * (xh * (dh_layer + dh_gate)).abs().sum(0)
    assert (err <= bound).all(), (err / bound).max()
    h_abs = h.detach().double().cpu().abs()
    err, bound = (gate.grad.double().cpu() - dgate).abs(), h_abs.t() @ dl + small * h_abs.sum(0)[:, None] * dp.abs().max()
    assert (err <= bound).all(), (err / bound).max()


def test_captured_with_its_backward():
    """norm -> gate product -> router with gradients by autograd inside a captured graph, replayed with other
    inputs and eager work between the replays, gives the eager run's bits."""
    T, H, E, k = 200, 512, 16, 4
    g = torch.Generator(device="cuda").manual_seed(6)
    x, nw = torch.randn(T, H, generator=g, device="cuda").bfloat16(), torch.ones(H, device="cuda")
    gate, dtw = torch.randn(H, E, generator=g, device="cuda") / H ** 0.5, torch.randn(T, k, generator=g, device="cuda")

    def step():
        a, b = x.detach().requires_grad_(), nw.detach().requires_grad_()
        h = moe.rms_norm(a, b)
        logits = h.float() @ gate
        idx, tw = moe.router(logits, k, score="sigmoid", scale=2.5)
        return [h.detach(), logits.detach(), idx, tw.detach(), *torch.autograd.grad(tw, (logits, a, b), dtw)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for n in range(3):
        x.copy_(torch.randn(T, H, generator=g, device="cuda"))
        dtw.normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in held]
        for a, b in zip(kept, step()):
            assert torch.equal(a, b), n
