"""Top-k router on the GPU: ids against a sort written out in Python on the same fp32 scores (equal,
ties included), weights and gradients against the definition in 64 bits.

Bounds, u = 2^-24: a weight is a ratio of exponentials.  The argument of exp is rounded by u |a|, the
fast exponential multiplies it by log2 e (another 1.5 u |a|) and is itself within 2 u, so e^a is off by
(2.5 |a| + 4) u relative; log(sigmoid(l)) is off by (2 |l| + 6) u; a sum over n terms adds n u.  Below
a = -104 the exponential is 0 in fp32 and its exact value under 2^-149, which TINY covers."""
import numpy as np
import pytest
import torch

import moe_workloads as mw
import token_dispatch_grouped_route_amd as moe

pytestmark = pytest.mark.gpu
U, TINY = 2.0 ** -24, 1e-37
F32_MAX = float(np.finfo(np.float32).max)


def choose(scores, k, n_group, topk_group):
    """The ids of one row of fp32 scores (-inf: out of service)."""
    E = len(scores)
    alive = [e for e in range(E) if scores[e] > -np.inf]
    if n_group > 1:
        size, value = E // n_group, []
        for g in range(n_group):
            best = sorted((scores[e] for e in alive if e // size == g), reverse=True)[:2]
            with np.errstate(over="ignore"):
                value.append(-np.inf if not best else best[0] if len(best) == 1 else np.float32(best[0] + best[1]))
        kept = sorted(range(n_group), key=lambda g: (-value[g], g))[:topk_group]
        alive = [e for e in alive if e // size in kept]
    ids = sorted(alive, key=lambda e: (-scores[e], e))[:k]
    return ids + [-1] * (k - len(ids))


def reference(logits, k, bias=None, score="softmax", renormalize=True, n_group=1, topk_group=1, scale=1.0, dw=None, idx=None):
    """(ids, weights, weight bounds, dlogits, dlogits bounds) in 64 bits."""
    l32 = logits.float().cpu().numpy().astype(np.float32)
    with np.errstate(invalid="ignore"):
        valid = l32 > -np.inf
    l32 = np.where(valid, np.minimum(l32, np.float32(F32_MAX)), np.float32(-np.inf))
    with np.errstate(over="ignore"):
        s32 = l32 + bias.cpu().numpy() if bias is not None else l32
    T, E = l32.shape
    if idx is None:
        idx = np.array([choose(np.where(valid[t], s32[t], -np.inf), k, n_group, topk_group) for t in range(T)], np.int32).reshape(T, k)
    w, wt, dl, dt = np.zeros((T, k)), np.full((T, k), TINY), np.zeros((T, E)), np.full((T, E), TINY)
    for t in range(T):
        on = [j for j in range(k) if idx[t, j] >= 0]
        if not on:
            continue
        ids = idx[t, on]
        l = l32[t].astype(np.float64)
        a = l[ids]
        sig = np.where(a >= 0, 1 / (1 + np.exp(-np.abs(a))), np.exp(-np.abs(a)) / (1 + np.exp(-np.abs(a))))
        if score == "softmax":
            pool = a if renormalize else l[valid[t]]
            e = np.exp(a - pool.max())
            p = e / np.exp(pool - pool.max()).sum()
            rel = (2.5 * min(pool.max() - a.min(), 104) + 4 + 2.5 * min(np.ptp(pool), 104) + 4 + len(pool) + 4) * U
        else:
            ls = np.minimum(a, 0) - np.log1p(np.exp(-np.abs(a)))
            big = min(np.abs(a).max(), 104)
            if renormalize:
                p = np.exp(ls - ls.max()) / np.exp(ls - ls.max()).sum()
                rel = (2 * (2 * (2 * big + 6) + 2.5 * big + 4) + k + 4) * U
            else:
                p, rel = sig, (2.5 * big + 8) * U
        w[t, on], wt[t, on] = scale * p, abs(scale) * p * (rel + 2 * U) + TINY
        if dw is None:
            continue
        g = scale * dw[t, on].double().cpu().numpy()
        q, mag = (p * g).sum(), (p * np.abs(g)).sum()
        d = p * (g - q) if renormalize else p * g
        d = d * (1 - sig) if score == "sigmoid" else d
        dense = score == "softmax" and not renormalize
        if dense:
            every = np.where(valid[t], np.exp(l - l[valid[t]].max()), 0)
            every = every / every.sum()
            dl[t] -= every * q
            dt[t] += every * mag * (3 * rel + 12 * U)
        big = min(np.abs(a).max(), 104)
        for n, e in enumerate(ids):
            dl[t, e] += d[n]
            dt[t, e] += p[n] * (abs(g[n]) + mag) * (3 * rel + (k + 16 + (2.5 * big + 8) * (score == "sigmoid")) * U)
    return idx, w, wt, dl, dt


def check(logits, k, seed=0, **how):
    idx, w = moe.route_topk(logits, k, **how)
    how2 = {n: v for n, v in how.items() if n in ("score", "renormalize", "scale")}
    dw = torch.randn(logits.shape[0], k, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed))
    dl = moe.route_topk_backward(logits, idx, dw, **how2)
    ri, rw, wt, rd, dt = reference(logits, k, dw=dw, **how)
    assert np.array_equal(idx.cpu().numpy(), ri)
    err = np.abs(w.double().cpu().numpy() - rw)
    assert (err <= wt).all(), ("weights", np.max(err / wt))
    fi = torch.finfo(logits.dtype)
    got = dl.double().cpu().numpy()
    assert dl.dtype == logits.dtype and np.isfinite(got).all()
    tol = dt + fi.eps / 2 * (np.abs(rd) + dt) + fi.smallest_normal * fi.eps
    err = np.abs(got - rd)
    assert (err <= tol).all(), ("dlogits", np.max(err / tol))
    return idx, w, dl


def logits_of(T, E, dtype, seed=0, scale=1.0):
    return (scale * torch.randn(T, E, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
# expert counts around every change of lanes per row and chunks per lane; more slots than 16 lanes
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 2, 2), (37, 8, 2), (3, 33, 8), (18, 64, 6), (9, 127, 16), (7, 129, 8), (11, 200, 17), (6, 256, 8), (5, 321, 9),
                                   (13, 384, 6), (4, 512, 8), (3, 513, 4), (2, 1000, 32), (4, 1024, 8)])
def test_router(T, E, k, score, renormalize, dtype):
    check(logits_of(T, E, dtype, E), k, score=score, renormalize=renormalize, scale=2.5)


@pytest.mark.parametrize("E,n_group,topk_group,k", [(16, 16, 3, 2), (64, 8, 3, 6), (256, 8, 4, 8), (256, 2, 1, 8), (96, 3, 2, 20), (1024, 16, 4, 8), (40, 5, 5, 3), (512, 16, 1, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_groups_and_bias(E, n_group, topk_group, k, dtype):
    bias = 0.5 * torch.randn(E, generator=torch.Generator().manual_seed(1)).cuda()
    for b in (None, bias):
        for score, renormalize in (("sigmoid", True), ("softmax", False)):
            check(logits_of(33, E, dtype, E), k, bias=b, n_group=n_group, topk_group=topk_group, score=score, renormalize=renormalize)


@pytest.mark.parametrize("E", [8, 256, 1000])
@pytest.mark.parametrize("n_group", [1, 4])
def test_ties_go_to_the_lower_id(E, n_group):
    l = torch.randint(-1, 2, (64, E), generator=torch.Generator().manual_seed(E)).float().cuda()
    l[0] = 0.25
    l[1] = torch.where(torch.arange(E, device="cuda") % 2 == 0, 0.0, -0.0)   # equal as numbers
    idx, _, _ = check(l, 8, n_group=n_group, topk_group=n_group)
    assert idx[0].tolist() == idx[1].tolist() == list(range(8))


@pytest.mark.parametrize("E,k", [(32, 8), (256, 8), (256, 15), (512, 6), (1000, 20), (1024, 32)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_that_differ_in_their_last_bits(E, k, sign):
    """Runs of scores one unit in the last place apart, of every length, across the last slot too: rows of
    pairs, rows with a run of r around slot k, whole rows of one run, rows where every fifth score is tied."""
    g = torch.Generator().manual_seed(E + k)
    T = 48
    ulp = 2.0 ** -23
    l = torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        base = 1.0 - torch.arange(E, dtype=torch.float64) / (4 * E)      # 1 .. 0.75, coarse steps
        if t % 4 == 0:
            base[1::2] = base[0::2] - ulp
        elif t % 4 == 1:
            r = 2 + t % 23
            at = max(0, k - 1 - t % 5)
            n = min(r, E - at)
            base[at:at + n] = base[at] - ulp * torch.arange(n, dtype=torch.float64)
        elif t % 4 == 2:
            base = 1.0 - ulp * torch.arange(E, dtype=torch.float64)
        else:
            base = 1.0 - ulp * (torch.arange(E, dtype=torch.float64) // 5)
        l[t] = sign * base[torch.randperm(E, generator=g)]
    l = l.float().cuda()
    check(l, k)
    check(l, k, bias=torch.zeros(E).cuda(), n_group=4, topk_group=3, score="sigmoid")
    check(l.bfloat16(), k, bias=(ulp * torch.randint(0, 4, (E,), generator=g)).float().cuda())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_best_all_in_one_lane(dtype):
    """Scores laid out so that one lane holds many of the row's best, whatever it keeps of them."""
    for E in (128, 256, 384, 512, 1024):
        l = logits_of(40, E, dtype, E)
        n = 4 if dtype == torch.float32 else 8
        for t in range(40):
            lane = t % 16
            ids = [e for e in range(E) if e // n % 16 == lane][: 2 + t % 14]
            l[t, ids] = (10 + torch.randperm(len(ids), generator=torch.Generator().manual_seed(t))).to(dtype).cuda()
        for k in (3, 8, 15, 24):
            check(l, k)


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("E,n_group,topk_group", [(16, 1, 1), (64, 4, 2), (520, 1, 1)])
def test_rows_with_few_or_no_experts_and_extreme_logits(E, n_group, topk_group, score, renormalize):
    inf, nan = float("inf"), float("nan")
    l = logits_of(14, E, torch.float32, 5)
    l[0] = -inf                       # nothing left
    l[1] = nan
    l[2] = -inf
    l[2, 5] = -3.0                    # one left
    l[3, 1::2] = nan                  # NaN is out of service, beside usable ones
    l[4, 7] = inf                     # a certain expert
    l[5, 2], l[5, 3] = inf, F32_MAX   # equal to each other
    l[6] = -F32_MAX
    l[7] = F32_MAX
    l[8] = -200.0
    l[9] = 200.0
    l[10] *= 100
    l[11, 1:] = -inf
    l[12, :E // 2] = -inf
    l[13] = 1e-40                     # subnormal
    for b in (None, torch.linspace(-1, 1, E).cuda()):
        idx, w, _ = check(l, 4, bias=b, n_group=n_group, topk_group=topk_group, score=score, renormalize=renormalize)
        assert (idx[:2] == -1).all() and (w[:2] == 0).all() and idx[2].tolist() == [5, -1, -1, -1]


def test_bias_takes_experts_out_and_never_touches_the_weights():
    l = logits_of(9, 32, torch.float32, 3)
    b = torch.zeros(32).cuda()
    b[::2] = -float("inf")
    b[1] = float("nan")
    idx, w, _ = check(l, 8, bias=torch.where(b != b, torch.tensor(-float("inf")).cuda(), b))
    got, _ = moe.route_topk(l, 8, bias=b)
    assert torch.equal(got, idx) and (idx % 2 == 1).all() and (idx != 1).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_logits_and_outputs(dtype):
    wide = logits_of(21, 80, dtype, 9)
    l = wide[:, 3:70]
    idx, w, dl = check(l, 5)
    store = torch.full((23, 75), 9.0, dtype=dtype, device="cuda")
    out = moe.route_topk_backward(l, idx, torch.ones_like(w), renormalize=False, dlogits=store[1:22, 5:72])
    assert torch.equal(out, moe.route_topk_backward(l.contiguous(), idx, torch.ones_like(w), renormalize=False))
    around = torch.ones_like(store, dtype=torch.bool)
    around[1:22, 5:72] = False
    assert (store[around] == 9.0).all()


def test_ids_outside_the_range_are_ignored_by_the_backward():
    l, dw = logits_of(4, 16, torch.float32), torch.ones(4, 3, device="cuda")
    idx = torch.tensor([[0, 3, 5]] * 4, dtype=torch.int32, device="cuda")
    idx[1, 1], idx[2, 2], idx[3] = -1, 16, -7
    dl = moe.route_topk_backward(l, idx, dw, score="sigmoid", renormalize=False)
    assert ((dl != 0).sum(1).cpu() == torch.tensor([3, 2, 2, 0])).all()


def test_no_tokens():
    l = torch.empty(0, 16, device="cuda")
    idx, w = moe.route_topk(l, 2)
    assert idx.shape == w.shape == (0, 2)
    assert moe.route_topk_backward(l, idx, w).shape == (0, 16)


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
def test_autograd_against_differences(score, renormalize):
    """Central differences of the 64-bit weights with the choice held; their truncation from two steps."""
    l = logits_of(6, 24, torch.float32, 7)
    leaf = l.clone().requires_grad_()
    idx, w = moe.router(leaf, 4, score=score, renormalize=renormalize, scale=1.5)
    assert not idx.requires_grad and idx.dtype == torch.int32
    up = torch.randn(6, 4, generator=torch.Generator().manual_seed(2)).cuda()
    (w * up).sum().backward()
    at, upd = idx.long(), up.double()

    def f(z):
        a = z.gather(1, at)
        if score == "softmax":
            p = torch.exp(a - torch.logsumexp(a if renormalize else z, 1, keepdim=True))
        else:
            p = torch.sigmoid(a)
            p = p / p.sum(1, keepdim=True) if renormalize else p
        return (1.5 * p * upd).sum().item()

    for seed in range(3):
        v = torch.randn(6, 24, generator=torch.Generator().manual_seed(seed)).double().cuda()
        d = lambda h: (f(l.double() + h * v) - f(l.double() - h * v)) / (2 * h)
        got = (leaf.grad.double() * v).sum().item()
        # an element is at most 150 u (|g| + sum p |g|) p off (the bounds above at |l| < 5), p <= 1
        slack = 150 * U * 1.5 * (upd.abs().sum(1, keepdim=True) * 2 * v.abs()).sum().item()
        assert abs(got - d(1e-4)) <= slack + abs(d(2e-4) - d(1e-4))


def test_same_bits_streams_and_graph_replays():
    l = logits_of(500, 256, torch.float32, 1)
    dw = torch.randn(500, 8, device="cuda")

    def both(stream=None):
        idx, w = moe.route_topk(l, 8, n_group=8, topk_group=4, score="sigmoid", stream=stream)
        return [idx, w, moe.route_topk_backward(l, idx, dw, score="sigmoid", stream=stream)]

    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = both(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = both()
    for n in range(3):
        l.copy_(logits_of(500, 256, torch.float32, 50 + n))
        for t in held:
            t.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(both(), held)), n


def test_against_the_workloads_routing():
    """The routing that the layer's seeded workloads carry: the k largest logits, softmax over them."""
    w = mw.get("tiny_fwd")
    d = mw.inputs(w, 0)
    logits = np.random.default_rng([0, 0]).standard_normal((w.T, w.E), dtype=np.float32)
    idx, weights = moe.route_topk(torch.from_numpy(logits).cuda(), w.k)
    assert np.array_equal(idx.cpu().numpy(), d["topk_idx"])
    assert np.max(np.abs(weights.cpu().numpy() - d["topk_weights"])) <= 40 * U


def test_refusals():
    l = torch.ones(4, 16, device="cuda")
    idx, w = moe.route_topk(l, 2)
    for bad in (lambda: moe.route_topk(l.cpu(), 2), lambda: moe.route_topk(l, 17), lambda: moe.route_topk(l, 0), lambda: moe.route_topk(l.double(), 2),
                lambda: moe.route_topk(l, 2, bias=torch.ones(16)), lambda: moe.route_topk(l, 2, bias=torch.ones(15, device="cuda")),
                lambda: moe.route_topk(l, 2, score="relu"), lambda: moe.route_topk(l, 2, n_group=3), lambda: moe.route_topk(l, 2, n_group=4, topk_group=5),
                lambda: moe.route_topk(l[0], 2), lambda: moe.route_topk(l.t(), 2), lambda: moe.route_topk(torch.ones(1, 1025, device="cuda"), 2),
                lambda: moe.route_topk(l, 2, topk_idx=idx.long()), lambda: moe.route_topk(l, 2, topk_w=w[:3]),
                lambda: moe.route_topk_backward(l, idx, w[:, :1]), lambda: moe.route_topk_backward(l, idx.long(), w), lambda: moe.route_topk_backward(l, idx, w, dlogits=l),
                lambda: moe.route_topk_backward(l, idx, w, dlogits=torch.empty(4, 15, device="cuda"))):
        with pytest.raises(moe.MoeError):
            bad()
