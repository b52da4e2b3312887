"""The router's choice by score (bias and expert groups on the sigmoids or the softmax, not on the logits) against
its definition in 64 bits.

Bounds, u = 2^-24: e^a of the fast exponential is off by (2.5 |a| + 4) u relative, so a sigmoid s by
s (1 - s) (2.5 |l| + 4) u and two roundings of its own (sum, quotient); a softmax by that of its exponential
and of the sum's, and by the quotient's and the sum's roundings: a lane adds at most 32, six more steps join the lanes; adding the bias rounds once more, a group's sum of two as well.  Rows in which
two values that the choice has to order lie within the sum of their bounds have no one answer; all others
have to give the definition's ids, and with N(0, 1) logits these are nearly all."""
import numpy as np
import pytest
import torch

import token_dispatch_grouped_route_amd as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TINY = 1e-37


def values(l, score):
    """(scores, their bounds) of 64-bit logits, -inf (bound 0) out of service."""
    on = l > -np.inf
    with np.errstate(invalid="ignore", over="ignore"):
        if score == "sigmoid":
            e = np.exp(-np.abs(l))
            s = np.where(l >= 0, 1, e) / (1 + e)
            t = s * (1 - s) * (2.5 * np.minimum(np.abs(l), 104) + 4) * U + 3 * U * s + TINY
        else:
            m = np.max(np.where(on, l, -np.inf), 1, keepdims=True)
            e = np.where(on, np.exp(l - m), 0)
            s = e / e.sum(1, keepdims=True)
            far = np.where(on, np.minimum(m - l, 104), 0)
            of_sum = (np.where(on, s, 0) * (2.5 * far + 4)).sum(1, keepdims=True)
            t = s * (2.5 * far + 4 + of_sum + 40) * U + TINY
    return np.where(on, s, -np.inf), np.where(on, t, 0)


def apart(order, v, t, n):
    """Whether the first n + 1 of `order` are further apart than their bounds."""
    return all(v[b] == -np.inf or v[a] - v[b] > t[a] + t[b] for a, b in zip(order[:n], order[1:n + 1]))


def choose(v, t, k, n_group, topk_group):
    """(ids, whether they follow beyond the bounds) of one row."""
    E = len(v)
    sure = True
    if n_group > 1:
        size = E // n_group
        best = np.sort(v.reshape(n_group, size), 1)[:, ::-1]
        where = np.argsort(-v.reshape(n_group, size), 1, kind="stable")
        tt = np.take_along_axis(t.reshape(n_group, size), where, 1)
        two = (best[:, 1] > -np.inf) if size > 1 else np.zeros(n_group, bool)
        gv = np.where(two, best[:, 0] + (best[:, 1] if size > 1 else 0), best[:, 0])
        gt = tt.max(1) * 2 + np.where(two, U * np.abs(gv), 0)   # the second best may be another one within its bound
        order = sorted(range(n_group), key=lambda g: (-gv[g], g))
        if topk_group < n_group:
            a, b = order[topk_group - 1], order[topk_group]
            rest = [g for g in order[topk_group:] if gv[g] > -np.inf]
            sure = all(gv[x] - gv[y] > gt[x] + gt[y] for x in order[:topk_group] for y in rest) if gv[a] > -np.inf and gv[b] > -np.inf else True
        keep = np.isin(np.arange(E) // size, order[:topk_group])
        v = np.where(keep, v, -np.inf)
    order = sorted((e for e in range(E) if v[e] > -np.inf), key=lambda e: (-v[e], e))
    sure = sure and apart(order, v, t, k)
    return order[:k] + [-1] * (k - min(k, len(order))), sure


def check(logits, k, bias=None, score="sigmoid", n_group=1, topk_group=1, renormalize=True, most_open=0.05):
    idx, w = moe.route_topk(logits, k, bias=bias, score=score, renormalize=renormalize, n_group=n_group, topk_group=topk_group, scale=2.5, choice="score")
    l = logits.double().cpu().numpy()
    l = np.where(l > -np.inf, l, -np.inf)
    v, t = values(l, score)
    if bias is not None:
        v = v + bias.double().cpu().numpy()
        t = t + U * np.where(np.isfinite(v), np.abs(v), 0)
    got, want, opened = idx.cpu().numpy(), [], 0
    for r in range(len(l)):
        ids, sure = choose(v[r], t[r], k, n_group, topk_group)
        opened += not sure
        if sure:
            assert got[r].tolist() == ids, (r, got[r].tolist(), ids)
        real = got[r][got[r] >= 0]
        assert len(set(real.tolist())) == len(real)
        want.append(ids)
    assert opened <= most_open * len(l), (opened, len(l))
    # the weights are those of the ids, whatever chose them: without bias and groups taken over the ids alone
    a = logits.float().cpu().numpy().astype(np.float64)
    for r in range(len(l)):
        on = got[r] >= 0
        x = a[r, got[r][on]]
        if score == "sigmoid":
            p = 1 / (1 + np.exp(-x))
        else:
            p = np.exp(x - l[r].max())
        p = p / (p.sum() if renormalize else 1 if score == "sigmoid" else np.exp(l[r] - l[r].max()).sum())
        big = max(np.abs(x).max(), np.ptp(l[r][l[r] > -np.inf])) if len(x) else 0
        # the bounds of exp, log(sigmoid) and the sums at these logits, as relative ones
        assert (np.abs(w[r].double().cpu().numpy()[on] - 2.5 * p) <= 2.5 * p * (14 * big + 60 + l.shape[1]) * U + TINY).all()
        assert (w[r].cpu().numpy()[~on] == 0).all()
    return idx, w


def logits_of(T, E, dtype, seed=0):
    return torch.randn(T, E, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("score,renormalize", [("sigmoid", True), ("sigmoid", False), ("softmax", True), ("softmax", False)])
@pytest.mark.parametrize("E,n_group,topk_group,k,size", [
    (256, 8, 4, 8, 0.1), (256, 1, 1, 8, 0.01), (64, 4, 2, 6, 0.5), (96, 3, 2, 20, 0.1), (40, 5, 5, 3, 0.1), (512, 16, 1, 8, 0.02), (1000, 8, 3, 17, 0.5),
    (129, 1, 1, 4, 0.2), (7, 1, 1, 7, 0.1), (1024, 16, 16, 32, 0.3), (16, 16, 3, 3, 0.1), (2, 1, 1, 1, 0.3), (321, 3, 2, 12, 0.05)])
def test_bias_and_groups_on_the_scores(E, n_group, topk_group, k, size, score, renormalize, dtype):
    g = torch.Generator().manual_seed(E)
    l = logits_of(48, E, dtype, E)
    # 16-bit logits repeat, so their rows are told apart by biases that differ; a softmax's scores are about 1 / E
    bias = (size * torch.randn(E, generator=g) * (1 if score == "sigmoid" else 4 / E)).cuda()
    check(l, k, bias, score, n_group, topk_group, renormalize)
    if n_group > 1 and dtype == torch.float32:
        check(l, k, None, score, n_group, topk_group, renormalize)


def test_the_two_choices_differ_where_they_should():
    """One row worked out by hand: a bias of 0.2 lifts a sigmoid of 0.6 over one of 0.75, but not the logits they
    come from; a group of one expert at a logit of -1 does not outweigh two of -0.6."""
    l = torch.tensor([[0.405, 1.099, -9.0, -9.0]], device="cuda")
    bias = torch.tensor([0.2, 0.0, 0.0, 0.0], device="cuda")
    assert moe.route_topk(l, 1, bias=bias, score="sigmoid", choice="score")[0].item() == 0
    assert moe.route_topk(l, 1, bias=bias, score="sigmoid", choice="logit")[0].item() == 1
    assert moe.route_topk(l, 1, bias=bias, score="sigmoid")[0].item() == 1
    l = torch.tensor([[-1.0, -float("inf"), -0.6, -0.6]], device="cuda")
    assert moe.route_topk(l, 1, n_group=2, score="sigmoid", choice="score")[0].item() == 2
    assert moe.route_topk(l, 1, n_group=2, score="sigmoid")[0].item() == 0


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_without_bias_and_groups_the_choice_is_the_logits(score, dtype):
    l = logits_of(64, 200, dtype, 3)
    l[0] = 30 + torch.arange(200, device="cuda") / 8     # sigmoids that are all 1 in fp32
    for renormalize in (True, False):
        a = moe.route_topk(l, 9, score=score, renormalize=renormalize, choice="score")
        b = moe.route_topk(l, 9, score=score, renormalize=renormalize)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("n_group", [1, 4])
@pytest.mark.parametrize("E", [32, 252])
def test_equal_scores_go_to_the_lower_id(E, n_group):
    l = torch.zeros(4, E, device="cuda")
    l[0] = 40 + torch.randperm(E, generator=torch.Generator().manual_seed(1)).cuda()   # saturated: every sigmoid is 1
    l[1] = -0.5
    l[2] = torch.where(torch.arange(E, device="cuda") % 2 == 0, 0.0, -0.0)
    l[3] = -300.0 - torch.randperm(E, generator=torch.Generator().manual_seed(2)).cuda()   # every sigmoid is 0
    idx, w = moe.route_topk(l, 8, bias=torch.full((E,), 0.25, device="cuda"), score="sigmoid", n_group=n_group, topk_group=n_group, choice="score")
    assert idx.tolist() == [list(range(8))] * 4 and torch.isfinite(w).all()


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)])
@pytest.mark.parametrize("E,n_group,topk_group", [(16, 1, 1), (64, 4, 2), (520, 1, 1), (1024, 16, 3)])
def test_rows_with_few_or_no_experts(E, n_group, topk_group, score, renormalize):
    inf, nan = float("inf"), float("nan")
    l = logits_of(8, E, torch.float32, 5)
    l[0] = -inf
    l[1] = nan
    l[2] = -inf
    l[2, 5] = -3.0
    l[3, 1::2] = nan
    l[4, 7] = inf
    l[5] = -200.0       # in service with a sigmoid of 0
    l[6, 1:] = -inf
    l[7, :E // 2] = -inf
    bias = torch.linspace(-0.1, 0.1, E).cuda()
    idx, w = moe.route_topk(l, 4, bias=bias, score=score, renormalize=renormalize, n_group=n_group, topk_group=topk_group, choice="score")
    assert torch.isfinite(w).all()
    assert (idx[:2] == -1).all() and (w[:2] == 0).all() and idx[2].tolist() == [5, -1, -1, -1] and idx[6].tolist() == [0, -1, -1, -1]
    assert (idx[3] % 2 == 0).all() and (idx[7] >= E // 2).all() and (idx[5] >= 0).all()
    assert idx[5].tolist() == [E - 1, E - 2, E - 3, E - 4]     # equal scores: the bias decides
    # one certain expert takes the whole softmax, so it leads whatever a small bias says
    if score == "softmax":
        assert idx[4, 0].item() == 7
    bias[3::4], bias[0] = -inf, nan
    idx, _ = moe.route_topk(l, 4, bias=bias, score=score, renormalize=renormalize, n_group=n_group, topk_group=topk_group, choice="score")
    assert (idx % 4 != 3).all() or (idx[idx % 4 == 3] == -1).all()
    assert (idx != 0).all() and (idx[6] == -1).all()


def test_strided_rows_no_tokens_streams_and_graph_replays():
    wide = logits_of(300, 270, torch.float32, 1)
    l, bias = wide[:, 5:261], 0.1 * torch.randn(256, device="cuda")
    how = dict(bias=bias, score="sigmoid", n_group=8, topk_group=4, scale=2.5, choice="score")
    first = moe.route_topk(l, 8, **how)
    assert all(torch.equal(a, b) for a, b in zip(first, moe.route_topk(l.contiguous(), 8, **how)))
    assert moe.route_topk(l[:0], 8, **how)[0].shape == (0, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = moe.route_topk(l, 8, stream=side, **how)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = moe.route_topk(l, 8, **how)
    for n in range(3):
        wide.copy_(logits_of(300, 270, torch.float32, 70 + n))
        for t in held:
            t.fill_(77)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, moe.route_topk(l, 8, **how))), n


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_gradient_of_the_chosen(score):
    """The gradient is that of the weights of the ids, as for the choice by logit."""
    l = logits_of(20, 64, torch.float32, 4)
    bias = (0.2 * torch.randn(64, generator=torch.Generator().manual_seed(8))).cuda()
    leaf = l.clone().requires_grad_()
    idx, w = moe.router(leaf, 6, bias=bias, score=score, n_group=4, topk_group=2, scale=1.5, choice="score")
    up = torch.randn(20, 6, generator=torch.Generator().manual_seed(2)).cuda()
    w.backward(up)
    assert torch.equal(leaf.grad, moe.route_topk_backward(l, idx, up, score=score, scale=1.5))
    z = l.double().cpu().requires_grad_()
    a = z.gather(1, idx.cpu().long())
    p = torch.softmax(a, 1) if score == "softmax" else torch.sigmoid(a) / torch.sigmoid(a).sum(1, keepdim=True)
    (1.5 * p * up.double().cpu()).sum().backward()
    # an element: p (g - q) (1 - s), each within 150 u at |l| < 5 (exp, log(sigmoid), sums of six terms), p and q of the magnitudes
    mag = 1.5 * up.double().cpu().abs().sum(1, keepdim=True)
    assert ((leaf.grad.double().cpu() - z.grad).abs() <= 150 * U * 2 * mag).all()


def test_refused_choice():
    l = torch.ones(4, 16, device="cuda")
    for bad in ("scores", None, 1):
        with pytest.raises(moe.MoeError):
            moe.route_topk(l, 2, choice=bad)
        with pytest.raises(moe.MoeError):
            moe.router(l, 2, choice=bad)


@pytest.mark.parametrize("choice", ["logit", "score"])
def test_a_bias_of_minus_infinity_bars_from_the_choice_alone(choice):
    """The softmax over all runs over every expert whose logit is usable, barred by its bias or not, and so does its
    gradient; an expert whose logit is out of service has no part in either."""
    E, k = 40, 5
    l = logits_of(30, E, torch.float32, 11)
    l[:, 7] = -float("inf")
    bias = torch.zeros(E, device="cuda")
    bias[::3] = -float("inf")
    idx, w = moe.route_topk(l, k, bias=bias, renormalize=False, choice=choice)
    assert (idx % 3 != 0).all() and (idx != 7).all() and (idx >= 0).all()
    z = l.double().cpu().requires_grad_()
    p = torch.softmax(z, 1).gather(1, idx.cpu().long())
    # relative, at |l - m| < 10: two exponentials within 29 u, 46 additions
    assert ((w.double().cpu() - p).abs() <= 110 * U * p).all()
    free, _ = moe.route_topk(l[:, torch.arange(E, device="cuda") % 3 != 0].contiguous(), k)
    assert torch.equal(free, idx - idx // 3 - 1)
    up = torch.randn(30, k, generator=torch.Generator().manual_seed(2))
    (p * up.double()).sum().backward()
    got = moe.route_topk_backward(l, idx, up.cuda(), renormalize=False).double().cpu()
    assert (got[:, 7] == 0).all() and (got[:, ::3] != 0).all()
    assert ((got - z.grad).abs() <= 150 * U * 2 * up.double().abs().sum(1, keepdim=True)).all()
