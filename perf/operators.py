"""The operators around the expert layer and their 4-bit serving form, as a user calls them.

Four operators: the row norm (layer norm and RMS norm, forward and backward), the top-k router
(logits to expert ids and weights, forward and backward), products of a few rows with 4-bit
group-scaled weights, and the expert layer on such weights for a few tokens.

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits, rounded once
at the end; with ``own`` true it calls token_dispatch_grouped_route_amd.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
NORM_EPS = 1e-5
F32_MAX = torch.finfo(torch.float32).max


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # decoding: one token in front of the expert layer at hidden size 7168; latency only
        norm_case("rms_one_token", "fwd", "rms", 1, 7168, "bf16", False),
        # a training batch of 8192 tokens in front of the layer
        norm_case("layer_norm_fwd", "fwd", "layer", 8192, 7168, "bf16", True),
        # a ragged batch in full precision, with a hidden size that divides into no vector
        norm_case("layer_norm_bwd_odd", "bwd", "layer", 1003, 5001, "fp32", True),
        # the rows one GPU of eight receives: the largest batch the layer is run on
        norm_case("rms_bwd_page", "bwd", "rms", 65536, 7168, "bf16", False),
        # the smallest routing: 256 tokens, 8 experts, top-2
        route_case("route_tiny", "fwd", 256, 8, 2, "fp32", "softmax", True),
        # sigmoid scores, a balancing bias and group-limited selection, 256 experts, top-8
        route_case("route_groups", "fwd", 8192, 256, 8, "fp32", "sigmoid", True, bias=True, n_group=8, topk_group=4, scale=2.5),
        # 384 experts, top-6, 16-bit logits (many ties), some experts taken out of service
        route_case("route_wide", "fwd", 65536, 384, 6, "bf16", "softmax", True, masked=True),
        # the router's training step at the page-scale batch, weights not renormalised (every logit gets a gradient)
        route_case("route_bwd", "bwd", 65536, 256, 8, "fp32", "softmax", False),
        # one token through one expert-sized projection (7168 to [gate | up] of 2048)
        linear_case("w4_one_token", 1, 7168, 4096, 128, "bf16", False),
        # a decode batch of 48 through the way back, zero points, groups of 64
        linear_case("w4_batch", 48, 2048, 7168, 64, "fp16", True),
        # one token through a whole layer of 64 small experts, top-6
        experts_case("experts_one_token", 1, 2048, 1408, 64, 64, 6, 128, "bf16", False),
        # a decode batch of 64 through one GPU's 32 of 256 experts, fine groups, zero points
        experts_case("experts_batch", 64, 7168, 2048, 256, 32, 8, 32, "bf16", True),
    ]


def norm_case(name, way, kind, rows, cols, dtype, bias):
    return {"name": name, "op": "norm", "way": way, "kind": kind, "rows": rows, "cols": cols, "dtype": dtype, "bias": bias}


def route_case(name, way, T, E, k, dtype, score, renorm, bias=False, masked=False, n_group=1, topk_group=1, scale=1.0):
    return {"name": name, "op": "route", "way": way, "T": T, "E": E, "k": k, "dtype": dtype, "score": score, "renorm": renorm,
            "bias": bias, "masked": masked, "n_group": n_group, "topk_group": topk_group, "scale": scale}


def linear_case(name, M, K, N, group, dtype, zeros):
    return {"name": name, "op": "linear", "M": M, "K": K, "N": N, "group": group, "dtype": dtype, "zeros": zeros}


def experts_case(name, T, H, I, E, EL, k, group, dtype, zeros):
    return {"name": name, "op": "experts", "T": T, "H": H, "I": I, "E": E, "EL": EL, "k": k, "group": group, "dtype": dtype,
            "zeros": zeros}


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes over the whole range of their operator, odd ones among them."""
    op = rng.choice(("norm", "route", "linear", "experts"))
    if op == "norm":
        cols = log_int(rng, 64, 16384)
        rows = log_int(rng, 1, min(65536, 65536 * 7168 // cols // 2))
        kind = rng.choice(("layer", "rms"))
        c = norm_case("", rng.choice(("fwd", "bwd")), kind, rows, cols, rng.choice(("bf16", "fp16", "fp32")),
                      kind == "layer" and rng.random() < 0.8)
    elif op == "route":
        n_group = rng.choice((1, 1, 2, 4, 8))
        E = n_group * log_int(rng, max(2, 8 // n_group), 512 // n_group)
        topk_group = rng.randint(1, n_group)
        k = min(rng.choice((1, 2, 4, 6, 8, 8, 16)), E // n_group * topk_group)
        renorm = rng.random() < 0.6 and k > 1   # one renormalised weight is 1, and its gradient 0
        c = route_case("", rng.choice(("fwd", "bwd")), log_int(rng, 1, 65536), E, k, rng.choice(("bf16", "fp16", "fp32")),
                       rng.choice(("softmax", "sigmoid")), renorm, rng.random() < 0.4, rng.random() < 0.3, n_group, topk_group,
                       rng.choice((1.0, 2.5)))
    elif op == "linear":
        group = rng.choice((32, 64, 128))
        c = linear_case("", log_int(rng, 1, 64), 128 * log_int(rng, 2, 64), log_int(rng, 128, 16384), group,
                        rng.choice(("bf16", "fp16")), rng.random() < 0.5)
    else:
        EL = rng.choice((8, 16, 32))
        E = EL * rng.choice((1, 2, 8))
        c = experts_case("", log_int(rng, 1, 128), 128 * log_int(rng, 4, 56), 128 * log_int(rng, 2, 16), E, EL,
                         rng.choice((1, 2, 4, 6, 8)), rng.choice((32, 64, 128)), rng.choice(("bf16", "fp16")), rng.random() < 0.5)
    c.pop("name")
    return c


def work(case):
    """Bytes and flops of one pass: every input read once, every output written once."""
    c, sz = case, BYTES[case["dtype"]]
    if c["op"] == "norm":
        n = c["rows"] * c["cols"]
        stats = c["rows"] * 4 * (2 if c["kind"] == "layer" else 1)
        w = c["cols"] * sz * (2 if c["bias"] else 1)
        if c["way"] == "fwd":
            return {"bytes": 2 * n * sz + w + stats, "flops": 8 * n}
        return {"bytes": 3 * n * sz + c["cols"] * sz + w + stats, "flops": 14 * n}
    if c["op"] == "route":
        n, p = c["T"] * c["E"], c["T"] * c["k"]
        if c["way"] == "fwd":
            return {"bytes": n * sz + 8 * p + 4 * c["E"] * c["bias"], "flops": 2 * n}
        # a renormalised weight depends on the chosen logits alone, the softmax over all on all of them
        read = n if c["score"] == "softmax" and not c["renorm"] else p
        return {"bytes": (n + read) * sz + 8 * p, "flops": 4 * n}
    if c["op"] == "linear":
        return {"bytes": weight_bytes(c, c["N"], c["K"]) + c["M"] * (c["K"] + c["N"]) * sz, "flops": 2 * c["M"] * c["N"] * c["K"]}
    # local experts that a uniform batch reaches, each streamed once; its local pairs
    hit = c["EL"] * (1 - (1 - c["k"] / c["E"]) ** c["T"]) if c["k"] < c["E"] else c["EL"]
    pairs = c["T"] * c["k"] * c["EL"] / c["E"]
    per = weight_bytes(c, 2 * c["I"], c["H"]) + weight_bytes(c, c["H"], c["I"])
    return {"bytes": hit * per + 2 * c["T"] * c["H"] * sz + 8 * c["T"] * c["k"], "flops": 6 * pairs * c["H"] * c["I"]}


def weight_bytes(c, N, K):
    return N * K / 2 + N * (K // c["group"]) * (BYTES[c["dtype"]] + (1 if c["zeros"] else 0))


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def prepare(case, seed):
    """Inputs on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": dict(case)}
    {"norm": norm_inputs, "route": route_inputs, "linear": linear_inputs, "experts": experts_inputs}[case["op"]](state, case, g)
    return state


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def norm_inputs(s, c, g):
    dt = DTYPES[c["dtype"]]
    R, C = c["rows"], c["cols"]
    # rows of a residual stream: each with a size and an offset of its own
    x = normal(g, R, C) * (0.5 + 2 * torch.rand(R, 1, generator=g, device="cuda")) + 0.3 * normal(g, R, 1)
    s["x"] = x.to(dt)
    s["weight"] = (1 + 0.2 * normal(g, C)).to(dt)
    s["bias"] = (0.1 * normal(g, C)).to(dt) if c["bias"] else None
    if c["way"] == "bwd":
        x = s["x"].float()
        mean = x.mean(1) if c["kind"] == "layer" else None
        centred = x - mean[:, None] if mean is not None else x
        s["mean"], s["rstd"] = mean, torch.rsqrt(centred.square().mean(1) + NORM_EPS)
        s["dy"] = normal(g, R, C).to(dt)


def route_inputs(s, c, g):
    T, E = c["T"], c["E"]
    logits = normal(g, T, E)
    if c["masked"]:   # about a tenth of the experts out of service
        logits = logits.masked_fill(torch.rand(E, generator=g, device="cuda") < 0.1, -math.inf)
    s["logits"] = logits.to(DTYPES[c["dtype"]])
    s["bias"] = 0.1 * normal(g, E) if c["bias"] else None
    if c["way"] == "bwd":
        s["topk_idx"] = chosen(c, s["logits"], s["bias"])
        s["dtopk_w"] = normal(g, T, c["k"])


def w4_weights(c, g, E, N, K):
    """Codes, scales and zero points of [E, N, K] weights of the size 1 / sqrt(K)."""
    groups = K // c["group"]
    codes = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = ((0.5 + torch.rand(E, N, groups, generator=g, device="cuda")) / (4.6 * math.sqrt(K))).to(DTYPES[c["dtype"]])
    zeros = torch.randint(5, 11, (E, N, groups), generator=g, device="cuda", dtype=torch.uint8) if c["zeros"] else None
    return codes, scales, zeros


def linear_inputs(s, c, g):
    s["x"] = normal(g, c["M"], c["K"]).to(DTYPES[c["dtype"]])
    s["w"] = tuple(t[0] if t is not None else None for t in w4_weights(c, g, 1, c["N"], c["K"]))


def experts_inputs(s, c, g):
    T, E = c["T"], c["E"]
    s["x"] = normal(g, T, c["H"]).to(DTYPES[c["dtype"]])
    top, idx = torch.sort(normal(g, T, E), dim=1, descending=True, stable=True)
    s["topk_idx"] = idx[:, :c["k"]].to(torch.int32).contiguous()
    s["topk_w"] = torch.softmax(top[:, :c["k"]], dim=1)
    s["w1"] = w4_weights(c, g, c["EL"], 2 * c["I"], c["H"])
    s["w2"] = w4_weights(c, g, c["EL"], c["H"], c["I"])


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(state):
    c = state["case"]
    if own:
        return own_run(state, c)
    return {"norm": plain_norm, "route": plain_route, "linear": plain_linear, "experts": plain_experts}[c["op"]](state, c)


def own_run(s, c):
    import token_dispatch_grouped_route_amd as moe

    if c["op"] == "norm":
        if c["way"] == "fwd":
            y, mean, rstd = moe.norm_forward(s["x"], s["weight"], s["bias"], eps=NORM_EPS, kind=c["kind"])
            return {"y": y, "mean": mean, "rstd": rstd}
        dx, dw, db = moe.norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], kind=c["kind"], bias=c["bias"])
        return {"dx": dx, "dw": dw, "db": db}
    if c["op"] == "route":
        how = {"score": c["score"], "renormalize": c["renorm"], "scale": c["scale"]}
        if c["way"] == "fwd":
            idx, w = moe.route_topk(s["logits"], c["k"], bias=s["bias"], n_group=c["n_group"], topk_group=c["topk_group"], **how)
            return {"topk_idx": idx, "topk_w": w}
        return {"dlogits": moe.route_topk_backward(s["logits"], s["topk_idx"], s["dtopk_w"], **how)}
    if c["op"] == "linear":
        return {"y": moe.w4_linear(s["x"], *s["w"])}
    if "shape" not in s:   # the shape and the workspace that a serving program keeps
        s["shape"] = moe.make_shape(c["T"], c["H"], c["I"], c["E"], c["EL"], c["k"])
        s["ws"] = moe.w4_alloc_workspace(s["shape"])
    return {"y": moe.forward_w4(s["shape"], s["x"], s["topk_idx"], s["topk_w"], s["w1"], s["w2"], s["ws"])}


def plain_norm(s, c):
    x, w = s["x"].float(), s["weight"].float()
    dt = s["x"].dtype
    if c["way"] == "fwd":
        mean = x.mean(1) if c["kind"] == "layer" else None
        xc = x - mean[:, None] if mean is not None else x
        rstd = 1 / torch.sqrt((xc * xc).mean(1) + NORM_EPS)
        y = xc * rstd[:, None] * w
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return {"y": y.to(dt), "mean": mean, "rstd": rstd}
    dy, rstd = s["dy"].float(), s["rstd"][:, None]
    xh = (x - s["mean"][:, None] if s["mean"] is not None else x) * rstd
    g = dy * w
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if c["kind"] == "layer":
        dx = dx - g.mean(1, keepdim=True)
    return {"dx": (dx * rstd).to(dt), "dw": (dy * xh).sum(0).to(dt), "db": dy.sum(0).to(dt) if c["bias"] else None}


def usable(logits):
    """fp32 logits, +inf as the largest finite number, and which experts they leave in service."""
    l = logits.float()
    return l.clamp(max=F32_MAX), l > -math.inf   # false for NaN too


def chosen(c, logits, bias):
    """int32 [T, k]: the experts of the largest scores (ties: the lower one), -1 where none is left."""
    l, valid = usable(logits)
    T, E, G = c["T"], c["E"], c["n_group"]
    score = torch.where(valid, l + bias if bias is not None else l, -math.inf)
    if G > 1:
        best = torch.sort(score.view(T, G, E // G), dim=2, descending=True).values
        first = best[:, :, 0]
        if E // G > 1:
            second = best[:, :, 1]
            first = torch.where(second > -math.inf, first + second, first)
        order = torch.sort(first, dim=1, descending=True, stable=True).indices[:, :c["topk_group"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=logits.device).scatter(1, order, True)
        score = torch.where(keep[:, :, None].expand(T, G, E // G).reshape(T, E), score, -math.inf)
    top, idx = torch.sort(score, dim=1, descending=True, stable=True)
    return torch.where(top > -math.inf, idx, -1)[:, :c["k"]].to(torch.int32)


def plain_route(s, c):
    l, valid = usable(s["logits"])
    idx = chosen(c, s["logits"], s["bias"]) if c["way"] == "fwd" else s["topk_idx"]
    there = idx >= 0
    at = idx.clamp(min=0).long()
    picked = l.gather(1, at)
    # softmax weights: exp(l - max) over a sum; sigmoid weights alike, with log(sigmoid(l)) for l
    sig = torch.where(picked >= 0, 1 / (1 + torch.exp(-picked)), torch.exp(picked.clamp(max=0)) / (1 + torch.exp(picked.clamp(max=0))))
    log_sig = picked.clamp(max=0) - torch.log1p(torch.exp(-picked.abs()))
    if c["renorm"]:
        v = torch.where(there, picked if c["score"] == "softmax" else log_sig, -math.inf)
        e = torch.where(there, torch.exp(v - v.amax(1, keepdim=True)), 0.0)
        p = torch.where(there, e / e.sum(1, keepdim=True), 0.0)
    elif c["score"] == "softmax":
        v = torch.where(valid, l, -math.inf)
        top = v.amax(1, keepdim=True)
        every = torch.where(valid, torch.exp(v - top), 0.0)
        every = torch.where(valid, every / every.sum(1, keepdim=True), 0.0)
        p = torch.where(there, every.gather(1, at), 0.0)
    else:
        p = torch.where(there, sig, 0.0)
    if c["way"] == "fwd":
        return {"topk_idx": idx, "topk_w": p * c["scale"]}
    g = torch.where(there, s["dtopk_w"], 0.0) * c["scale"]
    d = p * (g - (p * g).sum(1, keepdim=True)) if c["renorm"] else p * g
    if c["score"] == "sigmoid":   # 1 - sigmoid(l) = sigmoid(-l)
        d = d * torch.where(picked >= 0, torch.exp(-picked.clamp(min=0)) / (1 + torch.exp(-picked.clamp(min=0))), 1 / (1 + torch.exp(picked)))
    out = torch.zeros_like(l).scatter_add(1, at, torch.where(there, d, 0.0))
    if c["score"] == "softmax" and not c["renorm"]:
        out = out - every * (p * g).sum(1, keepdim=True)
    return {"dlogits": out.to(s["logits"].dtype)}


def plain_weights(codes, scales, zeros):
    """The fp32 weights [..., N, K] of codes, scales and zero points."""
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).float()
    q = q.unflatten(-1, (scales.shape[-1], -1))
    q = q - (zeros.float()[..., None] if zeros is not None else 8.0)
    return (q * scales.float()[..., None]).flatten(-2)


def plain_linear(s, c):
    return {"y": (s["x"].float() @ plain_weights(*s["w"]).t()).to(s["x"].dtype)}


def plain_experts(s, c):
    """The routed experts, each on its token where there are fewer pairs than experts, else every local
    expert on every token; then the routed ones weighted and summed."""
    x, T, k, EL = s["x"].float(), c["T"], c["k"], c["EL"]
    local = s["topk_idx"] < EL   # this GPU owns the experts [0, EL)
    ids = s["topk_idx"].clamp(max=EL - 1).long()
    few = T * k < EL
    if few:
        x = x.repeat_interleave(k, 0)[:, None]   # [T k, 1, H]
    w1, w2 = ((t[ids.flatten()] if few and t is not None else t for t in s[n]) for n in ("w1", "w2"))
    h = torch.matmul(x, plain_weights(*w1).transpose(1, 2).contiguous())   # [experts, rows, 2I]
    gate, up = h[..., :c["I"]], h[..., c["I"]:]
    o = torch.matmul(gate / (1 + torch.exp(-gate)) * up, plain_weights(*w2).transpose(1, 2).contiguous())
    rows = o.view(T, k, -1) if few else o[ids, torch.arange(T, device=x.device)[:, None]]
    w = torch.where(local, s["topk_w"], 0.0)
    return {"y": (rows * w[..., None]).sum(1).to(s["x"].dtype)}


# ------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": exact_norm, "route": exact_route, "linear": exact_linear, "experts": exact_experts}[case["op"]](s, case)


def exact_norm(s, c):
    layer = c["kind"] == "layer"
    outs = {}
    w, b = s["weight"].double(), s["bias"]
    if c["way"] == "fwd":
        mean, rstd, y = [], [], []
        for x in s["x"].split(4096):
            x = x.double()
            m = x.mean(1) if layer else torch.zeros(len(x), dtype=torch.float64, device=x.device)
            r = ((x - m[:, None]) ** 2).mean(1).add(NORM_EPS) ** -0.5
            out = (x - m[:, None]) * r[:, None] * w
            y.append(out + b.double() if b is not None else out)
            mean.append(m)
            rstd.append(r)
        return {"y": torch.cat(y), "mean": torch.cat(mean) if layer else None, "rstd": torch.cat(rstd)}
    dx, dw, db = [], 0.0, 0.0
    for i in range(0, c["rows"], 4096):
        x, dy, r = s["x"][i:i + 4096].double(), s["dy"][i:i + 4096].double(), s["rstd"][i:i + 4096].double()[:, None]
        z = (x - s["mean"][i:i + 4096].double()[:, None]) * r if layer else x * r
        # the Jacobian of z: r (I - 1 1' / C [layer] - z z' / C), applied to w dy
        v = w * dy
        u = v - z * ((z * v).sum(1, keepdim=True) / c["cols"])
        dx.append(r * (u - v.sum(1, keepdim=True) / c["cols"] if layer else u))
        dw, db = dw + (dy * z).sum(0), db + dy.sum(0)
    outs = {"dx": torch.cat(dx), "dw": dw, "db": db if c["bias"] else None}
    return outs


def exact_route(s, c):
    T, E, k, G = c["T"], c["E"], c["k"], c["n_group"]
    z = s["logits"].float().clamp(max=F32_MAX)
    z = z.masked_fill(~(z > -math.inf), -math.inf)
    ids = torch.arange(E, device=z.device)
    rows = torch.arange(T, device=z.device)

    def first_best(score, n):
        """The lowest index of the largest score of each row."""
        best = score.amax(1, keepdim=True)
        return torch.where(score == best, ids[:n], n).amin(1).clamp(max=n - 1)

    if c["way"] == "fwd":
        score = z + s["bias"] if s["bias"] is not None else z.clone()   # the 32-bit score is the definition's
        if G > 1:
            parts = score.view(T, G, E // G)
            gs = parts.amax(2)
            if E // G > 1:
                two = parts.topk(2, dim=2).values.sum(2)
                gs = torch.where(two > -math.inf, two, gs)
            kept = torch.zeros(T, G, dtype=torch.bool, device=z.device)
            for _ in range(c["topk_group"]):
                j = first_best(gs.masked_fill(kept, -math.inf), G)
                kept[rows, j] |= gs[rows, j] > -math.inf
            score = score.masked_fill(~kept.repeat_interleave(E // G, 1), -math.inf)
        picks = []
        for _ in range(k):
            j = first_best(score, E)
            picks.append(torch.where(score[rows, j] > -math.inf, j, -1))
            score[rows, j] = -math.inf
        idx = torch.stack(picks, 1)
    else:
        idx = s["topk_idx"].long()
    hit = idx >= 0
    z = z.double()
    a = z[rows[:, None], idx.clamp(min=0)].masked_fill(~hit, -math.inf)
    sigma = torch.sigmoid(a)
    if c["score"] == "softmax":
        norm = torch.logsumexp(a if c["renorm"] else z, 1, keepdim=True)
        p = torch.exp(a - norm)
    elif c["renorm"]:
        p = torch.softmax(torch.nn.functional.logsigmoid(a), 1)
    else:
        p = sigma
    p = torch.where(hit, p, 0.0)
    if c["way"] == "fwd":
        return {"topk_idx": None, "topk_w": c["scale"] * p}
    up = c["scale"] * s["dtopk_w"].double() * p
    d = up - p * up.sum(1, keepdim=True) if c["renorm"] else up
    if c["score"] == "sigmoid":
        d = d * torch.sigmoid(-a)
    grad = torch.zeros(T, E + 1, dtype=torch.float64, device=z.device)
    grad.scatter_(1, torch.where(hit, idx, E), torch.where(hit, d, 0.0))
    grad = grad[:, :E]
    if c["score"] == "softmax" and not c["renorm"]:
        grad = grad - torch.nan_to_num(torch.exp(z - norm)) * up.sum(1, keepdim=True)
    return {"dlogits": grad}


def exact_matrix(codes, scales, zeros, group):
    """[N, K] weights in 64 bits of one expert."""
    N, half = codes.shape
    w = torch.empty(N, 2 * half, dtype=torch.float64, device=codes.device)
    w[:, 0::2] = codes.remainder(16).double()
    w[:, 1::2] = codes.div(16, rounding_mode="floor").double()
    w -= zeros.double().repeat_interleave(group, 1) if zeros is not None else 8.0
    return w * scales.double().repeat_interleave(group, 1)


def exact_linear(s, c):
    return {"y": torch.mm(s["x"].double(), exact_matrix(*s["w"], c["group"]).t())}


def exact_experts(s, c):
    y = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
    for e in range(c["EL"]):
        token, slot = torch.nonzero(s["topk_idx"] == e, as_tuple=True)
        if not len(token):
            continue
        one = [t[e] if t is not None else None for t in s["w1"]]
        two = [t[e] if t is not None else None for t in s["w2"]]
        h = torch.mm(s["x"][token].double(), exact_matrix(*one, c["group"]).t())
        a = torch.nn.functional.silu(h[:, :c["I"]]) * h[:, c["I"]:]
        y.index_add_(0, token, torch.mm(a, exact_matrix(*two, c["group"]).t()) * s["topk_w"][token, slot].double()[:, None])
    return {"y": y}
