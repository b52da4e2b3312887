"""The dense operators of a block around the expert layer, and the expert layer's own form for few tokens, as
a user calls them.

Three operators: the linear map with bias, activation and residual in its epilogue (forward and backward: the
router's gate product, shared experts, dense layers), the block norm (the norm after a block, its gate, the
scaled residual sum and the norm before the next block in one pass; forward and backward), and the expert layer
on packed bf16 weights for the few tokens of a decode step.

With ``own`` false, ``run`` computes them from elementary torch operations in 32 bits, rounded once at the end;
with ``own`` true it calls token_dispatch_grouped_route_amd.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5


# ------------------------------------------------------------------------------------------------
# cases
# ------------------------------------------------------------------------------------------------
def listed():
    return [
        # decoding: one token through a shared expert's [gate | up] projection
        linear_case("linear_one_token", "fwd", 1, 7168, 2048, "bf16", "swiglu"),
        # a decode batch of 48 on its way back into the residual stream, weights stored by output column
        linear_case("linear_decode_back", "fwd", 48, 2048, 7168, "fp16", None, bias=True, residual=True, layout="nk"),
        # a training batch through a shared expert's [gate | up] projection
        linear_case("linear_shared_expert", "fwd", 8192, 7168, 2048, "bf16", "swiglu"),
        # the router's gate product: few columns, fp32 logits
        linear_case("linear_gate", "fwd", 8192, 7168, 256, "bf16", None, out="fp32"),
        # its training step: the gradients of the shared expert's projection
        linear_case("linear_shared_expert_bwd", "bwd", 8192, 7168, 2048, "bf16", "swiglu"),
        # a ragged batch and sizes that divide into no tile or vector
        linear_case("linear_bwd_odd", "bwd", 1003, 2049, 1407, "fp16", "gelu", bias=True),
        # decoding: one token between two blocks; latency only
        block_case("block_norm_one_token", "fwd", "rms", 1, 7168, "bf16", post=True, pre=True),
        # a training batch, the residual stream in fp32, a learned gate on the block's output
        block_case("block_norm_fwd", "fwd", "rms", 8192, 7168, "bf16", stream="fp32", post=True, gate=1, pre=True),
        # its training step with a 16-bit residual stream
        block_case("block_norm_bwd", "bwd", "rms", 8192, 7168, "bf16", post=True, gate=1, pre=True),
        # 17 samples of 59 tokens, each with a gate of its own, in full precision, an odd hidden size
        block_case("block_norm_bwd_odd", "bwd", "layer", 1003, 5001, "fp32", post=True, gate=17, pre=True, bias=True, scale=0.22),
        # one token through a whole layer of 64 small experts, top-6
        experts_case("experts_one_token", 1, 2048, 1408, 64, 64, 6),
        # a decode batch of 64 through one GPU's 32 of 256 experts
        experts_case("experts_batch", 64, 7168, 2048, 256, 32, 8),
    ]


def linear_case(name, way, M, K, N, dtype, act, bias=False, residual=False, layout="kn", out="same"):
    """y [M, N]; the weight has 2N columns where act is swiglu.  layout nk: the weight lies as [N, K]."""
    return {"name": name, "op": "linear", "way": way, "M": M, "K": K, "N": N, "dtype": dtype, "act": act or "none", "bias": bias,
            "residual": residual, "layout": layout, "out": out}


def block_case(name, way, kind, rows, cols, dtype, stream="same", post=False, gate=0, pre=False, bias=False, x_scale=1.0, scale=1.0):
    """gate: rows of the gate (0: none), each for an equal share of the rows; stream: the residual stream's type."""
    return {"name": name, "op": "block", "way": way, "kind": kind, "rows": rows, "cols": cols, "dtype": dtype, "stream": stream, "post": post,
            "gate": gate, "pre": pre, "bias": bias, "x_scale": x_scale, "scale": scale}


def experts_case(name, T, H, I, E, EL, k):
    return {"name": name, "op": "experts", "T": T, "H": H, "I": I, "E": E, "EL": EL, "k": k, "dtype": "bf16"}


def log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: sizes over the whole range of their operator, odd ones among them."""
    op = rng.choice(("linear", "linear", "block", "block", "experts"))
    if op == "linear":
        way = rng.choice(("fwd", "fwd", "bwd"))
        act = rng.choice((None, "relu", "gelu", "silu", "swiglu"))
        K, N = log_int(rng, 32, 7168), log_int(rng, 32, 4096)
        if rng.random() < 0.6:   # most models' sizes divide by something
            K, N = 64 * max(1, K // 64), 32 * max(1, N // 32)
        M = log_int(rng, 1, 64) if way == "fwd" and rng.random() < 0.4 else log_int(rng, 1, 8192)
        c = linear_case("", way, M, K, N, rng.choice(("bf16", "fp16")), act, rng.random() < 0.5, way == "fwd" and rng.random() < 0.4,
                        rng.choice(("kn", "nk")), rng.choice(("same", "same", "fp32")))
    elif op == "block":
        cols = log_int(rng, 64, 16384)
        share = log_int(rng, 1, min(8192, 8192 * 7168 // cols))
        groups = rng.choice((0, 0, 1, 1, 2, 5, 16))
        rows = max(1, share // max(1, groups)) * max(1, groups)
        kind = rng.choice(("rms", "layer"))
        post = rng.random() < 0.6
        c = block_case("", rng.choice(("fwd", "bwd")), kind, rows, cols, rng.choice(("bf16", "fp16", "fp32")), rng.choice(("same", "same", "fp32")),
                       post, groups, not post or rng.random() < 0.7, kind == "layer" and rng.random() < 0.7, rng.choice((1.0, 1.0, 1.86)),
                       rng.choice((1.0, 1.0, 0.22)))
    else:
        EL = rng.choice((8, 16, 32))
        E = EL * rng.choice((1, 2, 8))
        c = experts_case("", log_int(rng, 1, 128), 128 * log_int(rng, 4, 56), 128 * log_int(rng, 2, 16), E, EL, rng.choice((1, 2, 4, 6, 8)))
    c.pop("name")
    return c


def columns(c):
    return 2 * c["N"] if c["act"] == "swiglu" else c["N"]


def stream_bytes(c):
    return BYTES[c["dtype"] if c["stream"] == "same" else c["stream"]]


def work(case):
    """Bytes and flops of one pass: every input read once, every output written once."""
    c, sz = case, BYTES[case["dtype"]]
    if c["op"] == "linear":
        M, K, N, W = c["M"], c["K"], c["N"], columns(c)
        out = BYTES["fp32"] if c["out"] == "fp32" else sz
        if c["way"] == "fwd":
            return {"bytes": (M * K + K * W + W * c["bias"]) * sz + M * N * out * (2 if c["residual"] else 1), "flops": 2 * M * K * W}
        saved = M * W * sz if c["act"] != "none" else 0
        return {"bytes": 2 * (M * K + K * W) * sz + saved + M * N * out + W * sz * c["bias"], "flops": 4 * M * K * W}
    if c["op"] == "block":
        n, rs = c["rows"] * c["cols"], stream_bytes(c)
        vectors = (c["post"] + c["pre"]) * (1 + c["bias"]) + c["gate"]
        stats = 4 * c["rows"] * (c["post"] + c["pre"]) * (2 if c["kind"] == "layer" else 1)
        if c["way"] == "fwd":   # read x, b; write r and n
            return {"bytes": n * (2 * rs + sz * (1 + c["pre"])) + vectors * c["cols"] * sz + stats, "flops": 8 * n * (c["post"] + c["pre"]) + 3 * n}
        # read dr, b and, before a norm, r and dn; write dx, db and the vectors' gradients.  Without norm and gate b is not read
        reads = rs + (sz if c["post"] or c["gate"] else 0) + (rs + sz if c["pre"] else 0)
        return {"bytes": n * (reads + rs + sz) + 2 * vectors * c["cols"] * sz + stats, "flops": 14 * n * (c["post"] + c["pre"]) + 5 * n}
    # local experts that a uniform batch reaches, each streamed once; its local pairs
    hit = c["EL"] * (1 - (1 - c["k"] / c["E"]) ** c["T"]) if c["k"] < c["E"] else c["EL"]
    pairs = c["T"] * c["k"] * c["EL"] / c["E"]
    return {"bytes": hit * 6 * c["H"] * c["I"] + 4 * c["T"] * c["H"] + 8 * c["T"] * c["k"], "flops": 6 * pairs * c["H"] * c["I"]}


# ------------------------------------------------------------------------------------------------
# inputs
# ------------------------------------------------------------------------------------------------
def prepare(case, seed):
    """Inputs on the GPU, from the seed alone."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": dict(case)}
    {"linear": linear_inputs, "block": block_inputs, "experts": experts_inputs}[case["op"]](state, case, g)
    return state


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def linear_inputs(s, c, g):
    dt = DTYPES[c["dtype"]]
    M, K, N, W = c["M"], c["K"], c["N"], columns(c)
    out = torch.float32 if c["out"] == "fp32" else dt
    s["x"] = normal(g, M, K).to(dt)
    w = (normal(g, *((K, W) if c["layout"] == "kn" else (W, K))) / math.sqrt(K)).to(dt)
    s["w"] = w if c["layout"] == "kn" else w.t()
    s["bias"] = (0.1 * normal(g, W)).to(dt) if c["bias"] else None
    s["residual"] = normal(g, M, N).to(out) if c["residual"] else None
    if c["way"] == "bwd":
        s["dy"] = normal(g, M, N).to(out)
        s["z"] = normal(g, M, W).to(dt) if c["act"] != "none" else None   # what the forward kept: the map before the activation


def block_inputs(s, c, g):
    dt = DTYPES[c["dtype"]]
    st = dt if c["stream"] == "same" else torch.float32
    R, C = c["rows"], c["cols"]
    sized = lambda: normal(g, R, C) * (0.5 + 2 * torch.rand(R, 1, generator=g, device="cuda")) + 0.3 * normal(g, R, 1)
    s["x"] = sized().to(st)
    s["b"] = sized().to(dt)
    for name, there in (("post", c["post"]), ("pre", c["pre"])):
        weight, bias = (1 + 0.2 * normal(g, C)).to(dt), (0.1 * normal(g, C)).to(dt)
        s[name] = (weight, bias if c["bias"] else None) if there else None
    s["gate"] = (0.5 + 0.3 * normal(g, *((C,) if c["gate"] == 1 else (c["gate"], C)))).to(dt) if c["gate"] else None
    if c["way"] == "bwd":   # what the forward kept: its output r and the statistics
        r, _, stats = plain_block_rows(s, c)
        s["r"], s["stats"] = r.to(st), stats
        s["dr"] = normal(g, R, C).to(st)
        s["dn"] = normal(g, R, C).to(dt) if c["pre"] else None
        del s["x"]


def experts_inputs(s, c, g):
    T, H, I, E, EL = c["T"], c["H"], c["I"], c["E"], c["EL"]
    s["x"] = normal(g, T, H).to(torch.bfloat16)
    top, idx = torch.sort(normal(g, T, E), dim=1, descending=True, stable=True)
    s["topk_idx"] = idx[:, :c["k"]].to(torch.int32).contiguous()
    s["topk_w"] = torch.softmax(top[:, :c["k"]], dim=1)
    s["w1"] = torch.stack([(normal(g, H, 2 * I) / math.sqrt(H)).to(torch.bfloat16) for _ in range(EL)])   # [gate | up]
    s["w2"] = torch.stack([(normal(g, I, H) / math.sqrt(I)).to(torch.bfloat16) for _ in range(EL)])
    if own:   # the shape, the packed weights and the workspace that a serving program keeps
        import token_dispatch_grouped_route_amd as moe

        s["shape"] = moe.make_shape(T, H, I, E, EL, c["k"])
        w1p, w2p = moe.alloc_packed(s["shape"])
        moe.pack_weights(s["shape"], s.pop("w1"), s.pop("w2"), w1p, w2p)
        s["packed"] = w1p, w2p
        s["ws"] = moe.few_alloc_workspace(s["shape"])


# ------------------------------------------------------------------------------------------------
# one pass
# ------------------------------------------------------------------------------------------------
def run(state):
    c = state["case"]
    if own:
        return own_run(state, c)
    return {"linear": plain_linear, "block": plain_block, "experts": plain_experts}[c["op"]](state, c)


def own_run(s, c):
    import token_dispatch_grouped_route_amd as moe

    if c["op"] == "linear":
        act = None if c["act"] == "none" else c["act"]
        if c["way"] == "fwd":
            out = torch.float32 if c["out"] == "fp32" else None
            y, _ = moe.linear_forward(s["x"], s["w"], s["bias"], act=act, residual=s["residual"], out_dtype=out)
            return {"y": y}
        dx, dw, db = moe.linear_backward(s["dy"], s["x"], s["w"], s["z"], act=act, bias=c["bias"])
        return {"dx": dx, "dw": dw, "db": db}
    if c["op"] == "block":
        how = {"kind": c["kind"], "post": s["post"], "gate": s["gate"], "pre": s["pre"], "x_scale": c["x_scale"], "scale": c["scale"]}
        if c["way"] == "fwd":
            r, n, stats = moe.block_norm_forward(s["x"], s["b"], eps=EPS, **how)
            return {"r": r, "n": n, **named(stats)}
        grads = moe.block_norm_backward(s["dr"], s["dn"], s["r"], s["b"], s["stats"], **how)
        return dict(zip(("dx", "db", "dgate", "dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias"), grads))
    return {"y": moe.forward_few(s["shape"], s["x"], s["topk_idx"], s["topk_w"], *s["packed"], s["ws"])}


def named(stats):
    return dict(zip(("post_mean", "post_rstd", "pre_mean", "pre_rstd"), stats))


def sigmoid(z):
    e = torch.exp(-z.abs())
    return torch.where(z >= 0, 1 / (1 + e), e / (1 + e))


def phi(z):
    """The normal distribution up to z."""
    return 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))


def plain_act(z, act):
    if act == "swiglu":
        gate, up = z.chunk(2, dim=1)
        return gate * sigmoid(gate) * up
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "gelu":
        return z * phi(z)
    return z * sigmoid(z) if act == "silu" else z


def plain_slope(z, act):
    if act == "relu":
        return torch.where(z > 0, 1.0, 0.0)
    if act == "gelu":
        return phi(z) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    s = sigmoid(z)
    return s * (1 + z * (1 - s))


def plain_linear(s, c):
    x, w, act, dt = s["x"].float(), s["w"].float(), c["act"], s["x"].dtype
    if c["way"] == "fwd":
        z = x @ w
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = plain_act(z, act)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(torch.float32 if c["out"] == "fp32" else dt)}
    dy = s["dy"].float()
    if act == "none":
        dz = dy
    elif act == "swiglu":
        gate, up = s["z"].float().chunk(2, dim=1)
        dz = torch.cat((dy * up * plain_slope(gate, "silu"), dy * gate * sigmoid(gate)), dim=1)
    else:
        dz = dy * plain_slope(s["z"].float(), act)
    return {"dx": (dz @ w.t()).to(dt), "dw": (x.t() @ dz).to(dt), "db": dz.sum(0).to(dt) if c["bias"] else None}


def gate_rows(gate, rows):
    """The gate of each row, in fp32 ([C] or [G, C], one for every rows / G rows)."""
    gate = gate.float()
    return gate if gate.dim() == 1 else gate.repeat_interleave(rows // gate.shape[0], 0)


def plain_norm(v, kind):
    mean = v.mean(1) if kind == "layer" else None
    v = v - mean[:, None] if mean is not None else v
    rstd = 1 / torch.sqrt((v * v).mean(1) + EPS)
    return v * rstd[:, None], mean, rstd


def affine(v, wb):
    v = v * wb[0].float()
    return v + wb[1].float() if wb[1] is not None else v


def plain_block_rows(s, c):
    """r and n in fp32 and the statistics."""
    p, stats = s["b"].float(), [None] * 4
    if s["post"] is not None:
        p, stats[0], stats[1] = plain_norm(p, c["kind"])
        p = affine(p, s["post"])
    if s["gate"] is not None:
        p = gate_rows(s["gate"], c["rows"]) * p
    r = c["x_scale"] * s["x"].float() + c["scale"] * p
    n = None
    if s["pre"] is not None:
        n, stats[2], stats[3] = plain_norm(r, c["kind"])
        n = affine(n, s["pre"])
    return r, n, tuple(stats)


def norm_grad(g, h, rstd, kind):
    d = g - h * (g * h).mean(1, keepdim=True)
    if kind == "layer":
        d = d - g.mean(1, keepdim=True)
    return d * rstd[:, None]


def plain_block(s, c):
    dt, kind = s["b"].dtype, c["kind"]
    if c["way"] == "fwd":
        r, n, stats = plain_block_rows(s, c)
        return {"r": r.to(s["x"].dtype), "n": n.to(dt) if n is not None else None, **named(stats)}
    wt = dt
    out = dict.fromkeys(("dx", "db", "dgate", "dpost_weight", "dpost_bias", "dpre_weight", "dpre_bias"))
    post_mean, post_rstd, pre_mean, pre_rstd = s["stats"]
    t = s["dr"].float()
    if s["pre"] is not None:
        weight, bias = s["pre"]
        h = s["r"].float()
        h = (h - pre_mean[:, None] if pre_mean is not None else h) * pre_rstd[:, None]
        dn = s["dn"].float()
        out["dpre_weight"] = (dn * h).sum(0).to(wt)
        out["dpre_bias"] = dn.sum(0).to(wt) if bias is not None else None
        t = t + norm_grad(dn * weight.float(), h, pre_rstd, kind)
    out["dx"] = (c["x_scale"] * t).to(s["dr"].dtype)
    h = s["b"].float()
    if s["post"] is not None:
        h = (h - post_mean[:, None] if post_mean is not None else h) * post_rstd[:, None]
    t = c["scale"] * t
    if s["gate"] is not None:
        part = t * (affine(h, s["post"]) if s["post"] is not None else h)
        dgate = part.view(max(1, s["gate"].shape[0] if s["gate"].dim() == 2 else 1), -1, c["cols"]).sum(1)
        out["dgate"] = dgate.view(s["gate"].shape).to(wt)
        t = t * gate_rows(s["gate"], c["rows"])
    if s["post"] is not None:
        weight, bias = s["post"]
        out["dpost_weight"] = (t * h).sum(0).to(wt)
        out["dpost_bias"] = t.sum(0).to(wt) if bias is not None else None
        t = norm_grad(t * weight.float(), h, post_rstd, kind)
    out["db"] = t.to(dt)
    return out


def plain_experts(s, c):
    """The routed experts, each on its token where there are fewer pairs than experts, else every local
    expert on every token; then the routed ones weighted and summed."""
    x, T, k, EL = s["x"].float(), c["T"], c["k"], c["EL"]
    local = s["topk_idx"] < EL   # this GPU owns the experts [0, EL)
    ids = s["topk_idx"].clamp(max=EL - 1).long()
    few = T * k < EL
    w1, w2 = s["w1"], s["w2"]
    if few:
        x, w1, w2 = x.repeat_interleave(k, 0)[:, None], w1[ids.flatten()], w2[ids.flatten()]   # x [T k, 1, H]
    h = torch.matmul(x, w1.float())   # [experts, rows, 2I]
    gate, up = h[..., :c["I"]], h[..., c["I"]:]
    o = torch.matmul(gate * sigmoid(gate) * up, w2.float())
    rows = o.view(T, k, -1) if few else o[ids, torch.arange(T, device=x.device)[:, None]]
    w = torch.where(local, s["topk_w"], 0.0)
    return {"y": (rows * w[..., None]).sum(1).to(s["x"].dtype)}


# ------------------------------------------------------------------------------------------------
# the definition in 64 bits
# ------------------------------------------------------------------------------------------------
def exact(case, seed):
    global own
    was, own = own, False   # the logical weights, whichever side is measured
    try:
        s = prepare(case, seed)
    finally:
        own = was
    return {"linear": exact_linear, "block": exact_block, "experts": exact_experts}[case["op"]](s, case)


def exact_linear(s, c):
    F = torch.nn.functional
    w, bias = s["w"].double(), s["bias"]
    acts = {"none": lambda z: z, "relu": F.relu, "gelu": F.gelu, "silu": F.silu, "swiglu": lambda z: F.silu(z[:, :c["N"]]) * z[:, c["N"]:]}
    act = acts[c["act"]]
    if c["way"] == "fwd":
        z = torch.mm(s["x"].double(), w)
        y = act(z + bias.double() if bias is not None else z)
        return {"y": y + s["residual"].double() if s["residual"] is not None else y}
    dz = s["dy"].double()
    if c["act"] != "none":
        z = s["z"].double().requires_grad_()
        dz, = torch.autograd.grad(act(z), z, dz)
    return {"dx": torch.mm(dz, w.t()), "dw": torch.mm(s["x"].double().t(), dz), "db": dz.sum(0) if c["bias"] else None}


def exact_block(s, c):
    layer, C, R, step = c["kind"] == "layer", c["cols"], c["rows"], 1024
    gate = s["gate"]
    per = R // gate.shape[0] if gate is not None and gate.dim() == 2 else R
    rows_of = lambda lo, hi: gate.double().view(-1, C)[torch.arange(lo, hi, device=gate.device) // per]
    wide = lambda wb: [t.double() if t is not None else 0.0 for t in wb]
    parts = []
    if c["way"] == "fwd":
        def norm(v):
            m = v.mean(1) if layer else torch.zeros(len(v), dtype=torch.float64, device=v.device)
            q = ((v - m[:, None]) ** 2).mean(1).add(EPS) ** -0.5
            return (v - m[:, None]) * q[:, None], m if layer else None, q

        for lo in range(0, R, step):
            hi = min(R, lo + step)
            p, o = s["b"][lo:hi].double(), {}
            if s["post"] is not None:
                p, o["post_mean"], o["post_rstd"] = norm(p)
                w, b = wide(s["post"])
                p = p * w + b
            if gate is not None:
                p = p * rows_of(lo, hi)
            o["r"] = c["x_scale"] * s["x"][lo:hi].double() + c["scale"] * p
            if s["pre"] is not None:
                n, o["pre_mean"], o["pre_rstd"] = norm(o["r"])
                w, b = wide(s["pre"])
                o["n"] = n * w + b
            parts.append(o)
        joined = lambda k: torch.cat([o[k] for o in parts]) if parts[0].get(k) is not None else None
        return {k: joined(k) for k in ("r", "n", "post_mean", "post_rstd", "pre_mean", "pre_rstd")}

    def standard(v, mean, rstd, lo, hi):
        v = v[lo:hi].double()
        return (v - mean[lo:hi].double()[:, None] if mean is not None else v) * rstd[lo:hi].double()[:, None]

    def back(v, z, rstd, lo, hi):   # the Jacobian of z: rstd (I - 1 1' / C [layer] - z z' / C)
        u = v - z * ((z * v).sum(1, keepdim=True) / C)
        return rstd[lo:hi].double()[:, None] * (u - v.sum(1, keepdim=True) / C if layer else u)

    post_mean, post_rstd, pre_mean, pre_rstd = s["stats"]
    total = {}
    add = lambda k, v: total.__setitem__(k, total.get(k, 0.0) + v)
    dgate = torch.zeros(R // per, C, dtype=torch.float64, device="cuda") if gate is not None else None
    dx, db = [], []
    for lo in range(0, R, step):
        hi = min(R, lo + step)
        t = s["dr"][lo:hi].double()
        if s["pre"] is not None:
            w, _ = wide(s["pre"])
            z, dn = standard(s["r"], pre_mean, pre_rstd, lo, hi), s["dn"][lo:hi].double()
            add("dpre_weight", (dn * z).sum(0))
            add("dpre_bias", dn.sum(0))
            t = t + back(dn * w, z, pre_rstd, lo, hi)
        dx.append(c["x_scale"] * t)
        p = z = s["b"][lo:hi].double()
        if s["post"] is not None:
            w, b = wide(s["post"])
            z = standard(s["b"], post_mean, post_rstd, lo, hi)
            p = z * w + b
        dp = c["scale"] * t
        if gate is not None:
            dgate.index_add_(0, torch.arange(lo, hi, device="cuda") // per, dp * p)
            dp = dp * rows_of(lo, hi)
        if s["post"] is not None:
            add("dpost_weight", (dp * z).sum(0))
            add("dpost_bias", dp.sum(0))
            dp = back(dp * w, z, post_rstd, lo, hi)
        db.append(dp)
    biased = lambda k: s[k] is not None and s[k][1] is not None
    return {"dx": torch.cat(dx), "db": torch.cat(db), "dgate": dgate.view(gate.shape) if gate is not None else None,
            "dpost_weight": total.get("dpost_weight"), "dpost_bias": total["dpost_bias"] if biased("post") else None,
            "dpre_weight": total.get("dpre_weight"), "dpre_bias": total["dpre_bias"] if biased("pre") else None}


def exact_experts(s, c):
    y = torch.zeros(c["T"], c["H"], dtype=torch.float64, device="cuda")
    for e in range(c["EL"]):
        token, slot = torch.nonzero(s["topk_idx"] == e, as_tuple=True)
        if not len(token):
            continue
        h = torch.mm(s["x"][token].double(), s["w1"][e].double())
        a = torch.nn.functional.silu(h[:, :c["I"]]) * h[:, c["I"]:]
        y.index_add_(0, token, torch.mm(a, s["w2"][e].double()) * s["topk_w"][token, slot].double()[:, None])
    return {"y": y}
