"""Cases that measure the router's operators and the dense products around the expert FFN:
the linear layer (gate projection, dense up and down projections) and its gradients, the
scored routing and its gradient, and the gradient of the combine.

`run` computes one pass in its plain form (elementary torch operations), or through
combine_overlap_b200.moe where `own` is set.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "silu", "gelu")
FLT_MAX = 3.4028234663852886e38
MOST_MKN = 4096 * 4096 * 14336        # the largest listed product


def listed():
    return [
        # the gate projection of one decoded token; 60 experts: rows of W that are not 16-byte multiples
        dict(name="linear_gate_decode", op="linear", M=1, K=2048, N=60, act="none", dtype="float32",
             bias=True, residual=False, pre=False),
        # the gate projection of a long prompt batch (the imbalanced layer's d and E)
        dict(name="linear_gate_prompt", op="linear", M=16384, K=4096, N=128, act="none", dtype="float32",
             bias=False, residual=False, pre=False),
        # a dense up projection with its activation, as large as the Mixtral-shaped expert
        dict(name="linear_up_silu", op="linear", M=4096, K=4096, N=14336, act="silu", dtype="bfloat16",
             bias=True, residual=False, pre=False),
        # a shared expert's down projection onto the routed output, ragged batch, kept for training
        dict(name="linear_down_residual", op="linear", M=1001, K=1408, N=2048, act="none", dtype="bfloat16",
             bias=False, residual=True, pre=False),
        # training the gate projection: fp32 gradients of the logits
        dict(name="linear_gate_backward", op="linear_backward", M=16384, K=4096, N=128, act="none",
             dtype="float32", dw="float32", bias=True),
        # training a dense up projection with its activation
        dict(name="linear_up_backward", op="linear_backward", M=8192, K=2048, N=1408, act="silu",
             dtype="bfloat16", dw="bfloat16", bias=True),
        # a decode step of a few sequences, softmax gates
        dict(name="route_decode", op="route", T=7, E=64, k=6, score="softmax", bias=False, groups=1,
             topk_groups=1, top2=False, renorm=True, scale=1.0, masked=False),
        # a long prompt batch: sigmoid scores, balance bias, group-limited choice
        dict(name="route_prompt_groups", op="route", T=16384, E=256, k=8, score="sigmoid", bias=True, groups=8,
             topk_groups=4, top2=True, renorm=True, scale=2.5, masked=True),
        # training the router of the fine-grained layer: softmax over all experts, gates not renormalised
        dict(name="route_backward_softmax", op="route_backward", T=8192, E=64, k=6, score="softmax",
             renorm=False, scale=1.0, masked=False),
        # training a sigmoid router over many experts, some of them masked
        dict(name="route_backward_sigmoid", op="route_backward", T=32768, E=256, k=8, score="sigmoid",
             renorm=True, scale=2.5, masked=True),
        # the gradient of the Mixtral-shaped layer's combine
        dict(name="combine_backward", op="combine_backward", T=4096, d=4096, k=2, dropped=False),
        # a ragged batch of the fine-grained layer, with dropped slots
        dict(name="combine_backward_ragged", op="combine_backward", T=513, d=2048, k=6, dropped=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size spread over its logarithm: a multiple of 64, of 8, or any."""
    n = _log(rng, lo, hi)
    step = rng.choice((1, 8, 64, 64))
    return min(hi, max(lo, n // step * step or n))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_backward", "route", "route_backward", "combine_backward"))
    if op in ("linear", "linear_backward"):
        gate = rng.random() < 0.5
        K = _size(rng, 128, 8192)
        N = rng.randint(4, 256) if gate else _size(rng, 64, 14336)
        most = MOST_MKN if op == "linear" else MOST_MKN // 2
        M = _log(rng, 1, max(1, min(16384, most // (K * N))))
        act = "none" if gate else rng.choice(ACTS)
        dtype = "float32" if gate else "bfloat16"
        if op == "linear":
            return dict(op=op, M=M, K=K, N=N, act=act, dtype=dtype, bias=rng.random() < 0.5,
                        residual=not gate and rng.random() < 0.5, pre=act != "none" and rng.random() < 0.5)
        exact_terms = act == "none"
        return dict(op=op, M=M, K=K, N=N, act=act, dtype=dtype,
                    dw="float32" if exact_terms else "bfloat16", bias=rng.random() < 0.5)
    if op == "combine_backward":
        d = 8 * _log(rng, 8, 1024)
        k = rng.randint(1, 8)
        T = _log(rng, 1, min(32768, 4096 * 4096 * 2 // (d * k)))
        return dict(op=op, T=T, d=d, k=k, dropped=rng.random() < 0.5)
    T, E = _log(rng, 1, 32768), rng.choice((8, 16, 32, 60, 64, 96, 128, 160, 256, rng.randint(2, 256)))
    score = rng.choice(("softmax", "sigmoid"))
    k = rng.randint(1, min(8, E))
    case = dict(op=op, T=T, E=E, k=k, score=score, renorm=rng.random() < 0.6,
                scale=rng.choice((1.0, 2.5)), masked=rng.random() < 0.5)
    if op == "route":
        groups = rng.choice([g for g in (1, 2, 4, 8) if E % g == 0])
        topk_groups = rng.randint(1, groups)
        while topk_groups * (E // groups) < k:
            topk_groups += 1
        case.update(bias=rng.random() < 0.5, groups=groups, topk_groups=topk_groups, top2=rng.random() < 0.5)
    return case


# ---------------------------------------------------------------- inputs ---
def _logits(g, T, E, masked):
    z = torch.randn(T, E, generator=g, device="cuda")
    z += 0.5 * torch.randn(E, generator=g, device="cuda")
    z[::5] = (z[::5] * 16).round() / 16            # rows with equal logits
    if masked:
        z[torch.rand(T, E, generator=g, device="cuda") < 0.03] = -math.inf
        if T > 4:
            z[T // 2] = -math.inf                  # a row that the mask leaves empty
    return z


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    randn = lambda *n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
    op, s = case["op"], dict(case=case)
    if op in ("linear", "linear_backward"):
        M, K, N = case["M"], case["K"], case["N"]
        dtype = getattr(torch, case["dtype"])
        s["x"] = randn(M, K).to(torch.bfloat16)
        s["W"] = (randn(K, N) * K ** -0.5).to(torch.bfloat16)
        if op == "linear":
            s["bias"] = 0.1 * randn(N) if case["bias"] else None
            s["residual"] = randn(M, N).to(dtype) if case["residual"] else None
        else:
            s["dout"] = (randn(M, N) * 0.01).to(dtype)
            s["pre"] = randn(M, N).to(torch.bfloat16) if case["act"] != "none" else None
    elif op == "combine_backward":
        T, d, k = case["T"], case["d"], case["k"]
        slot = torch.argsort(torch.randint(0, 64, (T * k,), generator=g, device="cuda"), stable=True)
        row_of = torch.empty(T * k, dtype=torch.int32, device="cuda")
        row_of[slot] = torch.arange(T * k, dtype=torch.int32, device="cuda")
        if case["dropped"]:
            row_of[torch.rand(T * k, generator=g, device="cuda") < 0.05] = -1
        s.update(row_of=row_of, dout=(randn(T, d) * 0.1).to(torch.bfloat16), y=randn(T * k, d).to(torch.bfloat16),
                 gate=torch.softmax(randn(T, k), 1), dy=torch.zeros(T * k, d, dtype=torch.bfloat16, device="cuda"))
    else:
        T, E, k = case["T"], case["E"], case["k"]
        s["logits"] = _logits(g, T, E, case["masked"])
        if op == "route":
            s["bias"] = 0.1 * randn(E) if case["bias"] else None
        else:
            s["idx"] = torch.argsort(s["logits"], dim=1, descending=True, stable=True)[:, :k].to(torch.int32).contiguous()
            s["dgate"] = randn(T, k)
    return s


# ------------------------------------------------------------ plain forms ---
def _act(name, v):
    if name == "relu":
        return v.clamp(min=0)
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * 0.5 ** 0.5))
    return v


def _dact(name, v):
    if name == "relu":
        return (v > 0).to(v.dtype)
    if name == "silu":
        p = 1 / (1 + torch.exp(-v))
        return p * (1 + v * (1 - p))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(v * 0.5 ** 0.5)) + v * torch.exp(-0.5 * v * v) * (2 * math.pi) ** -0.5
    return torch.ones_like(v)


def _plain_linear(s, case):
    v = s["x"].float() @ s["W"].float()
    if s["bias"] is not None:
        v = v + s["bias"]
    out = _act(case["act"], v)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    res = dict(out=out.to(getattr(torch, case["dtype"])))
    if case["pre"]:
        res["pre"] = v.to(torch.bfloat16)
    return res


def _plain_linear_backward(s, case):
    dpre = s["dout"].float()
    if s["pre"] is not None:
        dpre = dpre * _dact(case["act"], s["pre"].float())
    res = dict(dx=(dpre @ s["W"].float().t()).to(torch.bfloat16),
               dW=(s["x"].float().t() @ dpre).to(getattr(torch, case["dw"])))
    if case["bias"]:
        res["dbias"] = dpre.sum(0)
    return res


def _scores(logits, kind):
    """Scores in 64 bits and which experts are not masked."""
    live = ~(torch.isnan(logits) | (logits == -math.inf))
    z = torch.where(live, logits.double(), 0.0).clamp(max=FLT_MAX)
    if kind == "sigmoid":
        p = 1 / (1 + torch.exp(-z))
        return torch.where(live, p, 0.0), live, z
    top = torch.where(live, z, -math.inf).amax(1, keepdim=True)
    e = torch.where(live, torch.exp(z - torch.where(top == -math.inf, 0.0, top)), 0.0)
    total = e.sum(1, keepdim=True)
    return e / torch.where(total > 0, total, 1.0), live, z


def _plain_route(s, case):
    # in 64 bits: the choice between scores that are next to each other
    T, E, k, G = case["T"], case["E"], case["k"], case["groups"]
    p, live, z = _scores(s["logits"], case["score"])
    biased = p if s["bias"] is None else p + s["bias"].double()
    key = torch.where(live, z if s["bias"] is None else biased, -1e300)
    if G > 1:
        of = torch.where(live, biased if case["top2"] else key, -math.inf).view(T, G, E // G)
        best = torch.sort(of, dim=2, descending=True).values[:, :, : 2 if case["top2"] else 1]
        best = torch.where(best[:, :, 0] == -math.inf, -math.inf, torch.where(best == -math.inf, 0.0, best).sum(2))
        chosen = torch.sort(best, dim=1, descending=True, stable=True).indices[:, : case["topk_groups"]]
        inside = torch.zeros(T, G, dtype=torch.bool, device=p.device).scatter_(1, chosen, True)
        key = torch.where(inside.repeat_interleave(E // G, 1), key, -math.inf)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    gate = torch.gather(p, 1, idx)
    if case["renorm"]:
        total = gate.sum(1, keepdim=True)
        gate = gate / torch.where(total > 0, total, 1.0)
    return dict(idx=idx.to(torch.int32), gate=(gate * case["scale"]).float())


def _plain_route_backward(s, case):
    z, idx, dg = s["logits"], s["idx"].long(), s["dgate"]
    live = ~(torch.isnan(z) | (z == -math.inf))
    z = torch.where(live, z, 0.0)
    if case["score"] == "sigmoid":
        p = torch.where(live, 1 / (1 + torch.exp(-z)), 0.0)
    else:
        top = torch.where(live, z, -math.inf).amax(1, keepdim=True)
        e = torch.where(live, torch.exp(z - torch.where(top == -math.inf, 0.0, top)), 0.0)
        total = e.sum(1, keepdim=True)
        p = e / torch.where(total > 0, total, 1.0)
    dp = case["scale"] * dg
    if case["renorm"]:
        w = torch.gather(p, 1, idx)
        total = w.sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        dp = (dp - (dp * w / total).sum(1, keepdim=True)) / total
    dp = torch.zeros_like(z).scatter_(1, idx, dp)
    if case["score"] == "sigmoid":
        return dict(dlogits=dp * p * (1 - p))
    return dict(dlogits=p * (dp - (p * dp).sum(1, keepdim=True)))


def _plain_combine_backward(s, case):
    T, d, k = case["T"], case["d"], case["k"]
    kept = (s["row_of"] >= 0).view(T, k)
    rows = s["row_of"].long()
    dout = s["dout"].float()
    y = s["y"].float()[rows.clamp(min=0)].view(T, k, d)
    dgate = torch.where(kept, (dout[:, None] * y).sum(2), 0.0)
    dy = (s["gate"][:, :, None] * dout[:, None]).view(T * k, d).to(torch.bfloat16)
    s["dy"][rows[kept.view(-1)]] = dy[kept.view(-1)]
    return dict(dy=s["dy"], dgate=dgate)


PLAIN = dict(linear=_plain_linear, linear_backward=_plain_linear_backward, route=_plain_route,
             route_backward=_plain_route_backward, combine_backward=_plain_combine_backward)


# --------------------------------------------------- the framework's calls ---
def _own(s, case):
    from combine_overlap_b200 import moe
    op = case["op"]
    acts = dict(none=moe.ACT_NONE, relu=moe.ACT_RELU, silu=moe.ACT_SILU, gelu=moe.ACT_GELU)
    if op == "linear":
        r = moe.linear(s["x"], s["W"], bias=s["bias"], residual=s["residual"], act=acts[case["act"]],
                       out_dtype=getattr(torch, case["dtype"]), pre=case["pre"])
        return dict(zip(("out", "pre"), r)) if case["pre"] else dict(out=r)
    if op == "linear_backward":
        dx, dW, dbias = moe.linear_backward(s["dout"], s["x"], s["W"], pre=s["pre"], act=acts[case["act"]],
                                            dW_dtype=getattr(torch, case["dw"]), want_dbias=case["bias"])
        return dict(dx=dx, dW=dW, dbias=dbias) if case["bias"] else dict(dx=dx, dW=dW)
    if op == "combine_backward":
        dy, dgate = moe.combine_backward(s["dout"], s["y"], s["row_of"], s["gate"], dy=s["dy"])
        return dict(dy=dy, dgate=dgate)
    score = moe.SCORE_SIGMOID if case["score"] == "sigmoid" else moe.SCORE_SOFTMAX
    if op == "route":
        idx, gate = moe.route_scored(s["logits"], case["k"], score=score, bias=s["bias"], n_groups=case["groups"],
                                     topk_groups=case["topk_groups"],
                                     group_score=moe.GROUP_TOP2 if case["top2"] else moe.GROUP_MAX,
                                     renorm=case["renorm"], scale=case["scale"])
        return dict(idx=idx, gate=gate)
    return dict(dlogits=moe.route_scored_backward(s["dgate"], s["logits"], s["idx"], score=score,
                                                  renorm=case["renorm"], scale=case["scale"]))


def run(state):
    case = state["case"]
    return _own(state, case) if own else PLAIN[case["op"]](state, case)


# ------------------------------------------------------------------- work ---
def work(case):
    op = case["op"]
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        size = 4 if case["dtype"] == "float32" else 2
        outs = M * N * size * (2 if case["residual"] else 1) + (2 * M * N if case["pre"] else 0)
        return dict(bytes=2 * (M * K + K * N) + outs + (4 * N if case["bias"] else 0), flops=2 * M * N * K)
    if op == "linear_backward":
        M, K, N = case["M"], case["K"], case["N"]
        size = 4 if case["dtype"] == "float32" else 2
        ins = 2 * (M * K + K * N) + M * N * size + (2 * M * N if case["act"] != "none" else 0)
        outs = 2 * M * K + K * N * (4 if case["dw"] == "float32" else 2) + (4 * N if case["bias"] else 0)
        return dict(bytes=ins + outs, flops=4 * M * N * K)
    if op == "combine_backward":
        T, d, k = case["T"], case["d"], case["k"]
        return dict(bytes=2 * T * d * (1 + 2 * k) + 12 * T * k, flops=3 * T * k * d)
    T, E, k = case["T"], case["E"], case["k"]
    if op == "route":
        return dict(bytes=4 * T * E + 8 * T * k, flops=T * E * (4 + k))
    # only the softmax over all experts needs every logit; else the k chosen ones
    reads = T * E if case["score"] == "softmax" and not case["renorm"] else T * k
    return dict(bytes=4 * (reads + T * E) + 8 * T * k, flops=4 * T * E)


# ------------------------------------------------- the definitions, 64 bits ---
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        u = torch.einsum("mk,kn->mn", s["x"].double(), s["W"].double())
        if case["bias"]:
            u += s["bias"].double()
        h = {"none": lambda: u, "relu": lambda: torch.relu(u), "silu": lambda: u * torch.sigmoid(u),
             "gelu": lambda: u * torch.special.ndtr(u)}[case["act"]]()
        out = h + s["residual"].double() if case["residual"] else h
        return dict(out=out, pre=u) if case["pre"] else dict(out=out)
    if op == "linear_backward":
        du = s["dout"].double()
        if case["act"] != "none":
            with torch.enable_grad():
                u = s["pre"].double().requires_grad_(True)
                h = {"relu": torch.relu, "silu": lambda t: t * torch.sigmoid(t),
                     "gelu": lambda t: t * torch.special.ndtr(t)}[case["act"]](u)
                du, = torch.autograd.grad(h, u, du)
        res = dict(dx=torch.einsum("mn,kn->mk", du, s["W"].double()), dW=torch.einsum("mk,mn->kn", s["x"].double(), du))
        if case["bias"]:
            res["dbias"] = torch.einsum("mn->n", du)
        return res
    if op == "combine_backward":
        T, d, k = case["T"], case["d"], case["k"]
        dy, dgate = torch.zeros(T * k, d, dtype=torch.float64, device="cuda"), torch.zeros(T, k, dtype=torch.float64, device="cuda")
        for j in range(k):
            r = s["row_of"].view(T, k)[:, j].long()
            t = torch.nonzero(r >= 0)[:, 0]
            dgate[t, j] = torch.einsum("td,td->t", s["dout"][t].double(), s["y"][r[t]].double())
            dy[r[t]] = s["gate"][t, j, None].double() * s["dout"][t].double()
        return dict(dy=dy, dgate=dgate)
    if op == "route":
        return dict(idx=None, gate=_exact_gates(s["logits"], _plain_route(s, case)["idx"].long(), case))
    with torch.enable_grad():
        z = torch.where(torch.isinf(s["logits"]), -1e4, s["logits"].double()).requires_grad_(True)
        gates = _exact_gates(z, s["idx"].long(), case)
        some = ~torch.isinf(s["logits"]).all(1)
        dz, = torch.autograd.grad((gates * s["dgate"].double() * some[:, None]).sum(), z)
    return dict(dlogits=torch.where(some[:, None] & ~torch.isinf(s["logits"]), dz, 0.0))


def _exact_gates(logits, idx, case):
    """Gates of the chosen experts, from the definition; a row of masked experts only has gates of 0."""
    z = logits.double()
    empty = torch.isinf(z).all(1, keepdim=True)
    z = torch.where(empty, 0.0, z)
    picked = torch.sigmoid(z).gather(1, idx) if case["score"] == "sigmoid" else torch.exp(
        z.gather(1, idx) - torch.logsumexp(z, 1, keepdim=True))
    if case["renorm"]:
        picked = picked / picked.sum(1, keepdim=True).clamp(min=1e-300)
    return torch.where(empty, 0.0, case["scale"] * picked)
