"""The layer operators' measured cases: linear, route, expert_linear, combine.

Each case is one call, or one call's gradients, as a model's program makes
it.  With ``own`` false, ``run`` computes it from elementary torch
operations in 32 bits (64 where a selection is decided); with ``own`` true
it calls the framework.  ``exact`` computes the same from the definition in
64 bits.

Symbols: m tokens, k inputs and n outputs of a product, E experts, K of them
per token.  ``w`` is the order of a weight (k x n): "kn" has its rows
contiguous, "nk" its columns (a weight kept as n x k and passed transposed).
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # one token of a served model: the whole weight is read for one row
        dict(name="linear_token_bf16", op="linear", dtype="bf16", m=1, n=4096, k=4096, w="nk",
             act="none", bias=False, residual=True, z=False),
        # a prompt, or a training step's forward pass: keeps the
        # pre-activations for the backward pass
        dict(name="linear_prompt_bf16", op="linear", dtype="bf16", m=8192, n=8192, k=4096, w="nk",
             act="gelu_tanh", bias=True, residual=False, z=True),
        # odd sizes in fp32 (the benchmark's ragged matrix product)
        dict(name="linear_ragged_f32", op="linear", dtype="f32", m=4097, n=3001, k=1023, w="kn",
             act="relu", bias=True, residual=True, z=False),
        # the gradients of a training step's layer
        dict(name="linear_backward_bf16", op="linear_backward", dtype="bf16", m=8192, n=4096,
             k=4096, w="nk", act="silu", bias=True),
        # the router of a served model's decode step: latency alone
        dict(name="route_decode", op="route", dtype="f32", m=4, experts=64, top=4, score="softmax",
             groups=1, top_groups=1, renorm=False, bias=False, scale=1.0, padded=0),
        # a long prompt over many experts in groups, with a balance bias and
        # padding rows that are not routed
        dict(name="route_prompt", op="route", dtype="f32", m=16384, experts=192, top=6,
             score="sigmoid", groups=6, top_groups=3, renorm=True, bias=True, scale=2.0,
             padded=77),
        # the router's gradient, an odd number of rows
        dict(name="route_backward_bf16", op="route_backward", dtype="bf16", m=8191, experts=128,
             top=8, score="softmax", renorm=False, scale=1.0, padded=0),
        # decode: a few rows for most experts, every weight read once
        dict(name="experts_decode_bf16", op="experts", dtype="bf16", m=16, experts=64, top=4, n=2048,
             k=1024, w="nk", act="silu", bias=False, gather=True, z=False),
        # a prompt over few large experts
        dict(name="experts_prompt_f16", op="experts", dtype="f16", m=8191, experts=8, top=2, n=4096,
             k=2048, w="kn", act="gelu", bias=True, gather=True, z=True),
        # the experts' gradients in a training step
        dict(name="experts_backward_bf16", op="experts_backward", dtype="bf16", m=4096, experts=16,
             top=4, n=1024, k=2048, w="nk", act="silu", bias=True, gather=True),
        # the experts' rows back to their tokens, onto the residual stream
        dict(name="combine_prompt_bf16", op="combine", dtype="bf16", m=8192, experts=64, top=8,
             n=2048, residual=True, padded=13),
        # its gradients
        dict(name="combine_backward_bf16", op="combine_backward", dtype="bf16", m=4095, experts=64,
             top=6, n=2048, padded=0),
    ]


def _log(rng, lo, hi):
    """A size of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _feature(rng, lo, hi):
    """A feature count: mostly whole 16-byte rows, sometimes odd."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.3 else max(8, v // 8 * 8)


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_backward", "route", "route_backward", "experts",
                     "experts_backward", "combine", "combine_backward"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    c = dict(op=op, dtype=dtype)
    if op in ("linear", "linear_backward"):
        while True:
            m, n, k = _log(rng, 1, 8192), _feature(rng, 16, 8192), _feature(rng, 16, 8192)
            if m * n * k <= 8192 * 4096 * 4096 // (8 if dtype == "f32" else 1):
                break
        c.update(m=m, n=n, k=k, w=rng.choice(("kn", "nk")), act=rng.choice(ACTS),
                 bias=rng.random() < 0.5)
        if op == "linear":
            c.update(residual=rng.random() < 0.5, z=rng.random() < 0.5)
    elif op in ("route", "route_backward"):
        groups = rng.choice((1, 1, 4, 8))
        experts = groups * rng.randint(max(1, 8 // groups), 256 // groups)
        top_groups = rng.randint(1, groups)
        top = rng.randint(1, min(8, experts // groups * top_groups))
        m = _log(rng, 1, 16384)
        c.update(m=m, experts=experts, top=top, score=rng.choice(("softmax", "sigmoid")),
                 renorm=rng.random() < 0.5, scale=rng.choice((1.0, 2.0)),
                 padded=rng.randint(0, m // 8))
        if op == "route":
            c.update(groups=groups, top_groups=top_groups, bias=rng.random() < 0.5)
    else:
        experts = rng.choice((8, 16, 60, 64))
        top = rng.randint(1, 8)
        if op in ("experts", "experts_backward"):
            while True:
                m, n, k = _log(rng, 1, 8192), _feature(rng, 32, 4096), _feature(rng, 32, 4096)
                if m * top * n * k <= 8192 * 2 * 4096 * 2048 // (8 if dtype == "f32" else 1) and \
                        experts * n * k <= 1 << 28:
                    break
            c.update(m=m, experts=experts, top=top, n=n, k=k, w=rng.choice(("kn", "nk")),
                     act=rng.choice(ACTS), bias=rng.random() < 0.5, gather=rng.random() < 0.7)
            if op == "experts":
                c.update(z=rng.random() < 0.5)
        else:
            m = _log(rng, 1, 8192)
            c.update(m=m, experts=experts, top=top, n=_feature(rng, 32, 4096),
                     padded=rng.randint(0, m // 8))
            if op == "combine":
                c.update(residual=rng.random() < 0.5)
    return c


# ---- inputs ----------------------------------------------------------------

def _weight(g, lead, k, n, order, dtype):
    """A weight (..., k, n) of the scale 1/sqrt(k), in the order asked for."""
    if order == "kn":
        w = torch.randn(*lead, k, n, generator=g, device="cuda")
        return w.mul_(k ** -0.5).to(dtype)
    w = torch.randn(*lead, n, k, generator=g, device="cuda")
    return w.mul_(k ** -0.5).to(dtype).transpose(-1, -2)


def _choices(g, case):
    """Random distinct experts per token, most wanted first (m x K; -1 in
    padding rows)."""
    m, E, K = case["m"], case["experts"], case["top"]
    e = torch.rand(m, E, generator=g, device="cuda").argsort(1)[:, :K].to(torch.int32)
    if case.get("padded"):
        e[m - case["padded"]:] = -1
    return e


def _plan(e, E):
    """Rows sorted by expert, then token: offsets, the rows' tokens (-1 behind
    the last one) and each (token, choice)'s row (-1: none)."""
    m, K = e.shape
    hit = e.long()[:, :, None] == torch.arange(E, device="cuda")     # m x K x E
    per = hit.sum(1)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = per.sum(0).cumsum(0)
    row = offsets[:-1] + per.cumsum(0) - per                         # m x E
    slots = row.gather(1, e.long().clamp(min=0))
    slots = torch.where(e >= 0, slots, torch.full_like(slots, -1))
    tokens = torch.full((m * K + 1,), -1, dtype=torch.int64, device="cuda")
    t = torch.arange(m, device="cuda")[:, None].expand(m, K)
    tokens[torch.where(slots >= 0, slots, torch.full_like(slots, m * K))] = t
    tokens = tokens[:m * K]
    tokens[offsets[E]:] = -1
    return offsets.to(torch.int32), tokens.to(torch.int32), slots.to(torch.int32)


def _empty(*shape, dtype):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def _zeros(*shape, dtype):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def _like(w):
    """A zeroed tensor of w's shape and order."""
    return torch.zeros_like(w, memory_format=torch.preserve_format)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = TYPES[case["dtype"]]
    op, m = case["op"], case["m"]
    s = dict(case=case)

    def rnd(*shape, dtype=T):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    if own:
        import precision_gemm_02_amd as pg
    if op in ("linear", "linear_backward"):
        n, k = case["n"], case["k"]
        s.update(X=rnd(m, k), W=_weight(g, (), k, n, case["w"], T))
        if op == "linear":
            s.update(bias=rnd(n) if case["bias"] else None,
                     R=rnd(m, n) if case["residual"] else None,
                     Y=_empty(m, n, dtype=T), Z=_empty(m, n, dtype=T) if case["z"] else None)
            if own:
                s["ws"] = _empty(max(16, pg.linear_workspace(m, n, k, T)), dtype=torch.uint8)
        else:
            s.update(dY=rnd(m, n), Z=rnd(m, n) if case["act"] != "none" else None,
                     dX=_empty(m, k, dtype=T), dW=_like(s["W"]),
                     db=_empty(n, dtype=T) if case["bias"] else None)
            if own:
                size = pg.linear_backward_workspace(m, n, k, T, act=case["act"])
                s["ws"] = _empty(max(16, size), dtype=torch.uint8)
    elif op in ("route", "route_backward"):
        E, K = case["experts"], case["top"]
        logits = (torch.randn(m, E, generator=g, device="cuda") * 1.5).to(T)
        if case["padded"]:
            logits[m - case["padded"]:] = -math.inf
        s.update(logits=logits)
        if op == "route":
            s.update(bias=torch.randn(E, generator=g, device="cuda") * 0.1 if case["bias"] else None,
                     weights=_empty(m, K, dtype=torch.float32), experts=_empty(m, K, dtype=torch.int32),
                     offsets=_empty(E + 1, dtype=torch.int32), slots=_empty(m, K, dtype=torch.int32),
                     tokens=torch.full((m * K,), -1, dtype=torch.int32, device="cuda"))
            if own:
                s["ws"] = _empty(max(16, pg.route_workspace(m, E, K)), dtype=torch.uint8)
        else:
            s.update(experts=_choices(g, case), dweights=rnd(m, K, dtype=torch.float32),
                     dlogits=_empty(m, E, dtype=T))
    else:
        E, K, n = case["experts"], case["top"], case["n"]
        if K > E:
            raise ValueError("more choices than experts")
        offsets, tokens, slots = _plan(_choices(g, case), E)
        s.update(offsets=offsets, tokens=tokens, slots=slots)
        R = m * K
        if op in ("experts", "experts_backward"):
            k = case["k"]
            # the plain form's loop over the experts reads the counts on the host
            s.update(bounds=offsets.tolist(), X=rnd(m if case["gather"] else R, k),
                     W=_weight(g, (E,), k, n, case["w"], T))
            if op == "experts":
                s.update(bias=rnd(E, n) if case["bias"] else None, Y=_zeros(R, n, dtype=T),
                         Z=_zeros(R, n, dtype=T) if case["z"] else None)
            else:
                s.update(dY=rnd(R, n), Z=rnd(R, n) if case["act"] != "none" else None,
                         dX=_zeros(R, k, dtype=T), dW=_like(s["W"]),
                         db=_empty(E, n, dtype=T) if case["bias"] else None)
                if own:
                    size = pg.expert_linear_backward_workspace(R, n, k, E, T, act=case["act"])
                    s["ws"] = _empty(max(16, size), dtype=torch.uint8)
        else:
            w = torch.rand(m, K, generator=g, device="cuda") / K
            s.update(Y=rnd(R, n), weights=w)
            if op == "combine":
                s.update(R=rnd(m, n) if case["residual"] else None, out=_empty(m, n, dtype=T))
            else:
                s.update(dout=rnd(m, n), dY=_zeros(R, n, dtype=T),
                         dweights=_empty(m, K, dtype=torch.float32))
    return s


# ---- the framework's operators ----------------------------------------------

def _run_own(s):
    import precision_gemm_02_amd as pg
    c = s["case"]
    op = c["op"]
    if op == "linear":
        pg.linear(s["X"], s["W"], s["Y"], bias=s["bias"], act=c["act"], residual=s["R"], Z=s["Z"],
                  ws=s["ws"])
        return {"Y": s["Y"], "Z": s["Z"]} if c["z"] else {"Y": s["Y"]}
    if op == "linear_backward":
        pg.linear_backward(s["dY"], s["X"], s["W"], Z=s["Z"], act=c["act"], dX=s["dX"], dW=s["dW"],
                           dbias=s["db"], ws=s["ws"])
        out = {"dX": s["dX"], "dW": s["dW"]}
        return dict(out, db=s["db"]) if c["bias"] else out
    if op == "route":
        pg.route(s["logits"], s["weights"], s["experts"], s["offsets"], s["tokens"], s["slots"],
                 bias=s["bias"], score=c["score"], groups=c["groups"], top_groups=c["top_groups"],
                 renorm=c["renorm"], scale=c["scale"], ws=s["ws"])
        return {x: s[x] for x in ("weights", "experts", "offsets", "tokens", "slots")}
    if op == "route_backward":
        pg.route_backward(s["dweights"], s["logits"], s["experts"], s["dlogits"], score=c["score"],
                          renorm=c["renorm"], scale=c["scale"])
        return {"dlogits": s["dlogits"]}
    if op == "experts":
        pg.expert_linear(s["X"], s["W"], s["Y"], s["offsets"],
                         tokens=s["tokens"] if c["gather"] else None, bias=s["bias"], act=c["act"],
                         Z=s["Z"])
        return {"Y": s["Y"], "Z": s["Z"]} if c["z"] else {"Y": s["Y"]}
    if op == "experts_backward":
        pg.expert_linear_backward(s["dY"], s["X"], s["W"], s["offsets"],
                                  tokens=s["tokens"] if c["gather"] else None, Z=s["Z"],
                                  act=c["act"], dX=s["dX"], dW=s["dW"], dbias=s["db"], ws=s["ws"])
        out = {"dX": s["dX"], "dW": s["dW"]}
        return dict(out, db=s["db"]) if c["bias"] else out
    if op == "combine":
        pg.combine(s["Y"], s["slots"], s["out"], weights=s["weights"], residual=s["R"])
        return {"out": s["out"]}
    pg.combine_backward(s["dout"], s["Y"], s["slots"], s["weights"], dY=s["dY"],
                        dweights=s["dweights"])
    return {"dY": s["dY"], "dweights": s["dweights"]}


# ---- the plain form -----------------------------------------------------------

def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + \
            z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        q = 1 / (1 + torch.exp(-z))
        return q * (1 + z * (1 - q))
    return torch.ones_like(z)


def _plain_route(s):
    c = s["case"]
    m, E, K = c["m"], c["experts"], c["top"]
    logits = s["logits"].double()
    masked = logits == -math.inf
    top = torch.where(masked, torch.zeros_like(logits), logits).amax(1, keepdim=True)
    if c["score"] == "softmax":
        e = torch.exp(torch.where(masked, torch.full_like(logits, -math.inf), logits - top))
        score = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        score = 1 / (1 + torch.exp(-logits))
    if c["groups"] == 1 and not c["bias"]:
        key = logits
    else:
        key = score + s["bias"].double() if c["bias"] else score
    none = torch.full_like(key, -math.inf)
    key = torch.where(masked, none, key)
    index = torch.arange(E, device="cuda")
    if c["groups"] > 1:
        grouped = key.view(m, c["groups"], -1)
        g1 = grouped.amax(2)
        first = grouped.argmax(2, keepdim=True)
        g2 = grouped.scatter(2, first, -math.inf).amax(2)
        both = g1 + torch.where(g2 == -math.inf, torch.zeros_like(g2), g2)
        keep = torch.zeros(m, c["groups"], dtype=torch.bool, device="cuda")
        for _ in range(c["top_groups"]):
            best = both.amax(1, keepdim=True)
            at = (both == best).to(torch.int8).argmax(1, keepdim=True)
            keep.scatter_(1, at, True)
            both = both.scatter(1, at, -math.inf)
        key = torch.where(keep[:, :, None].expand_as(grouped).reshape(m, E), key, none)
    chosen, picked = [], []
    for _ in range(K):
        best = key.amax(1)
        at = torch.where(key == best[:, None], index, E).amin(1)
        live = best > -math.inf
        chosen.append(torch.where(live, at, torch.full_like(at, -1)))
        picked.append(torch.where(live, score.gather(1, at[:, None])[:, 0], torch.zeros_like(best)))
        key = key.scatter(1, at[:, None], -math.inf)
    experts, w = torch.stack(chosen, 1), torch.stack(picked, 1)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, torch.zeros_like(w))
    experts = experts.to(torch.int32)
    offsets, tokens, slots = _plan(experts, E)
    return {"weights": (w * c["scale"]).float(), "experts": experts, "offsets": offsets,
            "tokens": tokens, "slots": slots}


def _plain_route_backward(s):
    c = s["case"]
    E = c["experts"]
    l, dw, e = s["logits"].float(), s["dweights"], s["experts"].long()
    live = e >= 0
    at = e.clamp(min=0)
    dw = torch.where(live, dw, torch.zeros_like(dw)) * c["scale"]
    if c["score"] == "softmax":
        top = l.amax(1, keepdim=True)
        x = torch.exp(l - torch.where(top == -math.inf, torch.zeros_like(top), top))
        score = x / x.sum(1, keepdim=True).clamp(min=1e-30)
    else:
        score = 1 / (1 + torch.exp(-l))
    p = torch.where(live, score.gather(1, at), torch.zeros_like(dw))
    if c["renorm"]:
        q = p / p.sum(1, keepdim=True).clamp(min=1e-30)
        inner = dw - (q * dw).sum(1, keepdim=True)       # d/d(p_j) times the sum
        if c["score"] == "softmax":
            d = q * inner
        else:
            d = q * inner * (1 - p)
        return {"dlogits": torch.zeros_like(l).scatter_add_(1, at, d).to(s["logits"].dtype)}
    if c["score"] == "softmax":
        d = torch.zeros_like(l).scatter_add_(1, at, p * dw)
        d = d - score * (p * dw).sum(1, keepdim=True)
    else:
        d = torch.zeros_like(l).scatter_add_(1, at, dw * p * (1 - p))
    return {"dlogits": d.to(s["logits"].dtype)}


def _plain_experts(s):
    c = s["case"]
    R, n = s["Y"].shape
    T = TYPES[c["dtype"]]
    x = s["X"].float()
    if c["gather"]:
        x = x[s["tokens"].clamp(min=0).long()]
    z = torch.zeros(R, n, device="cuda")
    b = s["bounds"]
    for e in range(c["experts"]):
        if b[e + 1] > b[e]:
            r = slice(b[e], b[e + 1])
            z[r] = x[r] @ s["W"][e].float()
            if c["bias"]:
                z[r] += s["bias"][e].float()
    out = {"Y": _act(z, c["act"]).to(T)}
    return dict(out, Z=z.to(T)) if c["z"] else out


def _plain_experts_backward(s):
    c = s["case"]
    R, n = s["dY"].shape
    E, k, T = c["experts"], c["k"], TYPES[c["dtype"]]
    b = s["bounds"]
    x = s["X"].float()
    if c["gather"]:
        x = x[s["tokens"].clamp(min=0).long()]
    dz = s["dY"].float()
    if c["act"] != "none":
        dz = dz * _act_grad(s["Z"].float(), c["act"])
    dx = torch.zeros(R, k, device="cuda")
    dw = torch.zeros(E, k, n, device="cuda")
    db = torch.zeros(E, n, device="cuda")
    for e in range(E):
        if b[e + 1] > b[e]:
            r = slice(b[e], b[e + 1])
            dx[r] = dz[r] @ s["W"][e].float().t()
            dw[e] = x[r].t() @ dz[r]
            db[e] = dz[r].sum(0)
    out = {"dX": dx.to(T), "dW": dw.to(T)}
    return dict(out, db=db.to(T)) if c["bias"] else out


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    op, T = c["op"], TYPES[c["dtype"]]
    if op == "linear":
        z = s["X"].float() @ s["W"].float()
        if c["bias"]:
            z = z + s["bias"].float()
        y = _act(z, c["act"])
        if c["residual"]:
            y = y + s["R"].float()
        return {"Y": y.to(T), "Z": z.to(T)} if c["z"] else {"Y": y.to(T)}
    if op == "linear_backward":
        dz = s["dY"].float()
        if c["act"] != "none":
            dz = dz * _act_grad(s["Z"].float(), c["act"])
        out = {"dX": (dz @ s["W"].float().t()).to(T), "dW": (s["X"].float().t() @ dz).to(T)}
        return dict(out, db=dz.sum(0).to(T)) if c["bias"] else out
    if op == "route":
        return _plain_route(s)
    if op == "route_backward":
        return _plain_route_backward(s)
    if op == "experts":
        return _plain_experts(s)
    if op == "experts_backward":
        return _plain_experts_backward(s)
    slots = s["slots"].long()
    live = (slots >= 0)[:, :, None]
    rows = s["Y"].float()[slots.clamp(min=0)]                       # m x K x n
    if op == "combine":
        y = torch.where(live, rows * s["weights"][:, :, None], torch.zeros_like(rows)).sum(1)
        if c["residual"]:
            y = y + s["R"].float()
        return {"out": y.to(T)}
    d = s["dout"].float()[:, None, :]
    dweights = torch.where(live, d * rows, torch.zeros_like(rows)).sum(2)
    dY = torch.zeros(s["Y"].shape[0] + 1, c["n"], dtype=T, device="cuda")
    dY[torch.where(slots >= 0, slots, torch.full_like(slots, s["Y"].shape[0]))] = \
        (d * s["weights"][:, :, None]).to(T)
    return {"dY": dY[:-1], "dweights": dweights}


# ---- what a pass cannot do without --------------------------------------------

def work(case):
    c = case
    op, b, m = c["op"], SIZE[c["dtype"]], c["m"]
    if op == "linear":
        n, k = c["n"], c["k"]
        items = m * k + k * n + m * n * (1 + c["residual"] + c["z"]) + n * c["bias"]
        return {"bytes": items * b, "flops": 2 * m * n * k}
    if op == "linear_backward":
        n, k = c["n"], c["k"]
        items = m * n * (1 if c["act"] == "none" else 2) + 2 * m * k + 2 * n * k + n * c["bias"]
        return {"bytes": items * b, "flops": 4 * m * n * k}
    E, K = c["experts"], c["top"]
    if op == "route":
        return {"bytes": m * E * b + 4 * E * c["bias"] + 16 * m * K + 4 * (E + 1),
                "flops": 10 * m * E}
    if op == "route_backward":
        return {"bytes": 2 * m * E * b + 8 * m * K, "flops": 10 * m * E}
    n = c["n"]
    if op in ("experts", "experts_backward"):
        k, R = c["k"], m * K
        hit = E * (1 - (1 - K / E) ** m)                # experts with a row, on average
        xin = m * k if c["gather"] else R * k
        if op == "experts":
            items = xin + R * n * (1 + c["z"]) + hit * (k * n + n * c["bias"])
            return {"bytes": int(items * b) + 4 * (E + 1) + 4 * R * c["gather"],
                    "flops": 2 * R * n * k}
        items = xin + R * k + R * n * (1 if c["act"] == "none" else 2) + \
            (hit + E) * k * n + E * n * c["bias"]
        return {"bytes": int(items * b) + 4 * (E + 1) + 4 * R * c["gather"], "flops": 4 * R * n * k}
    live = m - c["padded"]
    if op == "combine":
        return {"bytes": (live * K + m * (1 + c["residual"])) * n * b + 8 * m * K,
                "flops": 2 * live * K * n}
    return {"bytes": (2 * live * K + m) * n * b + 12 * m * K, "flops": 3 * live * K * n}


# ---- the definitions in 64 bits -------------------------------------------------

def _phi(z, act):
    """An activation and its derivative in 64 bits."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        on = (z > 0).double()
        return z * on, on
    if act == "silu":
        q = torch.sigmoid(z)
        return z * q, q + z * q * (1 - q)
    if act == "gelu":
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * cdf, cdf + z * (-z.square() / 2).exp() / math.sqrt(2 * math.pi)
    # tanh form: 0.5 (1 + tanh u) = sigmoid(2u)
    a, b = math.sqrt(2 / math.pi), 0.044715
    q = torch.sigmoid(2 * a * (z + b * z.pow(3)))
    return z * q, q + z * q * (1 - q) * 2 * a * (1 + 3 * b * z.square())


def _exact_route(s):
    c = s["case"]
    m, E, K, G = c["m"], c["experts"], c["top"], c["groups"]
    x = s["logits"].double()
    dead = torch.isinf(x) & (x < 0)
    if c["score"] == "softmax":
        score = torch.softmax(x.masked_fill(dead.all(1, keepdim=True), 0.0), 1)
    else:
        score = torch.sigmoid(x)
    key = x if G == 1 and not c["bias"] else score
    if c["bias"]:
        key = key + s["bias"].double()
    key = key.masked_fill(dead, -math.inf)
    if G > 1:
        by = key.view(m, G, E // G).sort(dim=2, descending=True).values[:, :, :2]
        total = by[:, :, 0] + (by[:, :, 1].masked_fill(by[:, :, 1] == -math.inf, 0.0)
                               if E // G > 1 else 0.0)
        order = total.sort(dim=1, descending=True, stable=True).indices
        drop = torch.ones(m, G, dtype=torch.bool, device="cuda")
        drop.scatter_(1, order[:, :c["top_groups"]], False)
        key = key.masked_fill(drop.repeat_interleave(E // G, 1), -math.inf)
    best = key.sort(dim=1, descending=True, stable=True)
    live = best.values[:, :K] > -math.inf
    e = best.indices[:, :K].masked_fill(~live, -1)
    w = score.gather(1, e.clamp(min=0)).masked_fill(~live, 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).masked_fill(~live.any(1, keepdim=True), 1.0)
    flat = e.flatten()
    order = flat.masked_fill(flat < 0, E).sort(dim=0, stable=True).indices
    count = torch.bincount(flat[flat >= 0], minlength=E)
    rows = int(count.sum())
    slots = torch.full_like(flat, -1)
    slots[order[:rows]] = torch.arange(rows, device="cuda")
    tokens = torch.full_like(flat, -1)
    tokens[:rows] = order[:rows] // K
    offsets = torch.cat([count.new_zeros(1), count.cumsum(0)])
    return {"weights": w * c["scale"], "experts": e.int(), "offsets": offsets.int(),
            "tokens": tokens.int(), "slots": slots.view(m, K).int()}


def _exact_route_backward(s):
    """Through the Jacobian of the weights, one choice at a time."""
    c = s["case"]
    x = s["logits"].double()
    x = x.masked_fill(torch.isinf(x).all(1, keepdim=True), 0.0)
    e = s["experts"].long()
    live = e >= 0
    score = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
    picked = score.gather(1, e.clamp(min=0)) * live
    gw = s["dweights"].double() * live * c["scale"]
    if c["renorm"]:
        total = picked.sum(1, keepdim=True).clamp(min=1e-300)
        gw = gw / total - (gw * picked).sum(1, keepdim=True) / total.square()
        gw = gw * live
    ds = torch.zeros_like(score)
    for j in range(c["top"]):
        ds.scatter_add_(1, e[:, j:j + 1].clamp(min=0), gw[:, j:j + 1])
    if c["score"] == "softmax":
        return {"dlogits": score * (ds - (score * ds).sum(1, keepdim=True))}
    return {"dlogits": ds * score * (1 - score)}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    op = c["op"]
    if op == "linear":
        z = s["X"].double().mm(s["W"].double())
        if c["bias"]:
            z.add_(s["bias"].double())
        y = _phi(z, c["act"])[0]
        if c["residual"]:
            y = y + s["R"].double()
        return {"Y": y, "Z": z} if c["z"] else {"Y": y}
    if op == "linear_backward":
        dz = s["dY"].double()
        if c["act"] != "none":
            dz = dz * _phi(s["Z"].double(), c["act"])[1]
        out = {"dX": dz.mm(s["W"].double().t()), "dW": dz.t().mm(s["X"].double()).t()}
        return dict(out, db=torch.ones(1, c["m"], dtype=torch.float64, device="cuda").mm(dz)[0]) \
            if c["bias"] else out
    if op == "route":
        return _exact_route(s)
    if op == "route_backward":
        return _exact_route_backward(s)
    off = s["offsets"].tolist()
    if op in ("experts", "experts_backward"):
        R, k, n, E = c["m"] * c["top"], c["k"], c["n"], c["experts"]
        zero = dict(dtype=torch.float64, device="cuda")
        out = {}
        if op == "experts":
            out["Y"] = torch.zeros(R, n, **zero)
            if c["z"]:
                out["Z"] = torch.zeros(R, n, **zero)
        else:
            out["dX"], out["dW"] = torch.zeros(R, k, **zero), torch.zeros(E, k, n, **zero)
            if c["bias"]:
                out["db"] = torch.zeros(E, n, **zero)
        for e in range(E):
            lo, hi = off[e], off[e + 1]
            if lo == hi:
                continue
            rows = s["tokens"][lo:hi].long() if c["gather"] else torch.arange(lo, hi, device="cuda")
            x, W = s["X"].index_select(0, rows).double(), s["W"][e].double()
            if op == "experts":
                z = x.mm(W)
                if c["bias"]:
                    z += s["bias"][e].double()
                out["Y"][lo:hi] = _phi(z, c["act"])[0]
                if c["z"]:
                    out["Z"][lo:hi] = z
            else:
                dz = s["dY"][lo:hi].double()
                if c["act"] != "none":
                    dz = dz * _phi(s["Z"][lo:hi].double(), c["act"])[1]
                out["dX"][lo:hi] = dz.mm(W.t())
                out["dW"][e] = dz.t().mm(x).t()
                if c["bias"]:
                    out["db"][e] = dz.sum(0)
        return out
    m, K, n = c["m"], c["top"], c["n"]
    if op == "combine":
        y = s["R"].double() if c["residual"] else torch.zeros(m, n, dtype=torch.float64, device="cuda")
        for j in range(K):
            at = s["slots"][:, j].long()
            w = s["weights"][:, j].double().masked_fill(at < 0, 0.0)
            y = y + w[:, None] * s["Y"].index_select(0, at.clamp(min=0)).double()
        return {"out": y}
    dY = torch.zeros(m * K, n, dtype=torch.float64, device="cuda")
    dw = torch.zeros(m, K, dtype=torch.float64, device="cuda")
    for j in range(K):
        t = (s["slots"][:, j] >= 0).nonzero()[:, 0]
        at = s["slots"][t, j].long()
        dY[at] = s["weights"][t, j].double()[:, None] * s["dout"][t].double()
        dw[t, j] = (s["dout"][t].double() * s["Y"][at].double()).sum(1)
    return {"dY": dY, "dweights": dw}
