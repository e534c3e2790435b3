"""The feed-forward block operators' measured cases: layer_norm, gated_linear,
quantize, linear_fp8, and the gradients of the first two.

Each case is one call, or one call's gradients, as a model's program makes
it.  With ``own`` false, ``run`` computes it from elementary torch
operations in 32 bits; with ``own`` true it calls the framework.  ``exact``
computes the same from the definition in 64 bits.

Symbols: m tokens, k inputs and n outputs of a product (n alone: the features
of a norm).  ``w`` is the order of a weight (k x n): "kn" has its rows
contiguous, "nk" its columns (a weight kept as n x k and passed transposed).
8-bit operands have one scale for each block of 128 along the summed index:
of every row ("rows") or of 128 rows together ("blocks").
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16,
         "e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
BLOCK = 128
EPS = 1e-5


def listed():
    return [
        # one token of a served model: latency alone
        dict(name="norm_token_bf16", op="norm", dtype="bf16", m=1, n=4096, affine=True, kept=False),
        # a training step's forward pass, odd sizes in fp32 (the ragged matrix
        # product's); keeps the rows' statistics
        dict(name="norm_ragged_f32", op="norm", dtype="f32", m=4097, n=3001, affine=True, kept=True),
        # its gradients in a training step, with the residual stream's added
        dict(name="norm_backward_bf16", op="norm_backward", dtype="bf16", m=8192, n=4096, affine=True,
             residual=True),
        # few long rows, odd, without weights
        dict(name="norm_backward_f16", op="norm_backward", dtype="f16", m=255, n=16383, affine=False,
             residual=False),
        # one token: both weights are read for one row
        dict(name="gated_token_bf16", op="gated", dtype="bf16", m=1, n=8192, k=4096, w="nk",
             act="silu", bias=False, z=False),
        # a training step's forward pass: keeps the pre-activations
        dict(name="gated_prompt_bf16", op="gated", dtype="bf16", m=8192, n=8192, k=4096, w="nk",
             act="silu", bias=False, z=True),
        # the gradients of a training step
        dict(name="gated_backward_bf16", op="gated_backward", dtype="bf16", m=8192, n=4096, k=4096,
             w="nk", act="silu", bias=False),
        # the same with biases in the other order, odd sizes
        dict(name="gated_backward_f16", op="gated_backward", dtype="f16", m=1023, n=2047, k=1024,
             w="kn", act="gelu", bias=True),
        # a prompt's activations, a scale for each row's 128 features
        dict(name="quantize_prompt_bf16", op="quantize", dtype="bf16", q="e4m3", r=8192, c=4096,
             order="rows", scales="rows"),
        # a weight kept as k x n, laid out as n x k with a scale for each block
        dict(name="quantize_weight_f32", op="quantize", dtype="f32", q="e4m3", r=4096, c=4096,
             order="columns", scales="blocks"),
        # a few tokens of a served model, onto the residual stream
        dict(name="fp8_decode_bf16", op="fp8", dtype="bf16", x="e4m3", q="e4m3", m=16, n=4096, k=4096,
             scales="blocks", act="none", bias=False, residual=True),
        # a prompt, an odd number of tokens
        dict(name="fp8_prompt_bf16", op="fp8", dtype="bf16", x="e4m3", q="e4m3", m=8191, n=8192,
             k=4096, scales="blocks", act="silu", bias=True, residual=False),
    ]


def _log(rng, lo, hi):
    """A size of [lo, hi], spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _feature(rng, lo, hi, to=8):
    """A feature count: mostly whole 16-byte rows, sometimes odd."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.3 else max(to, v // to * to)


def draw(rng):
    op = rng.choice(("norm", "norm_backward", "gated", "gated", "gated_backward", "quantize", "fp8",
                     "fp8"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    c = dict(op=op, dtype=dtype)
    if op in ("norm", "norm_backward"):
        while True:
            m, n = _log(rng, 1, 16384), _feature(rng, 16, 32768)
            if m * n <= 8192 * 8192:
                break
        c.update(m=m, n=n, affine=rng.random() < 0.7)
        if op == "norm":
            c.update(kept=rng.random() < 0.5)
        else:
            c.update(residual=rng.random() < 0.5)
    elif op in ("gated", "gated_backward"):
        most = 8192 * 4096 * (8192 if op == "gated" else 4096) // (8 if dtype == "f32" else 1)
        while True:
            m, n, k = _log(rng, 1, 8192), _feature(rng, 16, 8192), _feature(rng, 16, 8192)
            if m * n * k <= most:
                break
        c.update(m=m, n=n, k=k, w=rng.choice(("kn", "nk")), act=rng.choice(ACTS),
                 bias=rng.random() < 0.5)
        if op == "gated":
            c.update(z=rng.random() < 0.5)
    elif op == "quantize":
        while True:
            r, cols = _log(rng, 1, 16384), _feature(rng, 16, 16384, 16)
            if r * cols <= 8192 * 8192:
                break
        c.update(q=rng.choice(("e4m3", "e4m3", "e5m2")), r=r, c=cols,
                 order=rng.choice(("rows", "columns")), scales=rng.choice(("rows", "blocks")))
    else:
        while True:
            m, n, k = _log(rng, 1, 8192), _feature(rng, 16, 8192), _feature(rng, 16, 8192, 16)
            if m * n * k <= 8192 * 8192 * 4096:
                break
        c.update(x=rng.choice(("e4m3", "e4m3", "e5m2")), q=rng.choice(("e4m3", "e4m3", "e5m2")), m=m,
                 n=n, k=k, scales=rng.choice(("rows", "blocks")), act=rng.choice(ACTS),
                 bias=rng.random() < 0.5, residual=rng.random() < 0.5)
    return c


# ---- inputs ----------------------------------------------------------------

def _empty(*shape, dtype):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def _weight(g, k, n, order, dtype):
    """A weight (k, n) of the scale 1/sqrt(k), in the order asked for."""
    shape = (k, n) if order == "kn" else (n, k)
    w = torch.randn(*shape, generator=g, device="cuda").mul_(k ** -0.5).to(dtype)
    return w if order == "kn" else w.t()


def _like(w):
    """A zeroed tensor of w's shape and order."""
    return torch.zeros_like(w, memory_format=torch.preserve_format)


def _stream(g, m, n):
    """Rows as a residual stream has them: each with an offset and a spread of its
    own, some features far larger than the others."""
    x = torch.randn(m, n, generator=g, device="cuda")
    x *= 0.5 + torch.rand(m, 1, generator=g, device="cuda")
    x += torch.randn(m, 1, generator=g, device="cuda") * 0.5
    return x * (1 + 8 * (torch.rand(n, generator=g, device="cuda") < 0.01))


def _blocks(rows, by):
    """Blocks of `rows` rows: each its own, or 128 together."""
    return rows if by == "rows" else -(-rows // BLOCK)


def _whole(x, by):
    """x (r, c) as whole blocks (block rows, rows each, blocks, 128), zeros behind
    its edges."""
    r, c = x.shape
    high = 1 if by == "rows" else BLOCK
    p = torch.zeros(-(-r // high) * high, -(-c // BLOCK) * BLOCK, dtype=x.dtype, device="cuda")
    p[:r, :c] = x
    return p.view(p.shape[0] // high, high, -1, BLOCK)


def _spread(scales, r, c, by):
    """The scale of each element of an (r, c) matrix."""
    if by != "rows":
        scales = scales.repeat_interleave(BLOCK, 0)[:r]
    return scales.repeat_interleave(BLOCK, 1)[:, :c]


def _quantized(x, q, by):
    """8-bit values of x (r, c) and their scales."""
    s = _whole(x, by).abs().amax((1, 3)).div(LARGEST[q]).clamp(min=2.0 ** -126)
    return (x / _spread(s, *x.shape, by)).to(TYPES[q]), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = TYPES[case["dtype"]]
    op = case["op"]
    s = dict(case=case)

    def rnd(*shape, dtype=T):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    if own:
        import precision_gemm_02_amd as pg
    if op in ("norm", "norm_backward"):
        m, n = case["m"], case["n"]
        X = _stream(g, m, n).to(T)
        s.update(X=X, weight=(1 + 0.1 * rnd(n, dtype=torch.float32)).to(T) if case["affine"] else None)
        if op == "norm":
            s.update(bias=(0.1 * rnd(n, dtype=torch.float32)).to(T) if case["affine"] else None,
                     Y=_empty(m, n, dtype=T),
                     mean=_empty(m, dtype=torch.float32) if case["kept"] else None,
                     rstd=_empty(m, dtype=torch.float32) if case["kept"] else None)
        else:
            # the statistics that the forward pass kept
            x = X.double()
            mean = x.mean(1)
            var = (x - mean[:, None]).square().mean(1)
            s.update(mean=mean.float(), rstd=(var + EPS).rsqrt().float(), dY=rnd(m, n),
                     R=rnd(m, n) if case["residual"] else None, dX=_empty(m, n, dtype=T),
                     dw=_empty(n, dtype=T) if case["affine"] else None,
                     db=_empty(n, dtype=T) if case["affine"] else None)
            if own:
                size = pg.layer_norm_backward_workspace(m, n) if case["affine"] else 0
                s["ws"] = _empty(max(16, size), dtype=torch.uint8)
    elif op in ("gated", "gated_backward"):
        m, n, k = case["m"], case["n"], case["k"]
        s.update(X=rnd(m, k), Wg=_weight(g, k, n, case["w"], T), Wu=_weight(g, k, n, case["w"], T))
        if op == "gated":
            s.update(bg=rnd(n) if case["bias"] else None, bu=rnd(n) if case["bias"] else None,
                     Y=_empty(m, n, dtype=T), Zg=_empty(m, n, dtype=T) if case["z"] else None,
                     Zu=_empty(m, n, dtype=T) if case["z"] else None)
            if own:
                s["ws"] = _empty(max(16, pg.gated_linear_workspace(m, n, k, T)), dtype=torch.uint8)
        else:
            s.update(dY=rnd(m, n), Zg=rnd(m, n), Zu=rnd(m, n), dX=_empty(m, k, dtype=T),
                     dWg=_like(s["Wg"]), dWu=_like(s["Wu"]),
                     dbg=_empty(n, dtype=T) if case["bias"] else None,
                     dbu=_empty(n, dtype=T) if case["bias"] else None)
            if own:
                size = pg.gated_linear_backward_workspace(m, n, k, T)
                s["ws"] = _empty(max(16, size), dtype=torch.uint8)
    elif op == "quantize":
        r, c, by = case["r"], case["c"], case["scales"]
        X = _stream(g, r, c).to(T)
        if case["order"] == "columns":
            X = X.t().contiguous().t()
        s.update(X=X, Q=_empty(r, c, dtype=TYPES[case["q"]]),
                 scales=_empty(_blocks(r, by), -(-c // BLOCK), dtype=torch.float32))
    else:
        m, n, k = case["m"], case["n"], case["k"]
        X, sx = _quantized(_stream(g, m, k), case["x"], "rows")
        W, sw = _quantized(rnd(n, k, dtype=torch.float32) * k ** -0.5, case["q"], case["scales"])
        s.update(X=X, sx=sx, W=W.t(), sw=sw.t(), bias=rnd(n) if case["bias"] else None,
                 R=rnd(m, n) if case["residual"] else None, Y=_empty(m, n, dtype=T))
        if own:
            s["ws"] = _empty(max(16, pg.linear_fp8_workspace(m, n, k)), dtype=torch.uint8)
    return s


# ---- the framework's operators ----------------------------------------------

def _run_own(s):
    import precision_gemm_02_amd as pg
    c = s["case"]
    op = c["op"]
    if op == "norm":
        pg.layer_norm(s["X"], s["Y"], weight=s["weight"], bias=s["bias"], eps=EPS, mean=s["mean"],
                      rstd=s["rstd"])
        return {"Y": s["Y"], "mean": s["mean"], "rstd": s["rstd"]} if c["kept"] else {"Y": s["Y"]}
    if op == "norm_backward":
        pg.layer_norm_backward(s["dY"], s["X"], s["mean"], s["rstd"], weight=s["weight"],
                               residual=s["R"], dX=s["dX"], dweight=s["dw"], dbias=s["db"],
                               ws=s["ws"])
        return {"dX": s["dX"], "dw": s["dw"], "db": s["db"]} if c["affine"] else {"dX": s["dX"]}
    if op == "gated":
        pg.gated_linear(s["X"], s["Wg"], s["Wu"], s["Y"], bias_gate=s["bg"], bias_up=s["bu"],
                        act=c["act"], Z_gate=s["Zg"], Z_up=s["Zu"], ws=s["ws"])
        return {"Y": s["Y"], "Zg": s["Zg"], "Zu": s["Zu"]} if c["z"] else {"Y": s["Y"]}
    if op == "gated_backward":
        pg.gated_linear_backward(s["dY"], s["X"], s["Wg"], s["Wu"], s["Zg"], s["Zu"], act=c["act"],
                                 dX=s["dX"], dW_gate=s["dWg"], dW_up=s["dWu"], dbias_gate=s["dbg"],
                                 dbias_up=s["dbu"], ws=s["ws"])
        out = {"dX": s["dX"], "dWg": s["dWg"], "dWu": s["dWu"]}
        return dict(out, dbg=s["dbg"], dbu=s["dbu"]) if c["bias"] else out
    if op == "quantize":
        pg.quantize(s["X"], s["Q"], s["scales"])
        return {"Q": s["Q"], "scales": s["scales"]}
    pg.linear_fp8(s["X"], s["sx"], s["W"], s["sw"], s["Y"], bias=s["bias"], act=c["act"],
                  residual=s["R"], ws=s["ws"])
    return {"Y": s["Y"]}


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


def run(s):
    if own:
        return _run_own(s)
    c = s["case"]
    op, T = c["op"], TYPES[c["dtype"]]
    if op == "norm":
        x = s["X"].float()
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
        y = d * rstd
        if c["affine"]:
            y = y * s["weight"].float() + s["bias"].float()
        out = {"Y": y.to(T)}
        return dict(out, mean=mean[:, 0], rstd=rstd[:, 0]) if c["kept"] else out
    if op == "norm_backward":
        d, rstd = s["dY"].float(), s["rstd"][:, None]
        xh = (s["X"].float() - s["mean"][:, None]) * rstd
        g = d * s["weight"].float() if c["affine"] else d
        dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        if c["residual"]:
            dx = dx + s["R"].float()
        out = {"dX": dx.to(T)}
        return dict(out, dw=(d * xh).sum(0).to(T), db=d.sum(0).to(T)) if c["affine"] else out
    if op == "gated":
        x = s["X"].float()
        zg, zu = x @ s["Wg"].float(), x @ s["Wu"].float()
        if c["bias"]:
            zg, zu = zg + s["bg"].float(), zu + s["bu"].float()
        out = {"Y": (_act(zg, c["act"]) * zu).to(T)}
        return dict(out, Zg=zg.to(T), Zu=zu.to(T)) if c["z"] else out
    if op == "gated_backward":
        d, zg, zu, x = s["dY"].float(), s["Zg"].float(), s["Zu"].float(), s["X"].float()
        dg, du = d * zu * _act_grad(zg, c["act"]), d * _act(zg, c["act"])
        out = {"dX": (dg @ s["Wg"].float().t() + du @ s["Wu"].float().t()).to(T),
               "dWg": (x.t() @ dg).to(T), "dWu": (x.t() @ du).to(T)}
        return dict(out, dbg=dg.sum(0).to(T), dbu=du.sum(0).to(T)) if c["bias"] else out
    if op == "quantize":
        q, scales = _quantized(s["X"].float(), c["q"], c["scales"])
        return {"Q": q, "scales": scales}
    x = s["X"].float() * _spread(s["sx"], c["m"], c["k"], "rows")
    w = s["W"].t().float() * _spread(s["sw"].t(), c["n"], c["k"], c["scales"])
    y = x @ w.t()
    if c["bias"]:
        y = y + s["bias"].float()
    y = _act(y, c["act"])
    if c["residual"]:
        y = y + s["R"].float()
    return {"Y": y.to(T)}


# ---- what a pass cannot do without --------------------------------------------

def work(case):
    c = case
    op, b = c["op"], SIZE[c["dtype"]]
    if op == "norm":
        m, n = c["m"], c["n"]
        return {"bytes": (2 * m * n + 2 * n * c["affine"]) * b + 8 * m * c["kept"], "flops": 8 * m * n}
    if op == "norm_backward":
        m, n = c["m"], c["n"]
        return {"bytes": (m * n * (3 + c["residual"]) + 3 * n * c["affine"]) * b + 8 * m,
                "flops": (14 if c["affine"] else 10) * m * n}
    if op == "gated":
        m, n, k = c["m"], c["n"], c["k"]
        items = m * k + 2 * k * n + m * n * (3 if c["z"] else 1) + 2 * n * c["bias"]
        return {"bytes": items * b, "flops": 4 * m * n * k}
    if op == "gated_backward":
        m, n, k = c["m"], c["n"], c["k"]
        items = 3 * m * n + 2 * m * k + 4 * k * n + 2 * n * c["bias"]
        return {"bytes": items * b, "flops": 8 * m * n * k}
    if op == "quantize":
        r, cols = c["r"], c["c"]
        return {"bytes": r * cols * (b + 1) + 4 * _blocks(r, c["scales"]) * -(-cols // BLOCK),
                "flops": 3 * r * cols}
    m, n, k = c["m"], c["n"], c["k"]
    return {"bytes": m * k + k * n + 4 * -(-k // BLOCK) * (m + _blocks(n, c["scales"])) +
            b * (m * n * (1 + c["residual"]) + n * c["bias"]), "flops": 2 * m * n * k}


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


def _by_block(s, r, c, by):
    """Row and column blocks of an (r, c) matrix, with the scale of each."""
    high = 1 if by == "rows" else BLOCK
    i = torch.arange(r, device="cuda") // high
    j = torch.arange(c, device="cuda") // BLOCK
    return s.double().index_select(0, i).index_select(1, j)


def _exact_quantize(s):
    """The scales by reductions over an index of blocks, the values by the steps
    of the 8-bit type: 2^-bits of the power of two below, at least the smallest."""
    c, x = s["case"], s["X"].double()
    r, cols = x.shape
    blocks = -(-cols // BLOCK)
    j = torch.arange(cols, device="cuda") // BLOCK
    top = torch.zeros(r, blocks, dtype=torch.float64, device="cuda")
    top.scatter_reduce_(1, j.expand(r, cols), x.abs(), "amax")
    if c["scales"] == "blocks":
        i = torch.arange(r, device="cuda") // BLOCK
        high = torch.zeros(-(-r // BLOCK), blocks, dtype=torch.float64, device="cuda")
        top = high.scatter_reduce_(0, i[:, None].expand(r, blocks), top, "amax")
    scales = torch.maximum(top / LARGEST[c["q"]], torch.full_like(top, 2.0 ** -126))
    v = x / _by_block(scales, r, cols, c["scales"])
    bits, low = (3, -6) if c["q"] == "e4m3" else (2, -14)
    e = torch.frexp(v)[1].double() - 1
    step = torch.exp2(e.clamp(min=low) - bits)
    return {"Q": torch.round(v / step) * step, "scales": scales}


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    op = c["op"]
    if op == "norm":
        x = s["X"].double()
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + EPS).pow(-0.5)
        y = x.sub(mean[:, None]).mul(rstd[:, None])
        if c["affine"]:
            y = torch.addcmul(s["bias"].double(), y, s["weight"].double())
        return {"Y": y, "mean": mean, "rstd": rstd} if c["kept"] else {"Y": y}
    if op == "norm_backward":
        d, r = s["dY"].double(), s["rstd"].double()[:, None]
        h = s["X"].double().sub(s["mean"].double()[:, None]).mul(r)
        g = d.mul(s["weight"].double()) if c["affine"] else d
        n = c["n"]
        dx = (n * g - g.sum(1, keepdim=True) - h * (g * h).sum(1, keepdim=True)) * (r / n)
        if c["residual"]:
            dx = dx.add(s["R"].double())
        if not c["affine"]:
            return {"dX": dx}
        one = torch.ones(1, c["m"], dtype=torch.float64, device="cuda")
        return {"dX": dx, "dw": one.mm(h.mul(d))[0], "db": one.mm(d)[0]}
    if op == "gated":
        x = s["X"].double()
        zg, zu = x.mm(s["Wg"].double()), x.mm(s["Wu"].double())
        if c["bias"]:
            zg.add_(s["bg"].double())
            zu.add_(s["bu"].double())
        y = zu.mul(_phi(zg, c["act"])[0])
        return {"Y": y, "Zg": zg, "Zu": zu} if c["z"] else {"Y": y}
    if op == "gated_backward":
        d, x = s["dY"].double(), s["X"].double()
        value, slope = _phi(s["Zg"].double(), c["act"])
        dg, du = slope.mul(s["Zu"].double()).mul(d), value.mul(d)
        dx = dg.mm(s["Wg"].double().t()).addmm_(du, s["Wu"].double().t())
        out = {"dX": dx, "dWg": dg.t().mm(x).t(), "dWu": du.t().mm(x).t()}
        if c["bias"]:
            one = torch.ones(1, c["m"], dtype=torch.float64, device="cuda")
            out.update(dbg=one.mm(dg)[0], dbu=one.mm(du)[0])
        return out
    if op == "quantize":
        return _exact_quantize(s)
    # block after block of the summed index
    m, n, k = c["m"], c["n"], c["k"]
    sx, sw = s["sx"].double(), s["sw"].t().double()
    z = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    if c["scales"] == "blocks":
        sw = sw.index_select(0, torch.arange(n, device="cuda") // BLOCK)
    for b in range(-(-k // BLOCK)):
        at = slice(b * BLOCK, min(k, (b + 1) * BLOCK))
        z.addmm_(s["X"][:, at].double() * sx[:, b:b + 1], (s["W"][at].t().double() * sw[:, b:b + 1]).t())
    if c["bias"]:
        z.add_(s["bias"].double())
    y = _phi(z, c["act"])[0]
    return {"Y": y + s["R"].double() if c["residual"] else y}
