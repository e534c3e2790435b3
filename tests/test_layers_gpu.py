"""The layer operators on the GPU against plain 64-bit arithmetic on the CPU.

Sizes are small and chosen where the kernels can go wrong: one row, one
column, one inner index, one more or less than a tile, padded and unaligned
rows, experts without rows, tokens without experts.  Inputs of small whole
numbers make every sum exact in fp32, so that those results have to be equal
bit by bit; random inputs are held to bounds that count the roundings:

  a product of k terms summed in fp32: |error| <= (k + 2) 2^-24 sum |x||w|
  an activation: its slope is below 1.13, and its own evaluation is off by at
  most (|z| + 8) 2^-23 |z|
  each result: half a step of its type.
"""
import math
import random

import pytest
import torch

import precision_gemm_02_amd as pg
from layer_util import (Guarded, act64, half_step, ints, plan64, route64, slope64, weight)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]
ids = {F32: "f32", F16: "f16", BF16: "bf16"}.get


def gen(seed):
    return torch.Generator().manual_seed(seed)


def space(n):
    return torch.full((n + 16,), 0x7F, dtype=torch.uint8, device="cuda") if n else None


# (m, n, k): few-rows kernels (m <= 32), tiles of every class, edges of each
SHAPES = [(1, 1, 1), (1, 64, 64), (1, 257, 1023), (3, 17, 5), (16, 130, 72), (17, 64, 129),
          (32, 72, 520), (33, 65, 31), (64, 64, 128), (65, 129, 64), (128, 256, 40),
          (200, 136, 1), (300, 263, 264)]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("pad", [0, 5, 8])
def test_linear_exact_integers(dtype, order, shape, pad):
    m, n, k = shape
    g = gen(1)
    X = Guarded(m, k, dtype, pad=pad, data=ints(g, m, k).to(dtype))
    W = weight(g, (), k, n, order, dtype, integer=True, pad=pad)
    bias, R = ints(g, n).to(dtype).cuda(), ints(g, m, n).cuda()
    Y = Guarded(m, n, F32, pad=pad)
    Z = Guarded(m, n, dtype, pad=pad)
    pg.linear(X.t, W, Y.t, bias=bias, act="relu", residual=R, Z=Z.t)
    z = X.t.double().cpu() @ W.double().cpu() + bias.double().cpu()
    assert torch.equal(Y.t.double().cpu(), z.clamp(min=0) + R.double().cpu())
    assert torch.equal(Z.t.cpu(), z.to(dtype))       # one rounding, to nearest even
    Y.check("Y")
    Z.check("Z")
    # the same with the summed index shared between workgroups
    ws = space(pg.linear_workspace(m, n, k, dtype))
    Y2 = Guarded(m, n, F32, pad=pad)
    pg.linear(X.t, W, Y2.t, bias=bias, act="relu", residual=R, Z=Z.t, ws=ws)
    assert torch.equal(Y2.t, Y.t)
    Y2.check("Y")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("shape", [(70, 70, 66), (130, 262, 190), (300, 134, 1002), (140, 5, 130),
                                   (140, 130, 3), (65, 1, 4), (200, 66, 64)], ids=str)
@pytest.mark.parametrize("pad,shift", [(0, 0), (2, 2), (2, 1), (1, 0), (6, 4)])
def test_linear_alignments(dtype, order, shape, pad, shift):
    """Rows at 4-byte and at element boundaries, straddling chunks on every edge;
    the buffers' ends are the operands' ends."""
    m, n, k = shape
    g = gen(21)
    X = Guarded(m, k, dtype, pad=pad, shift=shift, data=ints(g, m, k).to(dtype))
    rows, cols = (k, n) if order == "kn" else (n, k)
    W = Guarded(rows, cols, dtype, pad=pad, shift=shift, data=ints(g, rows, cols).to(dtype))
    w = W.t if order == "kn" else W.t.t()
    Y = Guarded(m, n, F32, pad=pad, shift=shift)
    pg.linear(X.t, w, Y.t)
    want = X.t.double().cpu() @ w.double().cpu()
    assert torch.equal(Y.t.double().cpu(), want)
    Y.check("Y")
    # the gradients' products of the same operands
    dX = Guarded(m, n, dtype, pad=pad, shift=shift)
    dW = Guarded(n, n, F32, pad=pad, shift=shift)
    ws = space(pg.linear_backward_workspace(m, k, n, dtype))
    pg.linear_backward(X.t, dX.t, w.t(), dX=dX.t, ws=ws)
    assert torch.equal(dX.t.cpu(), want.to(dtype))
    dX.check("dX")
    D = Guarded(m, n, dtype, pad=pad, shift=shift, data=ints(g, m, n).to(dtype))
    ws = space(pg.linear_backward_workspace(m, n, n, dtype))
    pg.linear_backward(D.t, D.t, None, dW=dW.t, ws=ws)
    assert torch.equal(dW.t.double().cpu(), D.t.double().cpu().t() @ D.t.double().cpu())
    dW.check("dW")


@pytest.mark.parametrize("dtype", [F16, BF16], ids=ids)
@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("k", [66, 126, 130, 186, 188, 190, 194, 258, 1026])
@pytest.mark.parametrize("shape", [(65, 40), (129, 65), (257, 514)], ids=str)
def test_linear_waves_without_rows(dtype, order, k, shape):
    """Rows at 4-byte boundaries where whole waves of the last tiles have none, at
    inner sizes around the last whole tile: such a wave issues no loads of its
    own for the tiles that are read with guards, and still has to wait for the
    ones before."""
    m, n = shape
    g = gen(k)
    X = Guarded(m, k, dtype, pad=2, shift=2, data=ints(g, m, k).to(dtype))
    rows, cols = (k, n) if order == "kn" else (n, k)
    W = Guarded(rows, cols, dtype, pad=2, shift=2, data=ints(g, rows, cols).to(dtype))
    w = W.t if order == "kn" else W.t.t()
    want = X.t.double().cpu() @ w.double().cpu()
    for _ in range(8):
        Y = Guarded(m, n, F32, pad=2)
        pg.linear(X.t, w, Y.t)
        assert torch.equal(Y.t.double().cpu(), want)
        Y.check("Y")


# one more, one less and exactly whole tiles of the large class, long k over
# several workgroups
LARGE = [(2304, 2304, 192), (2305, 2312, 200), (4096, 2048, 64), (100, 96, 8192), (8, 64, 16384),
         (2, 3000, 4096), (515, 517, 999), (1030, 1026, 1002), (48, 2048, 2048), (1000, 1000, 1000)]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("shape", LARGE, ids=str)
def test_linear_exact_integers_large(dtype, order, shape):
    m, n, k = shape
    g = gen(2)
    X = ints(g, m, k).to(dtype).cuda()
    W = weight(g, (), k, n, order, dtype, integer=True)
    R = ints(g, m, n).cuda()
    want = X.double() @ W.double()
    for ws in (None, space(pg.linear_workspace(m, n, k, dtype))):
        Y = Guarded(m, n, F32, data=R)
        pg.linear(X, W, Y.t, residual=Y.t, ws=ws)    # in place
        assert torch.equal(Y.t.double(), want + R.double())
        Y.check("Y")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("shape", [(1, 200, 300), (70, 130, 96), (130, 67, 33)], ids=str)
def test_linear_random(dtype, act, shape):
    m, n, k = shape
    g = gen(3)
    X = (torch.randn(m, k, generator=g) * 1.5).to(dtype).cuda()
    W = weight(g, (), k, n, "nk", dtype, scale=k ** -0.5)
    bias, R = torch.randn(n, generator=g).to(dtype).cuda(), torch.randn(m, n, generator=g)
    R = R.to(dtype).cuda()
    Y, Z = torch.empty(m, n, dtype=dtype, device="cuda"), torch.empty(m, n, dtype=dtype, device="cuda")
    pg.linear(X, W, Y, bias=bias, act=act, residual=R, Z=Z)
    x, w = X.double().cpu(), W.double().cpu()
    z = x @ w + bias.double().cpu()
    sums = (k + 2) * 2.0 ** -24 * (x.abs() @ w.abs() + bias.double().cpu().abs())
    h = half_step(dtype)
    assert ((Z.double().cpu() - z).abs() <= h * z.abs() * (1 + h) + sums * (1 + h) + 1e-30).all()
    y = act64(z, act) + R.double().cpu()
    own = 1.13 * sums + (z.abs() + 8) * 2.0 ** -23 * z.abs() + 2.0 ** -23 * y.abs()
    tiny = torch.finfo(dtype).tiny * torch.finfo(dtype).eps      # a subnormal step
    assert ((Y.double().cpu() - y).abs() <= h * y.abs() * (1 + h) + own * (1 + h) + tiny).all()


PAIRS = [(F32, F32), (F16, F16), (BF16, BF16), (F16, F32), (BF16, F32)]


def logistic_argument(z, act):
    """x of z / (1 + exp(-x)): silu's z, and 2 u of 0.5 z (1 + tanh u), where 1 +
    tanh u itself would cancel in 64 bits."""
    return 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3) if act == "gelu_tanh" else z


@pytest.mark.parametrize("dtype,out", PAIRS, ids=lambda d: ids(d))
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_linear_activations_keep_their_tails(act, dtype, out):
    """Y = act(z) to a relative bound, z itself (one inner index, weight 1).

    fp32 results, in units of 2^-24 of the value: gelu 1.5 z^2 (the roundings of
    erfc's argument, whose condition is z^2 + 1) and 40 (16 units of the last
    place of erfcf, the products); the tanh form 5 of its argument and 16 (an exp
    of 3 units, sums, a division); silu 16.  16-bit results: 3e-6 (twice the
    polynomial's) and 2 z^2 + 16 for gelu, 8 of the argument and 16 for the others,
    and half a step.  The factor of z may be 0 where it is below the smallest normal
    number 2^-126 (exp(-2 u) passes 2^128 there): |z| times that."""
    z = torch.cat([torch.linspace(-12.9, 5, 1791), torch.linspace(-3, 3, 601)]).to(dtype)
    Y = torch.empty(z.numel(), 9, dtype=out, device="cuda")
    pg.linear(z[:, None].cuda(), torch.ones(1, 9, dtype=dtype, device="cuda"), Y, act=act)
    z = z.double()
    x = logistic_argument(z, act)
    want, w = act64(z, act) if act == "gelu" else z * torch.sigmoid(x), x.abs()
    if out is F32:
        units = {"gelu": 1.5 * z ** 2 + 40, "gelu_tanh": 5 * w + 16, "silu": 16}[act]
        own, h = units * 2.0 ** -24, 0.0
    else:
        own = 3e-6 + (2 * z ** 2 + 16) * 2.0 ** -24 if act == "gelu" else (8 * w + 16) * 2.0 ** -24
        h = half_step(out)
    flat = (1 + z.abs()) * torch.finfo(F32).tiny + torch.finfo(out).tiny * torch.finfo(out).eps / 2
    bound = want.abs() * (own + h + own * h) + flat
    for col in (0, 8):                       # whole chunks of columns and the edge
        assert ((Y[:, col].double().cpu() - want).abs() <= bound).all()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_bias_gradient_in_32_bits(act, dtype):
    """dbias of one row of ones is the slope, here as fp32: its terms to the
    roundings above, and 1 - q (q the logistic function) to 8 units of 1."""
    z = torch.linspace(-8, 5, 1041).to(dtype)[None]
    n = z.shape[1]
    db = torch.empty(n, device="cuda")
    ws = space(pg.linear_backward_workspace(1, n, 1, dtype, act))
    x = torch.zeros(1, 1, dtype=dtype, device="cuda")
    pg.linear_backward(torch.ones_like(z).cuda(), x, None, Z=z.cuda(), act=act, dbias=db, ws=ws)
    z = z[0].double()
    if act == "gelu":
        terms = 0.5 * torch.erfc(-z / math.sqrt(2)) + \
            z.abs() * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        bound = (1.5 * z ** 2 + 48) * terms
        want = slope64(z, act)
    else:
        c = 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * z ** 2) if act == "gelu_tanh" else 1
        x = logistic_argument(z, act)
        q, r = torch.sigmoid(x), torch.sigmoid(-x)
        want = q + z * q * r * c
        bound = (5 * x.abs() + 24) * (q + z.abs() * q * r * c) + 8 * z.abs() * q * c
    assert ((db.double().cpu() - want).abs() <= bound * 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_linear_special_values(dtype):
    """Infinities and NaN of one row stay in it; nothing is read past k."""
    m, n, k = 40, 48, 24
    g = gen(4)
    X = Guarded(m, k, dtype, pad=8, data=torch.randn(m, k, generator=g).to(dtype))
    X.t[3, 5] = math.inf
    X.t[7, 0] = math.nan
    W = weight(g, (), k, n, "kn", dtype, pad=8)
    for act in ("none", "relu", "gelu", "gelu_tanh", "silu"):
        Y = torch.empty(m, n, dtype=dtype, device="cuda")
        pg.linear(X.t, W, Y, act=act)
        assert Y[7].isnan().all()
        if act == "none":
            assert torch.equal(Y[3] > 0, W[5] > 0) and Y[3].isinf().all()
        rest = [r for r in range(m) if r not in (3, 7)]
        assert Y[rest].isfinite().all()


def test_linear_empty_and_zero_k():
    X, W = torch.zeros(4, 0, device="cuda"), torch.zeros(0, 5, device="cuda")
    bias = torch.arange(5.0, device="cuda")
    Y = torch.full((4, 5), 9.0, device="cuda")
    pg.linear(X, W, Y, bias=bias)
    assert torch.equal(Y, bias.expand(4, 5))
    Y = torch.full((4, 5), 9.0, device="cuda")
    pg.linear(torch.zeros(4, 3, device="cuda")[:0], torch.zeros(3, 5, device="cuda"), Y[:0])
    assert (Y == 9).all()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 64, 96), (5, 33, 17), (40, 130, 72),
                                   (257, 64, 129), (130, 264, 136), (1000, 24, 40)], ids=str)
@pytest.mark.parametrize("pad", [0, 8])
def test_linear_backward_exact_integers(dtype, order, shape, pad):
    m, n, k = shape
    g = gen(5)
    X = Guarded(m, k, dtype, pad=pad, data=ints(g, m, k, hi=1).to(dtype))
    dY = Guarded(m, n, dtype, pad=pad, data=ints(g, m, n, hi=1).to(dtype))
    Z = Guarded(m, n, dtype, pad=pad, data=ints(g, m, n).to(dtype))
    W = weight(g, (), k, n, order, dtype, integer=True, pad=pad)
    for act in ("none", "relu"):
        dX = Guarded(m, k, dtype, pad=pad)
        rows, cols = (k, n) if order == "kn" else (n, k)
        dW = Guarded(rows, cols, F32, pad=pad)
        db = torch.empty(n, device="cuda")
        ws = space(pg.linear_backward_workspace(m, n, k, dtype, act))
        pg.linear_backward(dY.t, X.t, W, Z=Z.t if act != "none" else None, act=act, dX=dX.t,
                           dW=dW.t if order == "kn" else dW.t.t(), dbias=db, ws=ws)
        dz = dY.t.double().cpu()
        if act == "relu":
            dz = dz * (Z.t.double().cpu() > 0)
        assert torch.equal(dX.t.cpu(), (dz @ W.double().cpu().t()).to(dtype))
        dw = X.t.double().cpu().t() @ dz
        assert torch.equal(dW.t.double().cpu(), dw if order == "kn" else dw.t())
        assert torch.equal(db.double().cpu(), dz.sum(0))
        dX.check("dX")
        dW.check("dW")


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_linear_backward_random(dtype, act):
    m, n, k = 150, 90, 70
    g = gen(6)
    X, dY = torch.randn(m, k, generator=g).to(dtype).cuda(), torch.randn(m, n, generator=g)
    dY, Z = dY.to(dtype).cuda(), (torch.randn(m, n, generator=g) * 2).to(dtype).cuda()
    W = weight(g, (), k, n, "nk", dtype)
    dX, dW = torch.empty_like(X), torch.empty(k, n, dtype=dtype, device="cuda")
    db = torch.empty(n, dtype=dtype, device="cuda")
    ws = space(pg.linear_backward_workspace(m, n, k, dtype, act))
    pg.linear_backward(dY, X, W, Z=Z, act=act, dX=dX, dW=dW, dbias=db, ws=ws)
    slope = slope64(Z.double().cpu(), act)
    dz = dY.double().cpu() * slope
    h = half_step(dtype)
    # dZ is rounded to the type; the slope itself (terms up to 1 + |z|, each
    # evaluated to (|z| + 8) 2^-23) is off by at most this
    z = Z.double().cpu().abs()
    edz = h * dz.abs() + dY.double().cpu().abs() * (1 + z) * (z + 8) * 2.0 ** -23
    w, x = W.double().cpu(), X.double().cpu()
    for got, want, err, mag, terms in (
            (dX, dz @ w.t(), edz @ w.t().abs(), dz.abs() @ w.t().abs(), n),
            (dW, x.t() @ dz, x.t().abs() @ edz, x.t().abs() @ dz.abs(), m),
            (db, dz.sum(0), edz.sum(0), dz.abs().sum(0), m)):
        bound = (err + (terms + 2) * 2.0 ** -24 * mag) * (1 + 2 * h) + h * want.abs()
        assert ((got.double().cpu() - want).abs() <= bound + 1e-7).all()


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_slopes_of_large_values(dtype, act):
    """The slope's limits, 1 and 0, at infinities and at finite values whose squares
    and cubes are not; a NaN reaches its own column alone."""
    big = torch.finfo(dtype).max
    z = [math.inf, big, min(big, 1e30), min(big, 1e20), 1e4, 2e4, 300, 60]
    n = 2 * len(z) + 1
    Z = torch.tensor([z + [-x for x in z] + [math.nan]]).to(dtype).cuda()
    W = torch.eye(n, dtype=dtype, device="cuda")[:, :n - 1].contiguous()
    ws = space(pg.linear_backward_workspace(1, n, n, dtype, act))
    for out in {dtype, F32}:
        db = torch.empty(n, dtype=out, device="cuda")
        dW = torch.empty(1, n, dtype=out, device="cuda")
        one = torch.ones(1, 1, dtype=dtype, device="cuda")
        pg.linear_backward(torch.ones_like(Z), one, None, Z=Z, act=act, dW=dW, dbias=db, ws=ws)
        want = [1.0] * len(z) + [0.0] * len(z)
        # at -60 silu's slope is -5e-25, beyond -10 the others' are below 1e-20
        assert (db[:-1].cpu().double() - torch.tensor(want)).abs().max() < 1e-20
        assert (dW[0, :-1].cpu().double() - torch.tensor(want)).abs().max() < 1e-20
    dX = torch.empty(1, n - 1, dtype=dtype, device="cuda")
    pg.linear_backward(torch.ones_like(Z)[:, :n - 1].contiguous(), None, W[:n - 1].contiguous(),
                       Z=Z[:, :n - 1].contiguous(), act=act, dX=dX, ws=ws)
    assert (dX[0].cpu().double() - torch.tensor(want)).abs().max() < 1e-20


def test_gradient_where_the_kept_pre_activation_overflows():
    """fp16: z = -70000 gives a finite result; Z keeps -inf, and its gradient is 0."""
    X, W = torch.full((1, 1), 700.0, device="cuda").half(), torch.full((1, 8), -100.0, device="cuda").half()
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        Y, Z = torch.empty(1, 8, device="cuda").half(), torch.empty(1, 8, device="cuda").half()
        pg.linear(X, W, Y, act=act, Z=Z)
        assert (Y == 0).all() and (Z == -math.inf).all()
        dX, dW = torch.empty(1, 1, device="cuda").half(), torch.empty(1, 8, device="cuda").half()
        ws = space(pg.linear_backward_workspace(1, 8, 1, F16, act))
        pg.linear_backward(torch.ones_like(Y), X, W, Z=Z, act=act, dX=dX, dW=dW, ws=ws)
        assert float(dX) == 0 and (dW == 0).all()


def test_linear_gradients_against_differences():
    """f32 gradients of sum(C * linear) against central differences in 64 bits."""
    m, n, k = 6, 9, 11
    g = gen(7)
    X, W0 = torch.randn(m, k, generator=g).cuda(), torch.randn(k, n, generator=g).cuda()
    b, C = torch.randn(n, generator=g).cuda(), torch.randn(m, n, generator=g).cuda()
    for act in ("gelu", "gelu_tanh", "silu"):
        Y, Z = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
        pg.linear(X, W0, Y, bias=b, act=act, Z=Z)
        dX, dW, db = torch.empty_like(X), torch.empty_like(W0), torch.empty_like(b)
        ws = space(pg.linear_backward_workspace(m, n, k, F32, act))
        pg.linear_backward(C, X, W0, Z=Z, act=act, dX=dX, dW=dW, dbias=db, ws=ws)

        def loss(x, w, bb):
            return float((act64(x @ w + bb, act) * C.double().cpu()).sum())
        x, w, bb = X.double().cpu(), W0.double().cpu(), b.double().cpu()
        h = 1e-5       # difference error h^2 f'''/6 ~ 1e-9, rounding 1e-15 / h = 1e-10
        for grad, t in ((dX, x), (dW, w), (db, bb)):
            flat, got = t.view(-1), grad.double().cpu().reshape(-1)
            for i in range(0, flat.numel(), 7):
                keep = float(flat[i])
                flat[i] = keep + h
                up = loss(x, w, bb)
                flat[i] = keep - h
                down = loss(x, w, bb)
                flat[i] = keep
                assert abs((up - down) / (2 * h) - float(got[i])) < 5e-5


def test_linear_backward_parts():
    """Each gradient alone, without what only the others read."""
    m, n, k = 64, 48, 32
    g = gen(8)
    X, dY = ints(g, m, k).cuda(), ints(g, m, n).cuda()
    W = weight(g, (), k, n, "kn", F32, integer=True)
    ws = space(pg.linear_backward_workspace(m, n, k, F32))
    dX, dW, db = torch.empty(m, k, device="cuda"), torch.empty(k, n, device="cuda"), \
        torch.empty(n, device="cuda")
    pg.linear_backward(dY, None, W, dX=dX, ws=ws)
    pg.linear_backward(dY, X, None, dW=dW, ws=ws)
    pg.linear_backward(dY, None, None, dbias=db, ws=ws)
    assert torch.equal(dX, dY @ W.t()) and torch.equal(dW, X.t() @ dY)
    assert torch.equal(db, dY.sum(0))
    # no rows: the weight's and bias's gradients are zero
    dW.fill_(7)
    db.fill_(7)
    pg.linear_backward(dY[:0], X[:0], W, dW=dW, dbias=db, ws=ws)
    assert (dW == 0).all() and (db == 0).all()


@pytest.mark.parametrize("m", [1, 16, 32, 33])
def test_bias_gradient_alone(m):
    """Neither X nor W: there is no inner size."""
    dY = ints(gen(32), m, 40).cuda()
    db = torch.empty(40, device="cuda")
    ws = space(pg.linear_backward_workspace(m, 40, 0, F32))
    pg.linear_backward(dY, None, None, dbias=db, ws=ws)
    assert torch.equal(db, dY.sum(0))
    pg.linear_backward(dY, torch.zeros(m, 0, device="cuda"), torch.zeros(0, 40, device="cuda"),
                       dX=torch.zeros(m, 0, device="cuda"), dW=torch.zeros(0, 40, device="cuda"),
                       dbias=db.fill_(7), ws=ws)
    assert torch.equal(db, dY.sum(0))


# ---- routing ---------------------------------------------------------------------

LOWEST = {F32: torch.finfo(F32).min, F16: -65504.0, BF16: torch.finfo(BF16).min}


def run_route(logits, top, **kw):
    m, E = logits.shape
    w = torch.full((m, top), -7.0, device="cuda")
    e = torch.full((m, top), -7, dtype=torch.int32, device="cuda")
    off = torch.full((E + 1,), -7, dtype=torch.int32, device="cuda")
    tok = torch.full((m * top,), -7, dtype=torch.int32, device="cuda")
    slots = torch.full((m, top), -7, dtype=torch.int32, device="cuda")
    ws = space(pg.route_workspace(m, E, top))
    pg.route(logits, w, e, off, tok, slots, ws=ws, **kw)
    return w, e, off, tok, slots


def check_route(logits, top, **kw):
    w, e, off, tok, slots = run_route(logits, top, **kw)
    bias = kw.pop("bias", None)
    we, ww = route64(logits.float().cpu(), LOWEST[logits.dtype], top,
                     bias=None if bias is None else bias.cpu(), **kw)
    assert torch.equal(e.cpu(), we)
    # 64-bit scores (a few 2^-53), rounded to fp32 once
    assert ((w.double().cpu() - ww).abs() <= ww.abs() * (2.0 ** -24 + 1e-12) + 1e-38).all()
    o, rows, s = plan64(we, logits.shape[1])
    assert off.tolist() == o and slots.tolist() == s
    assert tok.tolist() == rows + [-7] * (tok.numel() - len(rows))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("case", [
    # m, E, top, groups, top_groups, bias, renorm, scale
    (1, 1, 1, 1, 1, False, True, 1.0), (4, 64, 6, 1, 1, False, False, 1.0),
    (3, 8, 8, 1, 1, True, True, 2.5), (64, 60, 4, 4, 2, False, True, 1.0),
    (65, 128, 2, 8, 3, True, False, 0.5), (200, 100, 5, 1, 1, True, True, 1.0),
    (130, 256, 8, 8, 4, True, True, 2.0), (70, 300, 32, 1, 1, False, True, 1.0),
    (66, 1024, 3, 64, 5, True, True, 1.0), (129, 24, 3, 24, 4, False, True, 1.0)], ids=str)
def test_route(dtype, score, case):
    m, E, top, groups, top_groups, bias, renorm, scale = case
    g = gen(9)
    logits = (torch.randn(m, E, generator=g) * 2).to(dtype).cuda()
    b = (torch.randn(E, generator=g) * 0.1).cuda() if bias else None
    check_route(logits, top, bias=b, score=score, groups=groups, top_groups=top_groups,
                renorm=renorm, scale=scale)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_masks_ties_and_extremes(dtype, score):
    m, E = 70, 16
    g = gen(10)
    l = (torch.randn(m, E, generator=g)).to(dtype)
    l[0] = 0                                  # all equal: lowest indices
    l[1] = -math.inf                          # nothing left
    l[2] = LOWEST[dtype]                      # the same by the type's lowest value
    l[3, 2:] = -math.inf                      # fewer than top
    l[4, ::2] = LOWEST[dtype]
    l[5, 3] = math.inf
    l[6] = math.nan
    l[7, 1] = math.nan
    l[8] = torch.tensor([60000.0 if i % 2 else -60000.0 for i in range(E)]).to(dtype)
    l[9, 8:] = l[9, :8].clone()               # pairs of equal logits
    l[69] = -math.inf
    want = l.clone()
    want[want.isnan()] = -math.inf            # NaN counts as masked
    w, e, off, tok, slots = run_route(l.cuda(), 4, score=score)
    ref = want.float()
    ref[5, 3] = 1e30                          # +inf: the limit of a large logit
    we, ww = route64(ref, LOWEST[dtype], 4, score=score)
    assert torch.equal(e.cpu(), we)
    assert ((w.double().cpu() - ww).abs() <= ww * (2.0 ** -24 + 1e-12) + 1e-38).all()
    o, rows, s = plan64(we, E)
    assert off.tolist() == o and slots.tolist() == s and tok[:len(rows)].tolist() == rows
    assert (e[1] == -1).all() and (e[2] == -1).all() and (w[1] == 0).all()
    for kw in (dict(groups=4, top_groups=2), dict(bias=torch.zeros(E, device="cuda"))):
        ee = run_route(l.cuda(), 4, score=score, **kw)[1]
        kw2 = {x: (y.cpu() if x == "bias" else y) for x, y in kw.items()}
        assert torch.equal(ee.cpu(), route64(ref, LOWEST[dtype], 4, score=score, **kw2)[0])


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("top", [2, 5, 8])
def test_route_logits_far_apart(dtype, score, renorm, top):
    """Peaked rows without bias or groups: neighbours among the chosen logits whose
    bit patterns, as ordered integers, are more than 2^31 apart."""
    big = min(1e30, torch.finfo(dtype).max / 2)
    logits = torch.tensor([
        [10, -1, -2, -3, -4, -5, -6, -7], [2.5, -2.5, 0.5, -0.5, 1.5, -1.5, 0, -4],
        [big, -1e-3, -2e-3, -1, -2, -3, -4, -5], [-1, math.inf, -2, -3, -4, -5, -6, -7],
        [9, -0.6, -0.7, -0.8, -0.9, -1, -1.1, -1.2], [big, -big, 1, -1, 3, -3, 2, -2],
        [-3, -2, -1, 10, 4, -5, 7, -8]]).to(dtype)
    check_route(logits.repeat(11, 1).cuda(), top, score=score, renorm=renorm)


@pytest.mark.parametrize("groups", [1, 4])
def test_route_close_keys(groups):
    """Keys a few 1e-11 apart: below what the integer keys tell apart (2^-28), well
    above an exp's last bit (1e-16).  The bias of every second expert is chosen
    so that its key nearly meets its neighbour's."""
    m, E, top = 100, 32, 5
    g = gen(23)
    row = torch.randn(E, generator=g)
    logits = row.expand(m, E).clone()
    s = torch.sigmoid(row.double())
    bias = torch.zeros(E)
    for e in range(1, E, 2):
        # neighbours' scores differ by less than 2^-10, so that this bias's fp32
        # rounding is below 2^-35 = 3e-11
        row[e] = row[e - 1] + 1e-4 * (e + 1)
        s[e] = torch.sigmoid(row[e].double())
        bias[e] = float(s[e - 1] - s[e])
    logits = row.expand(m, E).contiguous()
    keys = s + bias.double()
    gap = (keys[0::2] - keys[1::2]).abs()
    assert float(gap.max()) < 2.0 ** -30 and float(gap.min()) > 1e-14
    check_route(logits.cuda(), top, bias=bias.cuda(), score="sigmoid", groups=groups,
                top_groups=max(1, groups // 2))


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups", [(1, 1), (3, 2), (12, 5)])
def test_route_masks_by_bias(dtype, score, groups, top_groups):
    """A bias that is infinite, NaN or beyond 3e38 masks its expert; a large
    finite one does not disturb the others' order."""
    m, E, top = 70, 12, 4
    g = gen(31)
    l = torch.randn(m, E, generator=g).to(dtype)
    for bad in (math.inf, -math.inf, math.nan, 3.2e38, -3.2e38):
        b = torch.randn(E, generator=g) * 0.1
        b[[1, 4, 5]] = bad
        w, e, off, tok, slots = run_route(l.cuda(), top, score=score, bias=b.cuda(), groups=groups,
                                          top_groups=top_groups)
        b[[1, 4, 5]] = -math.inf
        we, ww = route64(l.float(), LOWEST[dtype], top, bias=b, score=score, groups=groups,
                         top_groups=top_groups)
        assert torch.equal(e.cpu(), we), bad
        assert ((w.double().cpu() - ww).abs() <= ww.abs() * (2.0 ** -24 + 1e-12) + 1e-38).all()
    for large in (-1e4, -1e9, 1e6):
        b = torch.randn(E, generator=g) * 0.1
        b[[2, 7]] = large
        check_route(l.cuda(), top, bias=b.cuda(), score=score, groups=groups, top_groups=top_groups)
    every = torch.full((E,), math.nan, device="cuda")
    w, e, off, tok, slots = run_route(l.cuda(), top, score=score, bias=every, groups=groups,
                                      top_groups=top_groups)
    assert (e == -1).all() and (w == 0).all() and (off == 0).all() and (slots == -1).all()


def scores64(row, score):
    return torch.softmax(row.double(), 0) if score == "softmax" else torch.sigmoid(row.double())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 5, 16])
@pytest.mark.parametrize("E", [32, 200])
def test_route_close_scores(score, top, E):
    """Keys a few 1e-11 apart and not equal, closer than the integer keys tell."""
    row = torch.randn(E, generator=gen(35))
    step = 2e-3 if score == "softmax" else 2e-4
    row[1::2] = row[0::2] + step * (1 + torch.arange(E // 2) / E)
    s, bias = scores64(row, score), torch.zeros(E)
    # (one unit of the last place on from the nearest: never exactly equal)
    bias[1::2] = torch.nextafter((s[0::2] - s[1::2]).float(), torch.zeros(()))
    keys = s + bias.double()
    gap = (keys[0::2] - keys[1::2]).abs()
    # biases below 2^-9 are rounded by less than 2^-34; two sums of a softmax in 64
    # bits differ by a few 1e-16
    assert float(bias.abs().max()) < 2.0 ** -9 and float(gap.max()) < 2.0 ** -30
    assert float(gap.min()) > 2e-15
    check_route(row.expand(70, E).contiguous().cuda(), top, bias=bias.cuda(), score=score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top_groups", [1, 2, 3, 5, 7])
def test_route_close_group_sums(score, top_groups):
    """Groups in pairs whose sums of two keys are a few 1e-11 apart and not equal."""
    E, groups, top = 32, 8, 3
    row = torch.randn(groups, E // groups, generator=gen(36))
    row[1::2] = row[0::2] + 1e-4 * torch.rand(groups // 2, E // groups, generator=gen(37))
    row = row.reshape(E)
    s = scores64(row, score).view(groups, -1)
    two = s.topk(2, 1)
    bias = torch.zeros(groups, E // groups)
    for p in range(1, groups, 2):
        bias[p, two.indices[p, 0]] = float(two.values[p - 1].sum() - two.values[p].sum())
    sums = (s + bias.double()).topk(2, 1).values.sum(1)
    gap = (sums[0::2] - sums[1::2]).abs()
    assert float(gap.max()) < 2.0 ** -30 and float(gap.min()) > 2e-15
    check_route(row.expand(70, E).contiguous().cuda(), top, bias=bias.view(E).cuda(), score=score,
                groups=groups, top_groups=top_groups)


@pytest.mark.parametrize("m,E,top", [(32768, 24, 3), (32769, 24, 3), (70001, 100, 5), (33000, 700, 2)])
def test_route_plan_of_many_tokens(m, E, top):
    """Around and beyond 512 workgroups, where the counts are summed apart."""
    logits = torch.randn(m, E, generator=gen(38))
    logits[torch.rand(m, generator=gen(39)) < 0.05] = -math.inf
    logits[5, 1:] = -math.inf
    w, e, off, tok, slots = run_route(logits.cuda(), top)
    best = logits.cuda().sort(dim=1, descending=True, stable=True)
    live = best.values[:, :top] > -math.inf
    want = best.indices[:, :top].masked_fill(~live, -1).int()
    assert torch.equal(e, want)
    p = torch.softmax(best.values[:, :top].double(), 1).masked_fill(~live, 0)
    assert ((w.double() - p).abs() <= p * (2.0 ** -24 + 1e-12) + 1e-38).all()
    flat = want.flatten().long()
    rows = int((flat >= 0).sum())
    order = flat.masked_fill(flat < 0, E).sort(dim=0, stable=True).indices[:rows]
    place = torch.full((m * top,), -1, dtype=torch.int32, device="cuda")
    place[order] = torch.arange(rows, dtype=torch.int32, device="cuda")
    assert torch.equal(slots.flatten(), place)
    assert torch.equal(tok[:rows], (order // top).int()) and (tok[rows:] == -7).all()
    count = torch.bincount(flat[flat >= 0], minlength=E)
    assert off[0] == 0 and torch.equal(off[1:].long(), count.cumsum(0))


def test_route_no_tokens_and_padded_rows():
    E, top = 12, 3
    w, e, off, tok, slots = run_route(torch.zeros(0, E, device="cuda"), top)
    assert off.tolist() == [0] * (E + 1)
    big = torch.randn(300, 40, generator=gen(11)).cuda()
    check_route(big[:, 5:17], top)            # rows of a wider tensor


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("E,top", [(1, 1), (8, 2), (64, 6), (100, 8), (200, 4), (1000, 32)])
def test_route_backward(dtype, score, renorm, E, top):
    m, scale = 37, 1.7
    g = gen(12)
    l = (torch.randn(m, E, generator=g) * 2).to(dtype)
    e = torch.stack([torch.randperm(E, generator=g)[:top] for _ in range(m)]).int()
    if E > top:
        l[2, :] = l[2, :].masked_fill(torch.arange(E) >= E - 2, -math.inf)
        e[2] = torch.arange(top)
        e[3, top // 2:] = -1
    e[4] = -1
    dw = torch.randn(m, top, generator=g)
    out = Guarded(m, E, dtype, pad=3)
    pg.route_backward(dw.cuda(), l.cuda(), e.cuda(), out.t, score=score, renorm=renorm, scale=scale)
    x = l.double().requires_grad_(True)
    s = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
    live = (e >= 0).double()
    p = s.gather(1, e.clamp(min=0).long()) * live
    if renorm:
        p = p / (p.sum(1, keepdim=True) + (live.sum(1, keepdim=True) == 0))
    ((p * scale * dw.double()).sum()).backward()
    want = x.grad
    # fp32 scores (expf to 2 units, sums of E terms) against cancelling terms
    # no larger than scale * sum |dw|
    bound = half_step(dtype) * want.abs() + (E + top + 32) * 2.0 ** -24 * scale * \
        (s.detach() * dw.abs().sum(1, keepdim=True).double() + dw.abs().max(1, keepdim=True)[0])
    assert ((out.t.double().cpu() - want).abs() <= bound + 1e-7).all()
    out.check("dlogits")


def sigmoid_renorm_weights(x):
    """Sigmoids over their sum in 64 bits, of logits of any size."""
    low = x.clamp(max=0)
    p = torch.exp(low - low.amax(1, keepdim=True)) / (1 + torch.exp(-x.abs()))
    return p / p.sum(1, keepdim=True)


LOW = [[-100.0, -101, -102, -103], [-300, -301, -302, -310], [-89, -200, -95, -90],
       [-5, -120, -7, -6], [-20, 90, -100, 2], [-1000, -1000, -1001, -1004]]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("top", [2, 3])
def test_route_backward_of_low_sigmoids(dtype, top):
    """Renormalised sigmoids of logits far below -88, where exp(-x) is infinite in 32
    bits: the weights depend on the logits like a softmax."""
    l = torch.tensor(LOW).to(dtype)
    e = torch.tensor([[0, 1, 3], [2, 1, 0], [0, 3, 2], [1, 0, 3], [2, 0, 1], [1, 0, 2]])[:, :top]
    dw = torch.tensor([[1.0, -2, 0.5], [0.5, 3, -1], [1, 1.5, 2], [3, -1, 1], [-1, 2, 1], [1, -1, 0.25]])
    dw = dw[:, :top].contiguous()
    out = torch.empty(l.shape, dtype=dtype, device="cuda")
    pg.route_backward(dw.cuda(), l.cuda(), e.int().contiguous().cuda(), out, score="sigmoid")
    x = l.double()
    px = x.gather(1, e)
    r = sigmoid_renorm_weights(px)
    inner = dw.double() - (r * dw.double()).sum(1, keepdim=True)
    want = torch.zeros_like(x).scatter_(1, e, r * inner * torch.sigmoid(-px))
    # r to 12 units of 2^-24 (two exps of 3, sums, divisions) and the difference's
    # rounding in the exponent, |x| exp(x) < 0.37 of one; the same again for inner
    mag = r * (dw.double().abs() + (r * dw.double().abs()).sum(1, keepdim=True))
    bound = torch.zeros_like(x).scatter_(1, e, mag * 40 * 2.0 ** -24)
    bound = bound + want.abs() * half_step(dtype) + torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    assert ((out.double().cpu() - want).abs() <= bound).all()
    assert (out[0] != 0).sum() == top


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("top", [1, 2, 4])
def test_route_weights_of_low_sigmoids(dtype, top):
    """Renormalised sigmoids that are 0 in 64 bits still have their ratios."""
    l = torch.tensor(LOW + [[-701.0, -700, -702, -703], [-9000, -9001, -8990, -20000],
                            [-math.inf, -3000, -3001, -math.inf], [-2e4, -6e4, -5e4, -4e4],
                            [-math.inf, -math.inf, -math.inf, -math.inf]]).to(dtype)
    w, e, off, tok, slots = run_route(l.cuda(), top, score="sigmoid")
    we = route64(l.float(), LOWEST[dtype], top, score="sigmoid")[0]
    assert torch.equal(e.cpu(), we)
    live = we >= 0
    x = l.double().gather(1, we.clamp(min=0).long()).masked_fill(~live, -1e300)
    want = sigmoid_renorm_weights(x).masked_fill(~live, 0)
    assert ((w.double().cpu() - want).abs() <= want * (2.0 ** -24 + 1e-12) + 1e-38).all()


@pytest.mark.parametrize("dtype", [F32, BF16], ids=ids)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("top", [1, 2, 4])
def test_route_of_the_largest_logits(dtype, score, top):
    """Finite logits up to the type's largest keep their order, +inf before them."""
    big = torch.finfo(dtype).max
    l = torch.tensor([[1.0, 3.1e38, 3.3e38, 0], [3.05e38, 0, math.inf, 3.3e38],
                      [-3.3e38, big, 3.2e38, -1], [-3.3e38, -3.1e38, -3.2e38, -math.inf],
                      [3.1e38, 3.1e38, 3.2e38, math.nan], [-3.3e38, 3.3e38, -big, 5]]).to(dtype)
    ref = l.float().masked_fill(l.isnan(), -math.inf)
    w, e, off, tok, slots = run_route(l.cuda(), top, score=score, renorm=False)
    we, ww = route64(ref, LOWEST[dtype], top, score=score, renorm=False)
    assert torch.equal(e.cpu(), we)
    assert ((w.double().cpu() - ww).abs() <= ww * (2.0 ** -24 + 1e-12) + 1e-38).all()
    # with gradients of 1 the renormalised weights' is 0; otherwise p (1 - p) of the
    # sigmoid or p (1 - the chosen ones' sum) of the softmax, to 40 units of 2^-24
    x = ref.double().clamp(max=torch.finfo(F32).max)
    p = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
    chosen = torch.zeros_like(p).scatter_(1, we.clamp(min=0).long(), 1.0) * (ref > LOWEST[dtype])
    rest = 1 - (p * chosen).sum(1, keepdim=True) if score == "softmax" else 1 - p
    mag = chosen * p * (1 - p) if score == "sigmoid" else p * rest.abs() + p * (1 - p)
    d = torch.empty_like(l, device="cuda")
    for renorm in (False, True):
        pg.route_backward(torch.ones(6, top, device="cuda"), l.cuda(), e, d, score=score,
                          renorm=renorm)
        if renorm:
            want = torch.zeros_like(p)
        elif score == "sigmoid":
            want = chosen * p * (1 - p)
        else:
            want = p * (chosen - (p * chosen).sum(1, keepdim=True))
        bound = half_step(dtype) * want.abs() + 40 * 2.0 ** -24 * mag
        assert ((d.double().cpu() - want).abs() <= bound).all()


# ---- the experts' products ---------------------------------------------------------

def random_plan(g, m, top, E, drop=0.1, empty=()):
    allowed = [x for x in range(E) if x not in empty]
    e = torch.stack([torch.tensor(allowed)[torch.randperm(len(allowed), generator=g)[:top]]
                     for _ in range(m)]).int()
    e[torch.rand(m, generator=g) < drop] = -1
    o, rows, s = plan64(e, E)
    tok = torch.full((m * top,), -1, dtype=torch.int32)
    tok[:len(rows)] = torch.tensor(rows, dtype=torch.int32)
    return e, torch.tensor(o, dtype=torch.int32).cuda(), tok.cuda(), \
        torch.tensor(s, dtype=torch.int32).cuda()


EXPERT_SHAPES = [  # m, top, E, n, k
    (1, 1, 1, 8, 8), (1, 2, 8, 64, 64), (16, 4, 16, 80, 72), (40, 3, 5, 130, 65),
    (100, 2, 3, 136, 264), (300, 4, 6, 64, 40), (90, 8, 70, 33, 96), (700, 2, 4, 264, 128),
    (300, 2, 3, 134, 262)]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("shape", EXPERT_SHAPES, ids=str)
@pytest.mark.parametrize("gather", [True, False])
def test_expert_linear_exact_integers(dtype, order, shape, gather):
    m, top, E, n, k = shape
    g = gen(13)
    _, off, tok, _ = random_plan(g, m, top, E, empty=(1,) if E - 1 >= top and E > 1 else ())
    R = m * top
    X = Guarded(m if gather else R, k, dtype, pad=8, data=ints(g, m if gather else R, k).to(dtype))
    W = weight(g, (E,), k, n, order, dtype, integer=True)
    bias = ints(g, E, n).to(dtype).cuda()
    Y, Z = Guarded(R, n, F32, pad=1), Guarded(R, n, dtype)
    pg.expert_linear(X.t, W, Y.t, off, tokens=tok if gather else None, bias=bias, act="relu", Z=Z.t)
    o = off.tolist()
    x, w = X.t.double().cpu(), W.double().cpu()
    for e in range(E):
        r = torch.arange(o[e], o[e + 1])
        src = tok.cpu()[r].long() if gather else r
        z = x[src] @ w[e] + bias[e].double().cpu()
        assert torch.equal(Y.t.double().cpu()[r], z.clamp(min=0))
        assert torch.equal(Z.t.cpu()[r], z.to(dtype))
    Y.check("Y", rows=o[-1])
    Z.check("Z", rows=o[-1])


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("shape", EXPERT_SHAPES, ids=str)
@pytest.mark.parametrize("gather", [True, False])
def test_expert_linear_backward_exact_integers(dtype, order, shape, gather):
    m, top, E, n, k = shape
    g = gen(14)
    _, off, tok, _ = random_plan(g, m, top, E, empty=(1,) if E - 1 >= top and E > 1 else ())
    R, xr = m * top, m if gather else m * top
    X = ints(g, xr, k, hi=1).to(dtype).cuda()
    dY = ints(g, R, n, hi=1).to(dtype).cuda()
    Z = ints(g, R, n).to(dtype).cuda()
    o = off.tolist()
    dY[o[-1]:] = math.nan                            # rows behind the last are not read
    Z[o[-1]:] = math.nan
    W = weight(g, (E,), k, n, order, dtype, integer=True)
    dX = Guarded(R, k, dtype, pad=8)
    dW = torch.full_like(W, math.nan, dtype=F32)
    db = torch.full((E, n), math.nan, device="cuda")
    ws = space(pg.expert_linear_backward_workspace(R, n, k, E, dtype, "relu"))
    pg.expert_linear_backward(dY, X, W, off, tokens=tok if gather else None, Z=Z, act="relu",
                              dX=dX.t, dW=dW, dbias=db, ws=ws)
    for e in range(E):
        r = torch.arange(o[e], o[e + 1])
        src = tok.cpu()[r].long() if gather else r
        dz = dY.double().cpu()[r] * (Z.double().cpu()[r] > 0)
        assert torch.equal(dX.t.cpu()[r], (dz @ W[e].double().cpu().t()).to(dtype))
        assert torch.equal(dW[e].double().cpu(), X.double().cpu()[src].t() @ dz)
        assert torch.equal(db[e].double().cpu(), dz.sum(0))
    dX.check("dX", rows=o[-1])


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("bounds", [[0, 0, 4500, 4501, 6000], [0, 1500, 3000, 4500, 6000],
                                    [0, 6000, 6000, 6000, 6000], [0, 0, 0, 0, 0],
                                    [0, 63, 64, 65, 321]], ids=str)
@pytest.mark.parametrize("n,k", [(72, 40), (33, 70)])
def test_expert_gradients_over_long_rows(dtype, order, bounds, n, k):
    """Few tiles and many rows: each expert's rows are shared by workgroups."""
    R, E = 6000, 4
    g = gen(24)
    X, dY = ints(g, R, k, hi=1).to(dtype).cuda(), ints(g, R, n, hi=1).to(dtype).cuda()
    tok = torch.randperm(R, generator=g).int()
    off = torch.tensor(bounds, dtype=torch.int32, device="cuda")
    rows, cols = (k, n) if order == "kn" else (n, k)
    dW = torch.full((E, rows, cols), math.nan, device="cuda")
    dW = dW if order == "kn" else dW.transpose(1, 2)
    db = torch.full((E, n), math.nan, device="cuda")
    size = pg.expert_linear_backward_workspace(R, n, k, E, dtype)
    assert size > E * n * k * 4                  # the plan has room for partial sums
    W = weight(g, (E,), k, n, order, dtype, integer=True)
    pg.expert_linear_backward(dY, X, W, off, tokens=tok.cuda(), dW=dW, dbias=db, ws=space(size))
    x, dy = X.double().cpu()[tok.long()], dY.double().cpu()
    for e in range(E):
        s = slice(bounds[e], bounds[e + 1])
        assert torch.equal(dW[e].double().cpu(), x[s].t() @ dy[s])
        assert torch.equal(db[e].double().cpu(), dy[s].sum(0))


@pytest.mark.parametrize("gather", [True, False])
def test_expert_gradients_alone(gather):
    """Each gradient without what only the others read."""
    m, top, E, n, k = 30, 2, 5, 24, 40
    g = gen(34)
    _, off, tok, _ = random_plan(g, m, top, E)
    R, o = m * top, off.tolist()
    X, dY = ints(g, m if gather else R, k).cuda(), ints(g, R, n).cuda()
    W = weight(g, (E,), k, n, "nk", F32, integer=True)
    tokens = tok if gather else None
    ws = space(pg.expert_linear_backward_workspace(R, n, k, E, F32))
    dX, dW = Guarded(R, k, F32), torch.full((E, k, n), 9.0, device="cuda")
    db = torch.full((E, n), 9.0, device="cuda")
    pg.expert_linear_backward(dY, None, W, off, tokens=tokens, dX=dX.t, ws=ws)
    pg.expert_linear_backward(dY, X, None, off, tokens=tokens, dW=dW, ws=ws)
    pg.expert_linear_backward(dY, None, None, off, tokens=tokens, dbias=db, ws=ws)
    src = tok.long() if gather else torch.arange(R, device="cuda")
    for e in range(E):
        r = slice(o[e], o[e + 1])
        assert torch.equal(dX.t[r], dY[r] @ W[e].t())
        assert torch.equal(dW[e], X[src[r]].t() @ dY[r])
        assert torch.equal(db[e], dY[r].sum(0))
    dX.check("dX", rows=o[-1])


def test_zero_inner_size_in_tiles():
    bias = torch.arange(130.0, device="cuda")
    Y = torch.full((70, 130), 9.0, device="cuda")
    pg.linear(torch.zeros(70, 0, device="cuda"), torch.zeros(0, 130, device="cuda"), Y, bias=bias)
    assert torch.equal(Y, bias.expand(70, 130))
    dX = torch.full((70, 5), 9.0, device="cuda")
    pg.linear_backward(torch.zeros(70, 0, device="cuda"), None, torch.zeros(5, 0, device="cuda"),
                       dX=dX, ws=space(1 << 20))
    assert (dX == 0).all()


def test_expert_linear_skewed_and_large():
    """All rows on one expert of many, with the large tiles and the few-rows
    kernel's loop over row blocks."""
    g = gen(15)
    for m, E, n, k, dtype in ((600, 64, 64, 64, BF16), (60, 8, 512, 264, F16), (3000, 4, 1032, 72, BF16)):
        off = torch.zeros(E + 1, dtype=torch.int32)
        off[E // 2 + 1:] = m
        X = ints(g, m, k).to(dtype).cuda()
        W = weight(g, (E,), k, n, "nk", dtype, integer=True)
        Y = torch.empty(m, n, device="cuda")
        pg.expert_linear(X, W, Y, off.cuda())
        assert torch.equal(Y.double(), X.double() @ W[E // 2].double())


@pytest.mark.parametrize("dtype,E,R", [(BF16, 384, 24576), (F16, 1024, 33000), (F32, 300, 30000)],
                         ids=str)
def test_many_experts_with_many_columns(dtype, E, R):
    """Hundreds of experts with tens of tiles each, forwards and backwards."""
    n, k = 4096, 64
    g = gen(30)
    cut = torch.randint(0, R + 1, (E - 1,), generator=g).sort()[0].tolist()
    o = [0] + cut + [R]
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    X, D = ints(g, R, k, hi=1).to(dtype).cuda(), ints(g, R, k, hi=1).to(dtype).cuda()
    W = weight(g, (E,), k, n, "kn", dtype, integer=True)
    Y = torch.full((R, n), 9.0, dtype=dtype, device="cuda")
    pg.expert_linear(X, W, Y, off)
    dX = torch.full((R, n), 9.0, dtype=dtype, device="cuda")
    dW = torch.full((E, n, k), 9.0, device="cuda")
    ws = space(pg.expert_linear_backward_workspace(R, k, n, E, dtype))
    pg.expert_linear_backward(D, Y, W.transpose(1, 2), off, dX=dX, dW=dW, ws=ws)
    for e in range(E):
        r = slice(o[e], o[e + 1])
        y = X[r].double() @ W[e].double()          # sums of 64 terms up to 3: exact in 16 bits too
        assert torch.equal(Y[r].double(), y)
        assert torch.equal(dX[r].double(), D[r].double() @ W[e].double())
        assert torch.equal(dW[e].double(), y.t() @ D[r].double())


def test_expert_linear_bad_plans_stay_inside():
    """Bounds and tokens outside the buffers are clamped."""
    g = gen(16)
    m, E, n, k = 20, 3, 24, 16
    X, W = ints(g, m, k).cuda(), weight(g, (E,), k, n, "kn", F32, integer=True)
    Y = Guarded(m, n, F32)
    off = torch.tensor([-5, 8, 4, 1000], dtype=torch.int32, device="cuda")
    tok = torch.tensor([-1, 1 << 30] + list(range(18)), dtype=torch.int32, device="cuda")
    pg.expert_linear(X, W, Y.t, off, tokens=tok)
    Y.check("Y")
    assert torch.equal(Y.t[0], X[0] @ W[0]) and torch.equal(Y.t[1], X[m - 1] @ W[0])
    assert torch.equal(Y.t[2:4], X[:2] @ W[0])


# ---- rows back to their tokens -------------------------------------------------------

@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("m,top,n", [(1, 1, 1), (5, 3, 17), (64, 8, 64), (33, 4, 520), (9, 32, 2056)])
def test_combine_and_gradients(dtype, m, top, n):
    g = gen(17)
    E = 40
    _, off, tok, slots = random_plan(g, m, top, E, drop=0.2)
    R = m * top
    Y = torch.randn(R, n, generator=g).to(dtype).cuda()
    Y[int(off[-1]):] = math.nan
    w, res = torch.randn(m, top, generator=g).cuda(), torch.randn(m, n, generator=g).to(dtype)
    dout = torch.randn(m, n, generator=g).to(dtype).cuda()
    out = Guarded(m, n, dtype, pad=3, data=res)
    pg.combine(Y, slots, out.t, weights=w, residual=out.t)
    s, live = slots.cpu().long(), (slots >= 0).cpu()
    rows = Y.double().cpu()[s.clamp(min=0)].masked_fill(~live[:, :, None], 0)
    terms = rows * w.double().cpu()[:, :, None]
    want = terms.sum(1) + res.double()
    mag = terms.abs().sum(1) + res.double().abs()
    h = half_step(dtype)
    bound = h * want.abs() + (top + 3) * 2.0 ** -24 * mag * (1 + h)
    assert ((out.t.double().cpu() - want).abs() <= bound + 1e-9).all()
    out.check("out")
    plain = torch.empty(m, n, dtype=dtype, device="cuda")
    pg.combine(Y, slots, plain)
    want = rows.sum(1)
    bound = h * want.abs() + (top + 3) * 2.0 ** -24 * rows.abs().sum(1) * (1 + h)
    assert ((plain.double().cpu() - want).abs() <= bound + 1e-9).all()

    dY = Guarded(R, n, dtype, pad=8)
    dw = torch.full((m, top), math.nan, device="cuda")
    pg.combine_backward(dout, Y, slots, w, dY=dY.t, dweights=dw)
    d = dout.double().cpu()
    # below the type's smallest normal value the step is fixed at tiny * eps
    # (fp16: 2^-24), so half a step is this much whatever the value
    flat = torch.finfo(dtype).tiny * torch.finfo(dtype).eps / 2
    for t in range(m):
        for j in range(top):
            if live[t, j]:
                want = float(w[t, j]) * d[t]
                got = dY.t[s[t, j]].double().cpu()
                assert ((got - want).abs() <= (h + 2.0 ** -23) * want.abs() + flat).all()
                dot = (d[t] * rows[t, j])
                assert abs(float(dw[t, j]) - float(dot.sum())) <= (n + 2) * 2.0 ** -24 * \
                    float(dot.abs().sum()) + 1e-30
            else:
                assert float(dw[t, j]) == 0
    dY.check("dY", rows=int(off[-1]))


# ---- together, streams, graphs ----------------------------------------------------------

def moe_forward_backward(X, Wr, W1, W2, dout, top):
    """A routed pair of products and all its gradients, as a model runs it."""
    m, h = X.shape
    E, _, f = W1.shape
    T, new = X.dtype, lambda *s, d=X.dtype: torch.empty(*s, dtype=d, device="cuda")
    i32 = torch.int32
    s = {}
    s["logits"] = pg.linear(X, Wr, new(m, E, d=F32))
    s["w"], s["e"], s["slots"] = new(m, top, d=F32), new(m, top, d=i32), new(m, top, d=i32)
    s["off"], s["tok"] = new(E + 1, d=i32), new(m * top, d=i32)
    pg.route(s["logits"], s["w"], s["e"], s["off"], s["tok"], s["slots"],
             ws=space(pg.route_workspace(m, E, top)))
    R = m * top
    s["Z"], s["H"], s["Y"] = new(R, f), new(R, f), new(R, h)
    pg.expert_linear(X, W1, s["H"], s["off"], tokens=s["tok"], act="silu", Z=s["Z"])
    pg.expert_linear(s["H"], W2, s["Y"], s["off"])
    s["out"] = pg.combine(s["Y"], s["slots"], new(m, h), weights=s["w"], residual=X)
    # gradients
    s["dY"], s["dw"] = new(R, h), new(m, top, d=F32)
    pg.combine_backward(dout, s["Y"], s["slots"], s["w"], dY=s["dY"], dweights=s["dw"])
    s["dH"], s["dW2"] = new(R, f), torch.empty_like(W2)
    size = max(pg.expert_linear_backward_workspace(R, h, f, E, T),
               pg.expert_linear_backward_workspace(R, f, h, E, T, "silu"),
               pg.linear_backward_workspace(m, E, h, T))
    ws = space(size)
    pg.expert_linear_backward(s["dY"], s["H"], W2, s["off"], dX=s["dH"], dW=s["dW2"], ws=ws)
    s["dXr"], s["dW1"] = new(R, h), torch.empty_like(W1)
    pg.expert_linear_backward(s["dH"], X, W1, s["off"], tokens=s["tok"], Z=s["Z"], act="silu",
                              dX=s["dXr"], dW=s["dW1"], ws=ws)
    s["dlogits"] = pg.route_backward(s["dw"], s["logits"], s["e"], new(m, E, d=F32))
    s["dl"] = s["dlogits"].to(T)
    s["dXl"], s["dWr"] = new(m, h), torch.empty_like(Wr)
    pg.linear_backward(s["dl"], X, Wr, dX=s["dXl"], dW=s["dWr"], ws=ws)
    s["dX"] = pg.combine(s["dXr"], s["slots"], new(m, h), residual=s["dXl"])
    s["dX"] = s["dX"] + dout
    return s


def test_routed_layer_matches_autograd_in_64_bits():
    """The whole chain in fp32 against autograd of the same layer in 64 bits."""
    m, h, f, E, top = 90, 48, 72, 8, 2
    g = gen(18)
    X, dout = torch.randn(m, h, generator=g).cuda(), torch.randn(m, h, generator=g).cuda()
    Wr = (torch.randn(E, h, generator=g) * h ** -0.5).cuda().t()
    W1 = (torch.randn(E, f, h, generator=g) * h ** -0.5).cuda().transpose(1, 2)
    W2 = (torch.randn(E, f, h, generator=g) * f ** -0.5).cuda()
    s = moe_forward_backward(X, Wr, W1, W2, dout, top)
    leaves = [t.double().cpu().detach().requires_grad_(True) for t in (X, Wr, W1, W2)]
    x, wr, w1, w2 = leaves
    p = torch.softmax(x @ wr, 1)
    e = s["e"].cpu().long()
    assert torch.equal(p.topk(top, 1).indices, e)
    w = p.gather(1, e)
    w = w / w.sum(1, keepdim=True)
    out = x
    for j in range(top):
        z = torch.bmm(x[:, None], w1[e[:, j]])[:, 0]
        out = out + w[:, j:j + 1] * torch.bmm(act64(z, "silu")[:, None], w2[e[:, j]])[:, 0]
    (out * dout.double().cpu()).sum().backward()
    for name, got, want in (("out", s["out"], out.detach()), ("dX", s["dX"], x.grad),
                            ("dWr", s["dWr"], wr.grad), ("dW1", s["dW1"], w1.grad),
                            ("dW2", s["dW2"], w2.grad)):
        # seven fp32 stages of at most 90-term sums of values of order one: relative
        # to the largest entry (7 * 92 + 32) 2^-24 = 4e-5
        err = (got.double().cpu() - want).abs().max() / want.abs().max()
        assert err < 4e-5, (name, float(err))


@pytest.mark.parametrize("dtype", [BF16, F32], ids=ids)
def test_routed_layer_captured_and_replayed(dtype):
    """One graph of the chain, replayed with eager work in between; every
    replay equals the eager result of its inputs."""
    m, h, f, E, top = 130, 64, 96, 8, 2
    g = gen(19)

    def inputs():
        return [torch.randn(*s, generator=g).to(dtype).cuda() for s in
                ((m, h), (E, h), (E, f, h), (E, f, h), (m, h))]
    hold = inputs()

    def run():
        X, Wr, W1, W2, dout = hold
        return moe_forward_backward(X, Wr.t(), W1.transpose(1, 2), W2, dout, top)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    for _ in range(4):
        for t, v in zip(hold, inputs()):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        want = run()
        rows = int(want["off"][-1])
        for name in ("out", "dX", "dWr", "dW1", "dW2", "w", "e", "off", "slots"):
            assert torch.equal(captured[name], want[name]), name
        assert torch.equal(captured["tok"][:rows], want["tok"][:rows])


def test_streams_and_repeats():
    """Two calls at once on their own streams; identical inputs, identical bits."""
    g = gen(20)
    X = torch.randn(300, 520, generator=g).to(BF16).cuda()
    W = weight(g, (), 520, 264, "nk", BF16)
    Y = torch.empty(300, 264, dtype=BF16, device="cuda")
    ws = space(pg.linear_workspace(300, 264, 520, BF16))
    pg.linear(X, W, Y, ws=ws, act="gelu")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(Y) for _ in streams]
    spaces = [space(pg.linear_workspace(300, 264, 520, BF16)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o, w in zip(streams, outs, spaces):
            pg.linear(X, W, o, ws=w, act="gelu", stream=s)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, Y)


def test_offsets_beyond_32_bits():
    """Rows whose byte offsets pass 2^32 (a gathered row far into X, and Y)."""
    rows, k = (1 << 31) // 4096 + 70, 4096            # 2^31 elements and more, bf16
    X = torch.zeros(rows, k, dtype=BF16, device="cuda")
    X[-64:, 3] = torch.arange(64, dtype=BF16, device="cuda")
    W = torch.zeros(1, 16, k, dtype=BF16, device="cuda")
    W[:, :, 3] = 1
    tok = torch.arange(rows - 64, rows, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    Y = torch.empty(64, 16, device="cuda")
    pg.expert_linear(X, W.transpose(1, 2), Y, off, tokens=tok)
    assert torch.equal(Y[:, 0].cpu(), torch.arange(64.0))
    del X
    # the result itself that long: n = 16, ld = 2^27, 40 rows
    buf = torch.zeros(39 * (1 << 27) // 2 + 16, dtype=BF16, device="cuda")
    Yl = buf.as_strided((40, 16), (1 << 26, 1))
    Xs, Ws = torch.ones(40, 8, dtype=BF16, device="cuda"), torch.ones(8, 16, dtype=BF16, device="cuda")
    pg.linear(Xs, Ws, Yl)
    assert (Yl == 8).all()


def test_combine_of_more_tokens_than_a_launch_takes():
    """2^24 tokens with a workgroup each, and 2^26 choices with a wave each."""
    m, n, rows = (1 << 24) + 5, 1032, 16
    g = gen(33)
    Y = ints(g, rows, n).to(BF16).cuda()
    slots = torch.randint(-1, rows, (m, 1), generator=g, dtype=torch.int32).cuda()
    out = torch.empty(m, n, dtype=BF16, device="cuda")
    pg.combine(Y, slots, out)
    padded = torch.cat([torch.zeros(1, n, dtype=BF16, device="cuda"), Y])
    for t0 in range(0, m, 1 << 20):
        want = padded[slots[t0:t0 + (1 << 20), 0].long() + 1]
        assert torch.equal(out[t0:t0 + (1 << 20)], want)
    del out, want
    m, top, n = (1 << 22) + 3, 16, 8
    live = torch.tensor([0, 1, m // 2, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, m - 2, m - 1])
    R = live.numel() * top
    slots = torch.full((m, top), -1, dtype=torch.int32)
    slots[live] = torch.randperm(R, generator=g).int().view(-1, top)
    slots = slots.cuda()
    dout, Y = ints(g, m, n).to(BF16).cuda(), ints(g, R, n).to(BF16).cuda()
    w = torch.full((m, top), 2.0, device="cuda")
    dY = torch.full((R, n), 9.0, dtype=BF16, device="cuda")
    dw = torch.full((m, top), 9.0, device="cuda")
    pg.combine_backward(dout, Y, slots, w, dY=dY, dweights=dw)
    assert int((dw != 0).any(1).sum()) <= live.numel()
    for t in live.tolist():
        r = slots[t].long()
        assert torch.equal(dY[r], (2 * dout[t]).expand(top, n))
        assert torch.equal(dw[t], Y[r].float() @ dout[t].float())


# ---- calls over everything the documentation allows -----------------------------------------

def spread(rng, hi):
    return int(round(math.exp(rng.uniform(0, math.log(hi)))))


def placed(rng, rows, cols, dtype, data=None):
    """Rows at a random stride, from a random element of the buffer on."""
    return Guarded(rows, cols, dtype, pad=rng.choice((0, 0, 1, 2, 3, 8, 13)),
                   shift=rng.choice((0, 0, 1, 2, 4, 5)), data=data)


def placed_weight(rng, g, experts, k, n, dtype):
    """Experts' weights (None: one) in a random order, at random strides."""
    order, pad = rng.choice(("kn", "nk")), rng.choice((0, 0, 1, 2, 8))
    rows, cols = (k, n) if order == "kn" else (n, k)
    E, gap = experts or 1, rng.choice((0, 0, 1, 8, 24))
    size = rows * (cols + pad) + gap
    buf = torch.full((E * size + 8,), math.nan, dtype=dtype, device="cuda")[rng.choice((0, 1, 2, 8)):]
    w = buf.as_strided((E, rows, cols), (size, cols + pad, 1))
    if g is not None:
        w.copy_(ints(g, E, rows, cols, hi=2).to(dtype))
    w = w if order == "kn" else w.transpose(1, 2)
    return w if experts else w[0]


def optional(rng, make):
    return make() if rng.random() < 0.6 else None


@pytest.mark.parametrize("seed", range(60))
def test_random_linear_calls(seed):
    """Random shapes, strides, alignments, orders, types and options; exact."""
    rng, g = random.Random(seed), gen(seed)
    dtype, out32 = rng.choice(TYPES), rng.random() < 0.4
    m, n, k = spread(rng, 600), spread(rng, 600), spread(rng, 900)
    out, act = F32 if out32 else dtype, rng.choice(("none", "relu"))
    X = placed(rng, m, k, dtype, ints(g, m, k, hi=1).to(dtype))
    W = placed_weight(rng, g, None, k, n, dtype)
    bias = optional(rng, lambda: ints(g, n).to(dtype).cuda())
    R = optional(rng, lambda: placed(rng, m, n, out, ints(g, m, n).to(out)))
    Y = R if R is not None and rng.random() < 0.5 else placed(rng, m, n, out)
    res = 0 if R is None else R.t.double().cpu()
    Z = optional(rng, lambda: placed(rng, m, n, dtype))
    ws = optional(rng, lambda: space(pg.linear_workspace(m, n, k, dtype)))
    pg.linear(X.t, W, Y.t, bias=bias, act=act, residual=R.t if R else None, Z=Z.t if Z else None, ws=ws)
    x, w = X.t.double().cpu(), W.double().cpu()
    z = x @ w + (0 if bias is None else bias.double().cpu())
    assert torch.equal(Y.t.cpu(), ((z.clamp(min=0) if act == "relu" else z) + res).to(out))
    Y.check("Y")
    if Z:
        assert torch.equal(Z.t.cpu(), z.to(dtype))
        Z.check("Z")
    # the gradients of the same layer
    dY = placed(rng, m, n, dtype, ints(g, m, n, hi=1).to(dtype))
    Zb = placed(rng, m, n, dtype, ints(g, m, n).to(dtype))
    dX = optional(rng, lambda: placed(rng, m, k, dtype))
    dW = optional(rng, lambda: placed_weight(rng, None, None, k, n, out))
    db = optional(rng, lambda: torch.full((n,), 9.0, dtype=out, device="cuda"))
    wsb = space(pg.linear_backward_workspace(m, n, k, dtype, act))
    pg.linear_backward(dY.t, X.t, W, Z=Zb.t if act == "relu" else None, act=act,
                       dX=dX.t if dX else None, dW=dW, dbias=db, ws=wsb)
    dz = dY.t.double().cpu()
    if act == "relu":
        dz = dz * (Zb.t.double().cpu() > 0)
    if dX:
        assert torch.equal(dX.t.cpu(), (dz @ w.t()).to(dtype))
        dX.check("dX")
    if dW is not None:
        assert torch.equal(dW.cpu(), (x.t() @ dz).to(out))
    if db is not None:
        assert torch.equal(db.cpu(), dz.sum(0).to(out))


@pytest.mark.parametrize("seed", range(60))
def test_random_expert_calls(seed):
    """The same over experts, of which some have no rows and one may have most."""
    rng, g = random.Random(1000 + seed), gen(1000 + seed)
    dtype, out32 = rng.choice(TYPES), rng.random() < 0.4
    E, R, n, k = spread(rng, 90), spread(rng, 1500), spread(rng, 400), spread(rng, 400)
    out, act = F32 if out32 else dtype, rng.choice(("none", "relu"))
    last = rng.randint(0, R)
    o = sorted(rng.choice((0, last, rng.randint(0, last))) for _ in range(E - 1))
    o = [rng.choice((0, 0, min(o + [last]))) if E > 1 else 0] + o + [last]
    off = torch.tensor(o, dtype=torch.int32, device="cuda")
    gather = rng.random() < 0.6
    m = spread(rng, 300) if gather else R + rng.randint(0, 5)
    tok = torch.randint(0, m, (R,), generator=g, dtype=torch.int32).cuda() if gather else None
    src = tok.cpu().long() if gather else torch.arange(R)
    X = placed(rng, m, k, dtype, ints(g, m, k, hi=1).to(dtype))
    W = placed_weight(rng, g, E, k, n, dtype)
    bias = optional(rng, lambda: ints(g, E, n).to(dtype).cuda())
    Y, Z = placed(rng, R, n, out), optional(rng, lambda: placed(rng, R, n, dtype))
    pg.expert_linear(X.t, W, Y.t, off, tokens=tok, bias=bias, act=act, Z=Z.t if Z else None)
    dY = placed(rng, R, n, dtype, ints(g, R, n, hi=1).to(dtype))
    Zb = placed(rng, R, n, dtype, ints(g, R, n).to(dtype))
    dX = optional(rng, lambda: placed(rng, R, k, dtype))
    dW = optional(rng, lambda: placed_weight(rng, None, E, k, n, out))
    db = optional(rng, lambda: torch.full((E, n), 9.0, dtype=out, device="cuda"))
    ws = space(pg.expert_linear_backward_workspace(R, n, k, E, dtype, act))
    pg.expert_linear_backward(dY.t, X.t, W, off, tokens=tok, Z=Zb.t if act == "relu" else None,
                              act=act, dX=dX.t if dX else None, dW=dW, dbias=db, ws=ws)
    x, w, d = X.t.double().cpu(), W.double().cpu(), dY.t.double().cpu()
    if act == "relu":
        d = d * (Zb.t.double().cpu() > 0)
    for e in range(E):
        r = slice(o[e], o[e + 1])
        z = x[src[r]] @ w[e] + (0 if bias is None else bias[e].double().cpu())
        assert torch.equal(Y.t[r].cpu(), (z.clamp(min=0) if act == "relu" else z).to(out))
        if Z:
            assert torch.equal(Z.t[r].cpu(), z.to(dtype))
        if dX:
            assert torch.equal(dX.t[r].cpu(), (d[r] @ w[e].t()).to(dtype))
        if dW is not None:
            assert torch.equal(dW[e].cpu(), (x[src[r]].t() @ d[r]).to(out))
        if db is not None:
            assert torch.equal(db[e].cpu(), d[r].sum(0).to(out))
    if o[0] == 0:
        for t in (Y, Z, dX):
            if t:
                t.check(rows=last)


@pytest.mark.parametrize("seed", range(40))
def test_random_combine_calls(seed):
    """Rows at random strides, slots that are used once, twice (forwards), or not."""
    rng, g = random.Random(2000 + seed), gen(2000 + seed)
    dtype, m, n, top = rng.choice(TYPES), spread(rng, 300), spread(rng, 3000), rng.randint(1, 8)
    rows = m * top + rng.randint(0, 9)
    Y = placed(rng, rows, n, dtype, ints(g, rows, n).to(dtype))
    slots = torch.randint(-2, rows + 2, (m, top), generator=g, dtype=torch.int32)
    w = optional(rng, lambda: ints(g, m, top))
    R = optional(rng, lambda: placed(rng, m, n, dtype, ints(g, m, n).to(dtype)))
    out = R if R is not None and rng.random() < 0.5 else placed(rng, m, n, dtype)
    want = 0 if R is None else R.t.double().cpu()
    pg.combine(Y.t, slots.cuda(), out.t, weights=None if w is None else w.cuda(),
               residual=R.t if R else None)
    live = (slots >= 0) & (slots < rows)
    f = live.double() * (1 if w is None else w.double())
    y = Y.t.double().cpu()[slots.long().clamp(0, rows - 1)]
    assert torch.equal(out.t.cpu(), ((y * f[:, :, None]).sum(1) + want).to(dtype))
    out.check("out")
    once = torch.full((m * top,), -1, dtype=torch.int32)
    used = torch.rand(m * top, generator=g) < 0.8
    once[used] = torch.randperm(rows, generator=g)[:int(used.sum())].int()
    once = once.view(m, top)
    dout = placed(rng, m, n, dtype, ints(g, m, n, hi=1).to(dtype))
    dY = optional(rng, lambda: placed(rng, rows, n, dtype))
    dw = optional(rng, lambda: torch.full((m, top), 9.0, device="cuda"))
    pg.combine_backward(dout.t, Y.t, once.cuda(), None if w is None else w.cuda(),
                        dY=dY.t if dY else None, dweights=dw)
    d, live = dout.t.double().cpu(), once >= 0
    if dY:
        f = torch.ones(m, top).double() if w is None else w.double()
        got = dY.t.cpu()[once.long().clamp(min=0)]
        assert torch.equal(got[live], (d[:, None] * f[:, :, None]).to(dtype)[live])
        rest = torch.ones(rows, dtype=torch.bool)
        rest[once[live].long()] = False
        assert dY.t.cpu()[rest].isnan().all()
        dY.check("dY")
    if dw is not None:
        y = Y.t.double().cpu()[once.long().clamp(min=0)]
        assert torch.equal(dw.double().cpu(), (d[:, None] * y).sum(2) * live)


@pytest.mark.parametrize("seed", range(60))
def test_random_route_calls(seed):
    """Random numbers of experts, groups and choices; logits that are close, far
    apart, equal or masked; biases of all sizes."""
    rng, g = random.Random(3000 + seed), gen(3000 + seed)
    dtype, score = rng.choice(TYPES), rng.choice(("softmax", "sigmoid"))
    groups = rng.choice((1, 1, 1, 2, 3, 5, 8, 13, 40, 64))
    E = groups * spread(rng, 1024 // groups)
    top_groups = rng.randint(1, groups)
    top = rng.randint(1, min(32, E // groups * top_groups))
    m = spread(rng, 150) if E < 100 else spread(rng, 20)
    l = torch.randn(m, E, generator=g) * rng.choice((0.01, 1, 1, 3, 10, 100))
    if rng.random() < 0.4:                        # equal logits
        l = (l * 2).round() / 2
    l = l.to(dtype)
    if rng.random() < 0.5:
        l[torch.rand(m, E, generator=g) < rng.choice((0.1, 0.9))] = rng.choice((-math.inf, LOWEST[dtype]))
    wide = torch.zeros(m, E + 3, dtype=dtype, device="cuda")
    wide[:, 1:E + 1] = l.cuda()
    bias = optional(rng, lambda: torch.randn(E, generator=g) * rng.choice((1e-6, 0.1, 1, 1e3)))
    kw = dict(score=score, groups=groups, top_groups=top_groups, renorm=rng.random() < 0.5,
              scale=rng.choice((1.0, 2.5)))
    check_route(wide[:, 1:E + 1], top, bias=None if bias is None else bias.cuda(), **kw)
