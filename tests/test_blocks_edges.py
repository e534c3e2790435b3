"""The block operators on the GPU where numbers leave their types' range, and in the kernels
that only wide or long calls take."""
import math

import pytest
import torch

import precision_gemm_02_amd as pg
from layer_util import Guarded, ints, weight

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]
ids = {F32: "f32", F16: "f16", BF16: "bf16"}.get
U = 2.0 ** -24
INF, NAN = math.inf, math.nan


def gen(seed):
    return torch.Generator().manual_seed(seed)


def space(n):
    return torch.full((n + 16,), 0x7F, dtype=torch.uint8, device="cuda")


# ---- pre-activations beyond their type -------------------------------------------------

@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("out", [F16, F32], ids=ids)
def test_gated_gradient_where_a_kept_pre_activation_overflows(act, out):
    """fp16: sums of -70000 in the gate, or of 70000 beside an inactive gate, give a finite
    result; Z keeps an infinity, and its gradients are 0."""
    X = torch.full((1, 1), 700.0, device="cuda").half()
    for gate, up in ((-100.0, 2.0), (-1.0, 100.0), (-1.0, -100.0), (-100.0, -100.0)):
        Wg, Wu = (torch.full((1, 8), w, device="cuda").half() for w in (gate, up))
        Y, Zg, Zu = (torch.empty(1, 8, device="cuda").half() for _ in range(3))
        pg.gated_linear(X, Wg, Wu, Y, act=act, Z_gate=Zg, Z_up=Zu)
        assert bool((Y == 0).all())
        assert bool((Zg.isinf() == (gate == -100)).all()) and bool((Zu.isinf() == (abs(up) == 100)).all())
        dX = torch.full((1, 1), NAN, device="cuda").half()
        dWg, dWu = (torch.full((1, 8), NAN, dtype=out, device="cuda") for _ in range(2))
        dbg, dbu = (torch.full((8,), NAN, dtype=out, device="cuda") for _ in range(2))
        pg.gated_linear_backward(torch.ones_like(Y), X, Wg, Wu, Zg, Zu, act=act, dX=dX, dW_gate=dWg,
                                 dW_up=dWu, dbias_gate=dbg, dbias_up=dbu,
                                 ws=space(pg.gated_linear_backward_workspace(1, 8, 1, F16)))
        for t in (dX, dWg, dWu, dbg, dbu):
            assert bool((t == 0).all()), (gate, up, t)


# (dY, Zg, Zu) -> (dZg, dZu) for an activation that is 0 with slope 0 far below 0, and the
# identity with slope 1 far above it; a factor of 0 makes a product 0 unless another is a NaN
FAR = [((1, -INF, 2), (0, 0)), ((1, -INF, INF), (0, 0)), ((1, -INF, -INF), (0, 0)),
       ((1, -1000, INF), (0, 0)), ((1, -1000, -INF), (0, 0)),
       ((0, INF, 2), (0, 0)), ((0, 1000, INF), (0, 0)), ((0, INF, -INF), (0, 0)),
       ((1, INF, 2), (2, INF)), ((-1, INF, 2), (-2, -INF)), ((1, 1000, INF), (INF, 1000)),
       ((1, 1000, -INF), (-INF, 1000)), ((2, INF, INF), (INF, INF)),
       ((NAN, -INF, 2), (NAN, NAN)), ((NAN, -1000, INF), (NAN, NAN)),
       ((1, NAN, 2), (NAN, NAN)), ((1, NAN, INF), (NAN, NAN)), ((0, NAN, INF), (NAN, NAN)),
       ((1, -1000, NAN), (NAN, 0)), ((1, -INF, NAN), (NAN, 0)), ((0, 1000, NAN), (NAN, 0)),
       ((3, 1000, 2), (6, 3000))]


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("rows,out32", [(1, True), (1, False), (40, True)])
def test_gated_slopes_far_out(act, dtype, rows, out32):
    """Each column's own bias gradients, of one row and of one among rows of zeros; where
    all of a call's products vanish, so do dX and dW."""
    n, k = len(FAR), 24
    out = F32 if out32 else dtype
    d, zg, zu = torch.zeros(rows, n), torch.ones(rows, n), torch.ones(rows, n)
    at = rows // 2
    d[at], zg[at], zu[at] = (torch.tensor([float(c[0][j]) for c in FAR]) for j in range(3))
    d, zg, zu = (t.to(dtype).cuda() for t in (d, zg, zu))
    want = [torch.tensor([float(c[1][j]) for c in FAR]).to(out) for j in range(2)]
    if act == "relu":             # (its slope is 1 where z > 0 and else 0, of a NaN too)
        want[0] = torch.where(zg[at].isnan().cpu() & d[at].isfinite().cpu(), torch.zeros(n, dtype=out), want[0])
    got = [torch.full((n,), 7.0, dtype=out, device="cuda") for _ in range(2)]
    ws = space(pg.gated_linear_backward_workspace(rows, n, k, dtype))
    pg.gated_linear_backward(d, None, None, None, zg, zu, act=act, dbias_gate=got[0], dbias_up=got[1], ws=ws)
    for g, w in zip(got, want):
        g = g.cpu()
        assert torch.equal(g.isnan(), w.isnan()), (g, w)
        assert torch.equal(g[~w.isnan()], w[~w.isnan()]), (g, w)
    none = [j for j, c in enumerate(FAR) if c[1] == (0, 0)]
    d, zg, zu = (t[:, none].contiguous() for t in (d, zg, zu))
    g = gen(1)
    X, Wg, Wu = (torch.randn(*s, generator=g).to(dtype).cuda()
                 for s in ((rows, k), (k, len(none)), (k, len(none))))
    dX, dWg, dWu = (torch.full_like(t, NAN) for t in (X, Wg, Wu))
    pg.gated_linear_backward(d, X, Wg, Wu, zg, zu, act=act, dX=dX, dW_gate=dWg, dW_up=dWu, ws=ws)
    for t in (dX, dWg, dWu):
        assert bool((t == 0).all())


# ---- the longest rows of 8 bits ----------------------------------------------------------

def x_at(t, at):
    return t.view(torch.uint8)[:, at].view(t.dtype).cpu().double()


@pytest.mark.parametrize("k", [(1 << 31) - 4096, (1 << 31) - 4097])
def test_linear_fp8_longest_rows(k):
    """The largest summed index, shared between workgroups and not: numbers in the first
    and last blocks of the splits and of the rows."""
    m, n = 2, 3
    X, W = (torch.zeros(r, k, dtype=torch.uint8, device="cuda") for r in (m, n))
    at = torch.cat([torch.arange(0, k, k // 61), torch.arange(k - 200, k)]).cuda()
    g = gen(3)
    x, w = (torch.randint(-4, 5, (r, len(at)), generator=g).float().to(torch.float8_e4m3fn).cuda()
            for r in (m, n))
    X[:, at], W[:, at] = x.view(torch.uint8), w.view(torch.uint8)
    X, W = X.view(torch.float8_e4m3fn), W.view(torch.float8_e4m3fn)
    at = at.unique()                         # (of a place named twice one number is left)
    want = x_at(X, at) @ x_at(W, at).t()
    one = torch.ones(1, 1, device="cuda")
    blocks = -(-k // 128)
    for out in (F32, BF16):
        for ws in (None, space(pg.linear_fp8_workspace(m, n, k))):
            Y = torch.full((m, n), NAN, dtype=out, device="cuda")
            pg.linear_fp8(X, one.expand(m, blocks), W.t(), one.expand(blocks, n), Y, ws=ws)
            assert torch.equal(Y.cpu(), want.to(out))


# ---- rows whose squares leave fp32 ---------------------------------------------------------

def norm64(x, eps):
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    return mean, rstd, (x - mean) * rstd


@pytest.mark.parametrize("dtype", [F32, BF16], ids=ids)
@pytest.mark.parametrize("n", [40, 128, 500, 900, 2000, 2999, 8000, 16000, 30001, 40000])
@pytest.mark.parametrize("eps,powers", [(1e-5, (0, 62, 64, 70, 100, 125, 3)), (0.0, (0, -50, -60, -80, -100, 70))])
def test_layer_norm_of_huge_and_tiny_rows(dtype, n, eps, powers):
    """The definition holds over the types' whole range, row by row, also where a row's sum
    of squares is infinite in fp32, or nothing."""
    g = gen(n)
    x = torch.randn(3 * len(powers), n, generator=g) + torch.randn(3 * len(powers), 1, generator=g)
    x *= torch.exp2(torch.tensor(powers, dtype=torch.float32)).repeat(3)[:, None]
    X = x.to(dtype).cuda()
    w, b = (torch.randn(n, generator=g).to(dtype).cuda() for _ in range(2))
    Y = torch.full_like(X, NAN)
    mean, rstd = (torch.full((X.shape[0],), NAN, device="cuda") for _ in range(2))
    pg.layer_norm(X, Y, weight=w, bias=b, eps=eps, mean=mean, rstd=rstd)
    x = X.double().cpu()
    mu, r, h = norm64(x, eps)
    # the statistics: a sum of n numbers of which a thread adds at most 64 one after the other,
    # its parts by halves (at most 26 steps): 90 u of their magnitude, that of what is left of the
    # mean once more; rstd 60 u and the mean's part squared.  Then x - mean, times rstd, times
    # weight, plus bias: a rounding each, and Y's own.
    mag, left = x.abs().mean(1, keepdim=True), (x - mu).abs().mean(1, keepdim=True)
    e_mean = 2 * U * mag + 92 * U * (left + 90 * U * mag)
    e_rstd = r * (60 * U) + r * (90 * U * mag * r) ** 2
    w, b = w.double().cpu(), b.double().cpu()
    e = ((x - mu).abs() * (3 * U * r + e_rstd) + r * (e_mean + 2 * U * (x.abs() + mu.abs()))) * w.abs()
    y = h * w + b
    e += 2 * U * ((h * w).abs() + y.abs() + b.abs())
    half = torch.finfo(dtype).eps / 2
    assert bool(((Y.double().cpu() - y).abs() <= e * (1 + half) + half * y.abs()).all())
    assert bool(((mean.double().cpu() - mu[:, 0]).abs() <= (e_mean + U * mu.abs())[:, 0]).all())
    assert bool(((rstd.double().cpu() - r[:, 0]).abs() <= (e_rstd + U * r)[:, 0]).all())


@pytest.mark.parametrize("dtype", [F32, BF16], ids=ids)
@pytest.mark.parametrize("n", [40, 500, 3000, 20000, 40000])
def test_layer_norm_of_the_largest_numbers(dtype, n):
    """Rows of one number, whose sum is infinite in fp32, beside an ordinary one, one with an
    infinity, and one that goes from end to end of the range."""
    top = torch.finfo(dtype).max
    X = torch.full((5, n), top, dtype=dtype, device="cuda")
    X[1] = torch.randn(n, generator=gen(1)).to(dtype)
    X[2, n // 2] = INF
    X[3] = -top
    X[4, : n // 2] = -top
    Y, alone = torch.full_like(X, NAN), torch.full_like(X[1:2], NAN)
    mean, rstd = (torch.full((5,), NAN, device="cuda") for _ in range(2))
    pg.layer_norm(X, Y, eps=0.25, mean=mean, rstd=rstd)
    pg.layer_norm(X[1:2], alone, eps=0.25)
    assert torch.equal(Y[1:2], alone)
    assert bool((Y[0] == 0).all()) and bool((Y[3] == 0).all()) and bool(Y[2].isnan().any())
    assert float(mean[0]) == top and float(mean[3]) == -top and float(rstd[0]) == 2 == float(rstd[3])
    # half the numbers each: the mean is 0, the spread the number itself
    assert float(mean[4]) == 0 and bool((Y[4].double().cpu().abs() - 1).abs().max() <= 4 * U)


# ---- few rows: wide products, long rows of 8 bits --------------------------------------------

E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
ids8 = {E4M3: "e4m3", E5M2: "e5m2"}.get
# columns that fill the chip with workgroups of twice the width, with and without a partly
# filled last one (test_blocks_plan_edges.py holds that these sizes take those kernels)
WIDE = [(8161, 1001), (8200, 1032), (8191, 72)]


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("order", ["kn", "nk"])
@pytest.mark.parametrize("m", [1, 16, 17, 32])
@pytest.mark.parametrize("n,k", WIDE)
def test_wide_gated_products_of_few_rows(dtype, order, m, n, k):
    """Whole numbers: exact sums and products."""
    g = gen(m + n + k)
    pad = n % 8
    X = Guarded(m, k, dtype, pad=pad, data=ints(g, m, k, hi=1).to(dtype))
    Wg, Wu = (weight(g, (), k, n, order, dtype, integer=True, pad=pad) for _ in range(2))
    bg, bu = (ints(g, n).to(dtype).cuda() for _ in range(2))
    Y, Zg, Zu = Guarded(m, n, F32, pad=pad), Guarded(m, n, dtype, pad=pad), Guarded(m, n, dtype, pad=pad)
    pg.gated_linear(X.t, Wg, Wu, Y.t, bias_gate=bg, bias_up=bu, act="relu", Z_gate=Zg.t, Z_up=Zu.t,
                    ws=space(pg.gated_linear_workspace(m, n, k, dtype)))
    x = X.t.double().cpu()
    zg, zu = (x @ w.double().cpu() + b.double().cpu() for w, b in ((Wg, bg), (Wu, bu)))
    assert torch.equal(Y.t.double().cpu(), zg.clamp(min=0) * zu)
    assert torch.equal(Zg.t.cpu(), zg.to(dtype)) and torch.equal(Zu.t.cpu(), zu.to(dtype))
    for t in (Y, Zg, Zu):
        t.check()
    Y = Guarded(m, n, dtype)
    pg.gated_linear(X.t, Wg, Wu, Y.t, act="none")
    want = (zg - bg.double().cpu()) * (zu - bu.double().cpu())
    assert torch.equal(Y.t.cpu(), want.to(dtype))
    Y.check()


def eights(g, r, c, dtype, pad):
    """Small whole numbers in 8 bits, NaN around their rows."""
    buf = torch.full((r, c + pad), 0x7F, dtype=torch.uint8)
    buf[:, :c] = torch.randint(-4, 5, (r, c), generator=g).float().to(dtype).view(torch.uint8)
    return buf.cuda()[:, :c].view(dtype)


def spread64(s, rows, cols):
    s = s.double().cpu()
    if s.shape[0] != rows:
        s = s.repeat_interleave(128, 0)[:rows]
    return s.repeat_interleave(128, 1)[:, :cols]


def held_exactly(m, n, k, tx, tw, rows, pad):
    """linear_fp8 of whole numbers and scales that are powers of two, with each type of
    result, with and without a workspace."""
    g = gen(m + n + k + rows)
    X, W = eights(g, m, k, tx, pad), eights(g, n, k, tw, pad)
    sx, sw = (torch.exp2(torch.randint(-1, 2, (r, -(-k // 128)), generator=g).float()).cuda()
              for r in (m, -(-n // rows)))
    bias, R = ints(g, n), ints(g, m, n)
    xd, wd = X.cpu().double() * spread64(sx, m, k), W.cpu().double() * spread64(sw, n, k)
    z = xd @ wd.t() + bias.double()
    # multiples of 1/4 (of two scales) below 2^22, also without cancellation: exact in fp32
    assert float((xd.abs() @ wd.abs().t()).max()) < 2 ** 22 - 3
    for out in TYPES:
        for ws in (None, space(pg.linear_fp8_workspace(m, n, k))):
            Y, Z = Guarded(m, n, out, pad=pad), Guarded(m, n, out, pad=pad)
            pg.linear_fp8(X, sx, W.t(), sw.t(), Y.t, bias=bias.to(out).cuda(), act="relu",
                          residual=R.to(out).cuda(), Z=Z.t, ws=ws)
            assert torch.equal(Z.t.cpu(), z.to(out))
            assert torch.equal(Y.t.cpu(), (z.clamp(min=0) + R.double()).to(out))
            Y.check("Y")
            Z.check("Z")


@pytest.mark.parametrize("types", [(E4M3, E4M3), (E5M2, E4M3), (E4M3, E5M2)], ids=lambda t: ids8(t[0]) + ids8(t[1]))
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("m", [1, 16, 17, 32])
@pytest.mark.parametrize("n,k", WIDE)
def test_wide_8_bit_products_of_few_rows(types, rows, m, n, k):
    held_exactly(m, n, k, *types, rows, pad=n % 8)


# shared between workgroups and not; more blocks than a workgroup's room for scales
# (16384 with 16 rows and a scale for each column, 30720 with block scales)
@pytest.mark.parametrize("k", [4096, 4224, 8320, 8337, 11000, 16512, 16517, 30848, 31000])
@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("m,n", [(1, 1), (1, 72), (16, 40), (17, 16), (32, 129)])
def test_long_8_bit_products_of_few_rows(rows, k, m, n):
    held_exactly(m, n, k, E4M3, E4M3, rows, pad=k % 2 * 3)
