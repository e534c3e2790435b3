"""The block operators on the GPU against plain 64-bit arithmetic on the CPU.

Sizes are small and chosen where the kernels can go wrong: one row, one
column, one more or less than a chunk, a class of row lengths or a tile, padded
and unaligned rows.  Inputs of small whole numbers make sums exact, so that
those results have to be equal bit by bit; random inputs are held to bounds that
count the roundings (u = 2^-24, of fp32), each result's own half step on top.
"""
import math

import pytest
import torch

import precision_gemm_02_amd as pg
from layer_util import Guarded, half_step, ints

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TYPES = [F32, F16, BF16]
ids = {F32: "f32", F16: "f16", BF16: "bf16"}.get
U = 2.0 ** -24


def gen(seed):
    return torch.Generator().manual_seed(seed)


def space(n):
    return torch.full((n + 16,), 0x7F, dtype=torch.uint8, device="cuda")


def held(t, want, err, name=""):
    """t equals want within err before its rounding to its own type."""
    fi = torch.finfo(t.dtype)
    step = torch.maximum(want.abs() + err, torch.tensor(fi.tiny, dtype=torch.float64)) * half_step(t.dtype)
    off = (t.double().cpu() - want).abs()
    bad = ~(off <= err + step)
    assert not bool(bad.any()), (name, int(bad.sum()), float(off[bad].max()))


# ---- layer norm --------------------------------------------------------------------

# (m, n): each class of row lengths, its ends, rows per workgroup
NORMS = [(1, 1), (3, 2), (16, 7), (17, 128), (5, 129), (9, 512), (4, 513), (6, 1000), (3, 1025),
         (2, 2048), (3, 2049), (2, 4095), (2, 4097), (2, 8192), (2, 8193), (1, 16384), (2, 16385),
         (1, 32768), (2, 32769), (1, 70001), (300, 24), (1030, 136)]


def norm64(x, w, b, eps):
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + eps)
    h = d * rstd
    y = h if w is None else h * w
    return mean, rstd, h, y if b is None else y + b


def stats_err(x, mean, rstd):
    """Bounds on the statistics: the mean is a sum of n numbers of which a thread adds
    at most 64 one after the other, its parts by halves (at most 10 + 16 steps), and
    the rest of it is added afterwards: 90 u of the mean magnitude, once again small;
    the variance's relative error is 96 u (64 + 26 sums, squares, the mean's own
    square) on top of twice the mean's relative to the spread, rstd's half of it."""
    mag = x.abs().mean(1, keepdim=True)
    # the remainder of the mean is added in fp32: what is left is its rounding and
    # 90 u of the mean of |x - mean|
    left = (x - mean).abs().mean(1, keepdim=True)
    e_mean = 2 * U * mag + 92 * U * (left + 90 * U * mag)
    e_rstd = rstd * (60 * U) + rstd * (90 * U * mag * rstd) ** 2
    return e_mean, e_rstd


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("shape", NORMS, ids=str)
@pytest.mark.parametrize("affine,pad", [(True, 0), (False, 3), (True, 8)])
def test_layer_norm(dtype, shape, affine, pad):
    m, n = shape
    g = gen(m * 100003 + n)
    data = torch.randn(m, n, generator=g) * 2 + torch.randn(m, 1, generator=g)
    X = Guarded(m, n, dtype, pad=pad, shift=pad % 2, data=data.to(dtype))
    w = torch.randn(n, generator=g).to(dtype).cuda() if affine else None
    b = torch.randn(n, generator=g).to(dtype).cuda() if affine else None
    Y = Guarded(m, n, dtype, pad=pad, shift=pad % 2)
    mean, rstd = (Guarded(1, m, F32, fill=7.0) for _ in range(2))
    eps = 1e-5
    assert pg.layer_norm(X.t, Y.t, weight=w, bias=b, eps=eps, mean=mean.t[0], rstd=rstd.t[0]) is Y.t
    x = X.t.double().cpu()
    w64, b64 = (None if t is None else t.double().cpu() for t in (w, b))
    mu, r, h, y = norm64(x, w64, b64, eps)
    e_mean, e_rstd = stats_err(x, mu, r)
    held(mean.t[0], mu[:, 0], e_mean[:, 0], "mean")
    held(rstd.t[0], r[:, 0], e_rstd[:, 0], "rstd")
    # h: the difference to the mean (one rounding of x - mean, one of the rest of it,
    # 92 u of the mean magnitude left), times rstd
    e_h = (x - mu).abs() * (3 * U * r + e_rstd) + r * (e_mean + 2 * U * (x.abs() + mu.abs()))
    e = e_h if w64 is None else e_h * w64.abs() + 2 * U * (h * w64).abs()
    if b64 is not None:
        e = e + 2 * U * (y.abs() + b64.abs())
    held(Y.t, y, e, "Y")
    for t, name in ((Y, "Y"), (mean, "mean"), (rstd, "rstd"), (X, "X")):
        t.check(name)


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_layer_norm_without_spread(dtype):
    """Rows of one value: the variance is 0, and so is every output."""
    for n in (1, 100, 3001, 40000):
        X = torch.full((3, n), 5.0, dtype=dtype, device="cuda")
        Y = torch.full_like(X, math.nan)
        rstd, mean = torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
        pg.layer_norm(X, Y, eps=0.25, mean=mean, rstd=rstd)
        assert bool((Y == 0).all()) and bool((rstd == 2).all()) and bool((mean == 5).all())


def test_layer_norm_far_from_zero():
    """A large offset does not cost the spread: the variance comes from the
    differences, and what is left of the mean corrects both."""
    x = torch.randn(4, 3000, generator=gen(3), dtype=torch.float64) + 4096.0
    X = x.float().cuda()
    Y = torch.empty_like(X)
    pg.layer_norm(X, Y)
    want = norm64(X.double().cpu(), None, None, 1e-5)[3]
    # x - mean is exact to one rounding of a number below 8 (mean rounded to a
    # multiple of 2^-11 first, x a multiple of 2^-12: the difference is exact), the
    # rest of the mean is known to 92 u of numbers below 8
    assert float((Y.double().cpu() - want).abs().max()) <= 8 * 200 * U


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
def test_layer_norm_keeps_nan_to_its_row(dtype):
    for n in (40, 700, 3000, 20000, 50000):
        X = torch.randn(6, n, generator=gen(n)).to(dtype).cuda()
        Y, Y2 = torch.empty_like(X), torch.empty_like(X)
        pg.layer_norm(X, Y)
        X[2, n // 2] = math.nan
        X[4, n - 1] = math.inf
        pg.layer_norm(X, Y2)
        assert bool(Y2[2].isnan().all()) and bool(Y2[4].isnan().any())
        for r in (0, 1, 3, 5):
            assert torch.equal(Y[r], Y2[r])


def back64(d, x, mean, rstd, w, r):
    h = (x - mean[:, None]) * rstd[:, None]
    g = d if w is None else d * w
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    return dx if r is None else dx + r, (d * h).sum(0), d.sum(0), h, g


@pytest.mark.parametrize("dtype", TYPES, ids=ids)
@pytest.mark.parametrize("shape", NORMS, ids=str)
@pytest.mark.parametrize("affine,pad,out", [(True, 0, None), (True, 3, F32), (False, 8, None)])
def test_layer_norm_backward(dtype, shape, affine, pad, out):
    m, n = shape
    g = gen(m * 100003 + n + 1)
    x = (torch.randn(m, n, generator=g) * 2 + torch.randn(m, 1, generator=g)).to(dtype)
    X = Guarded(m, n, dtype, pad=pad, shift=pad % 2, data=x)
    dY = Guarded(m, n, dtype, pad=pad, data=torch.randn(m, n, generator=g).to(dtype))
    R = Guarded(m, n, dtype, pad=pad, data=torch.randn(m, n, generator=g).to(dtype)) if pad else None
    w = torch.randn(n, generator=g).to(dtype).cuda() if affine else None
    mu, r, _, _ = norm64(x.double(), None, None, 1e-5)
    mean, rstd = mu[:, 0].float().cuda(), r[:, 0].float().cuda()
    dX = Guarded(m, n, dtype, pad=pad, shift=pad % 2)
    dw, db = (Guarded(1, n, out or dtype) for _ in range(2))
    ws = space(pg.layer_norm_backward_workspace(m, n))
    kw = dict(weight=w, residual=None if R is None else R.t)
    if affine:
        kw.update(dweight=dw.t[0], dbias=db.t[0], ws=ws)
    pg.layer_norm_backward(dY.t, X.t, mean, rstd, dX=dX.t, **kw)
    d64, x64, w64 = dY.t.double().cpu(), x.double(), None if w is None else w.double().cpu()
    m64, r64 = mean.double().cpu(), rstd.double().cpu()
    dx, sw, sb, h, gg = back64(d64, x64, m64, r64, w64, None if R is None else R.t.double().cpu())
    # h has two roundings, g one; a mean over the row 92 u of the mean magnitude (see
    # stats_err) besides its terms' own; then four roundings on the way to dX
    e_h = 2 * U * h.abs() + U * r64[:, None] * (x64.abs() + m64[:, None].abs())
    e1 = 93 * U * gg.abs().mean(1, keepdim=True)
    e2 = 95 * U * (gg * h).abs().mean(1, keepdim=True) + (gg.abs() * e_h).mean(1, keepdim=True)
    m1, m2 = gg.abs().mean(1, keepdim=True), (gg * h).abs().mean(1, keepdim=True)
    e = r64[:, None] * (5 * U * (gg.abs() + m1 + h.abs() * m2) + e1 + h.abs() * e2 + e_h * m2)
    if R is not None:
        e = e + 2 * U * (R.t.double().cpu().abs() + dx.abs())
    held(dX.t, dx, e, "dX")
    dX.check("dX")
    if affine:
        # at most 1024 rows one after the other, then groups
        steps = min(m, 1024) + 64
        held(dw.t[0], sw, steps * U * (d64 * h).abs().sum(0) + (d64.abs() * e_h).sum(0) +
             3 * U * (d64 * h).abs().sum(0), "dweight")
        held(db.t[0], sb, steps * U * d64.abs().sum(0), "dbias")
        dw.check("dweight")
        db.check("dbias")
        # each alone, and without dX, is the same up to the order of the sums
        dw2, db2 = torch.full_like(dw.t[0], math.nan), torch.full_like(db.t[0], math.nan)
        pg.layer_norm_backward(dY.t, X.t, mean, rstd, weight=w, dweight=dw2, ws=ws)
        pg.layer_norm_backward(dY.t, X.t, mean, rstd, weight=w, dbias=db2, ws=ws)
        held(dw2, sw, steps * U * (d64 * h).abs().sum(0) + (d64.abs() * e_h).sum(0) +
             3 * U * (d64 * h).abs().sum(0), "dweight alone")
        held(db2, sb, steps * U * d64.abs().sum(0), "dbias alone")
    if R is not None:                        # the residual may be dX itself
        again = R.t.clone()
        pg.layer_norm_backward(dY.t, X.t, mean, rstd, dX=again, **dict(kw, residual=again))
        assert torch.equal(again, dX.t)


def test_layer_norm_backward_without_rows():
    for dtype in TYPES:
        n = 40
        E = torch.empty(0, n, dtype=dtype, device="cuda")
        s = torch.empty(0, device="cuda")
        dw, db = (torch.full((n,), math.nan, dtype=dtype, device="cuda") for _ in range(2))
        pg.layer_norm_backward(E, E, s, s, dX=E, dweight=dw, dbias=db,
                               ws=space(pg.layer_norm_backward_workspace(0, n)))
        assert bool((dw == 0).all()) and bool((db == 0).all())


def test_layer_norm_gradients_against_differences():
    """dX, dweight and dbias against central differences of the forward pass in 64 bits."""
    m, n, eps = 3, 37, 1e-5
    g = gen(8)
    x, w, b, d = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((m, n), (n,), (n,), (m, n)))
    x, w, b, d = x.float().double(), w.float().double(), b.float().double(), d.float().double()

    def loss(x, w, b):
        return float((norm64(x, w, b, eps)[3] * d).sum())

    X, D = x.float().cuda(), d.float().cuda()
    Y, mean, rstd = torch.empty_like(X), torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    pg.layer_norm(X, Y, weight=w.float().cuda(), bias=b.float().cuda(), eps=eps, mean=mean, rstd=rstd)
    dX, dw, db = torch.empty_like(X), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    pg.layer_norm_backward(D, X, mean, rstd, weight=w.float().cuda(), dX=dX, dweight=dw, dbias=db,
                           ws=space(pg.layer_norm_backward_workspace(m, n)))
    s = 1e-5

    def diff(t, i, f):
        up, down = t.clone(), t.clone()
        up.view(-1)[i] += s
        down.view(-1)[i] -= s
        return (f(up) - f(down)) / (2 * s)

    # differences: s^2 times a third derivative (below 1e3 here) and 1e-16 * |loss| / s
    tol = 1e-5
    for i in range(0, m * n, 5):
        assert abs(float(dX.view(-1)[i]) - diff(x, i, lambda t: loss(t, w, b))) < tol
    for i in range(0, n, 5):
        assert abs(float(dw[i]) - diff(w, i, lambda t: loss(x, t, b))) < tol
        assert abs(float(db[i]) - diff(b, i, lambda t: loss(x, w, t))) < tol
