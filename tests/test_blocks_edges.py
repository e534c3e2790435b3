"""The block operators on the GPU where numbers leave their types' range, and in the kernels
that only wide or long calls take."""
import math

import pytest
import torch

import precision_gemm_02_amd as pg

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
