"""Host-side checks of the layer operators (CPU only: no HIP call is made):
exports, argument codes, workspace sizes and the binding's refusals."""
import ctypes
import os
import re

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "pgemm_layers.h")

pg = pytest.importorskip("precision_gemm_02_amd", reason="libpgemm.so not built")
from precision_gemm_02_amd import layer_ops as lo  # noqa: E402

L = pg.library()
FAKE = 1 << 20          # 16-byte aligned placeholder address, never dereferenced
BF, F32 = torch.bfloat16, torch.float32


def R(data=FAKE, ld=64):
    return lo._Rows(data, ld)


def Wt(data=FAKE, ld=64, order=0, stride=4096):
    return lo._Weight(data, ld, order, stride)


KIND = lo._Kind(2, 2, 0)


def test_exports_every_declared_function():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = set(re.findall(r"\b(pgemm_[a-z0-9_]*)\s*\(", text))
    assert set(pg.LAYER_EXPORTS) == names
    for name in names:
        assert hasattr(L, name)


def linear(pos=None, value=None):
    args = [KIND, 8, 64, 64, R(), Wt(), None, R(None), R(None), R(), None, 0, None]
    if pos is not None:
        args[pos - 1] = value
    return L.pgemm_linear(*args)


@pytest.mark.parametrize("pos,value", [
    (1, lo._Kind(5, 5, 0)), (1, lo._Kind(2, 1, 0)), (1, lo._Kind(2, 2, 9)), (2, -1), (3, -1),
    (4, -1), (5, R(None)), (5, R(FAKE, 63)), (5, R(FAKE + 1)), (6, Wt(None)), (6, Wt(FAKE, 63)),
    (6, Wt(FAKE, 64, 7)), (7, FAKE + 1), (8, R(FAKE, 10)), (9, R(FAKE + 1)), (10, R(None)),
    (10, R(FAKE, 63)), (11, FAKE + 8)])
def test_linear_argument_codes(pos, value):
    assert linear(pos, value) == -pos


def test_linear_empty_touches_nothing():
    none = R(None)
    assert L.pgemm_linear(KIND, 0, 64, 64, none, Wt(None), None, none, none, none, None, 0, None) == 0
    assert L.pgemm_linear(KIND, 4, 0, 64, none, Wt(None), None, none, none, none, None, 0, None) == 0


def test_linear_backward_argument_codes():
    need = L.pgemm_linear_backward_workspace(lo._Kind(2, 2, 4), 8, 64, 64)
    ok = [lo._Kind(2, 2, 4), 8, 64, 64, R(), R(), R(), Wt(), R(), Wt(), FAKE, FAKE, need, None]
    for pos, value in ((1, lo._Kind(2, 1, 0)), (2, -1), (3, -1), (4, -1), (5, R(None)),
                       (6, R(None)), (7, R(None)), (8, Wt(None)), (9, R(FAKE, 1)),
                       (10, Wt(FAKE, 64, 3)), (11, FAKE + 1), (12, None), (12, FAKE + 4),
                       (13, need - 1)):
        args = list(ok)
        args[pos - 1] = value
        assert L.pgemm_linear_backward(*args) == -pos, pos


def test_route_argument_codes():
    out = lo._RouteOut(FAKE, FAKE, FAKE, FAKE, FAKE)
    need = L.pgemm_route_workspace(100, 64, 4)
    assert need > 0 and L.pgemm_route_workspace(64, 64, 4) == 0
    ok = [0, 100, 64, 4, 0, 8, 4, 1, 1.0, R(), FAKE, out, FAKE, need, None]
    for pos, value in ((1, 3), (2, -1), (3, 0), (3, 1025), (4, 0), (4, 33), (5, 2), (6, 0), (6, 7),
                       (7, 0), (7, 9), (10, R(FAKE, 63)), (11, FAKE + 2),
                       (12, lo._RouteOut(FAKE, None, FAKE, FAKE, FAKE)),
                       (12, lo._RouteOut(FAKE, FAKE, None, FAKE, FAKE)), (13, None), (14, need - 1)):
        args = list(ok)
        args[pos - 1] = value
        assert L.pgemm_route(*args) == -pos, (pos, value)
    args = list(ok)
    args[3], args[6] = 9, 1              # more than one group of 8 holds
    assert L.pgemm_route(*args) == -4
    args = [0, 10, 64, 4, 0, 1, 1.0, FAKE, R(), FAKE, R(), None]
    for pos, value in ((1, 4), (2, -1), (3, 2000), (4, 0), (5, 3), (8, None), (9, R(None)),
                       (10, None), (11, R(FAKE, 3))):
        a = list(args)
        a[pos - 1] = value
        assert L.pgemm_route_backward(*a) == -pos, pos


def test_expert_argument_codes():
    plan = lo._Plan(4, FAKE, FAKE, 8)
    bad_plans = [lo._Plan(0, FAKE, FAKE, 8), lo._Plan(2000, FAKE, FAKE, 8),
                 lo._Plan(4, None, FAKE, 8), lo._Plan(4, FAKE, FAKE + 2, 8),
                 lo._Plan(4, FAKE, FAKE, -1),
                 lo._Plan(4, FAKE, None, 31)]   # without tokens X has as many rows as Y
    ok = [KIND, 32, 64, 64, plan, R(), Wt(), FAKE, R(), R(), None]
    for pos, value in [(1, lo._Kind(9, 9, 0)), (2, -1), (3, -1), (4, -1), (6, R(None)),
                       (7, Wt(FAKE, 64, 0, 100)), (8, FAKE + 1), (9, R(FAKE, 3)),
                       (10, R(None))] + [(5, p) for p in bad_plans]:
        args = list(ok)
        args[pos - 1] = value
        assert L.pgemm_expert_linear(*args) == -pos, pos
    need = L.pgemm_expert_linear_backward_workspace(KIND, 32, 64, 64, 4)
    ok = [KIND, 32, 64, 64, plan, R(), R(), R(), Wt(), R(), Wt(), FAKE, FAKE, need, None]
    for pos, value in [(1, lo._Kind(2, 1, 0)), (2, -1), (6, R(None)), (8, R(None)), (9, Wt(None)),
                       (10, R(FAKE, 2)), (11, Wt(FAKE, 64, 0, 5)), (12, FAKE + 1), (13, None),
                       (14, need - 1)] + [(5, p) for p in bad_plans]:
        args = list(ok)
        args[pos - 1] = value
        assert L.pgemm_expert_linear_backward(*args) == -pos, pos


def test_combine_argument_codes():
    ok = [2, 8, 64, 2, 16, R(), FAKE, FAKE, R(), R(), None]
    for pos, value in ((1, 7), (2, -1), (3, -1), (4, 0), (4, 33), (5, -1), (6, R(None)), (7, None),
                       (8, FAKE + 1), (9, R(FAKE, 2)), (10, R(None))):
        args = list(ok)
        args[pos - 1] = value
        assert L.pgemm_combine(*args) == -pos, pos
    ok = [2, 8, 64, 2, 16, R(), R(), FAKE, FAKE, R(), FAKE, None]
    for pos, value in ((1, 7), (2, -1), (3, -1), (4, 0), (5, -1), (6, R(None)), (7, R(None)),
                       (8, None), (9, FAKE + 1), (10, R(FAKE, 2)), (11, FAKE + 2)):
        args = list(ok)
        args[pos - 1] = value
        assert L.pgemm_combine_backward(*args) == -pos, pos


def flat(args):
    """A call's arguments as pgemm_layer_call's packed members."""
    out = []
    for a in args:
        if isinstance(a, ctypes.Structure):
            out += flat(getattr(a, f) for f, _ in a._fields_)
        else:
            out.append(0 if a is None else a)
    return out


def test_packed_calls_equal_the_functions():
    """Every argument reaches its place: a bad value gives the same code."""
    out, plan = lo._RouteOut(FAKE, FAKE, FAKE, FAKE, FAKE), lo._Plan(4, FAKE, FAKE, 8)
    silu = lo._Kind(2, 2, 4)
    need = L.pgemm_linear_backward_workspace(silu, 8, 64, 64)
    needr = L.pgemm_route_workspace(100, 64, 4)
    neede = L.pgemm_expert_linear_backward_workspace(silu, 32, 64, 64, 4)
    calls = [
        (L.pgemm_linear, [KIND, 8, 64, 64, R(), Wt(), FAKE, R(), R(), R(), FAKE + 8, 0, None]),
        (L.pgemm_linear_backward, [silu, 8, 64, 64, R(), R(), R(), Wt(), R(), Wt(), FAKE, FAKE,
                                   need - 1, None]),
        (L.pgemm_route, [0, 100, 64, 4, 0, 8, 4, 1, 1.0, R(), FAKE, out, FAKE, needr - 1, None]),
        (L.pgemm_route_backward, [0, 10, 64, 4, 0, 1, 1.0, FAKE, R(), FAKE, R(FAKE, 3), None]),
        (L.pgemm_expert_linear, [KIND, 32, 64, 64, plan, R(), Wt(), FAKE, R(), R(FAKE, 3), None]),
        (L.pgemm_expert_linear_backward, [silu, 32, 64, 64, plan, R(), R(), R(), Wt(), R(), Wt(),
                                          FAKE, FAKE, neede - 1, None]),
        (L.pgemm_combine, [2, 8, 64, 2, 16, R(), FAKE, FAKE, R(), R(FAKE, 3), None]),
        (L.pgemm_combine_backward, [2, 8, 64, 2, 16, R(), R(), FAKE, FAKE, R(), FAKE + 2, None])]
    bad = {ctypes.c_int: -1, lo._Rows: R(FAKE + 1, 64), lo._Weight: Wt(FAKE, 64, 9),
           lo._Kind: lo._Kind(7, 7, 0), lo._Plan: lo._Plan(0, FAKE, FAKE, 8),
           lo._RouteOut: lo._RouteOut(FAKE, FAKE, FAKE + 1, FAKE, FAKE),
           ctypes.c_void_p: FAKE + 1}
    for op, (fn, args) in enumerate(calls):
        # the last bad argument alone, then also each earlier one
        assert fn(*args) < 0
        for pos, kind in enumerate(fn.argtypes[:-1]):
            a = list(args)
            if kind in bad:
                a[pos] = bad[kind]
            want = fn(*a)
            assert want < 0 and want > -100
            assert L.pgemm_layer_call(op, lo._PACK[op](*flat(a))) == want, (fn.__name__, pos)
    assert L.pgemm_layer_call(8, b"") == -1 and L.pgemm_layer_call(0, None) == -2


def test_workspace_sizes():
    # enough rows need none; one row of a long sum can use some
    assert pg.linear_workspace(8192, 8192, 4096, BF) == 0
    assert pg.linear_workspace(1, 512, 8192, BF) > 0
    assert pg.linear_workspace(0, 512, 8192, BF) == 0
    # dZ unless there is no activation
    none = pg.linear_backward_workspace(512, 256, 128, BF)
    silu = pg.linear_backward_workspace(512, 256, 128, BF, "silu")
    assert silu - none == 512 * 256 * 2
    for m in (0, 1, 7, 1000):
        for n in (0, 1, 9, 300):
            assert pg.linear_backward_workspace(m, n, 16, F32, "gelu") >= 0
            assert pg.expert_linear_backward_workspace(m, n, 16, 3, F32, "gelu") >= 0


@pytest.mark.parametrize("dtype", [BF, torch.float16, F32])
def test_workspaces_of_empty_sizes(dtype):
    """No inner size, no rows, no columns: sizes, whatever the others are."""
    for m in (0, 1, 16, 32, 33, 5000):
        for n in (0, 1, 64, 5000):
            for k in (0, 1, 64, 5000):
                for act in ("none", "silu"):
                    need = pg.linear_backward_workspace(m, n, k, dtype, act)
                    assert need >= m * n * dtype.itemsize * (act != "none")
                    assert pg.expert_linear_backward_workspace(m, n, k, 3, dtype, act) >= 0
                assert (pg.linear_workspace(m, n, k, dtype) == 0) or m * n * k > 0


@pytest.fixture
def anywhere(monkeypatch):
    """Let CPU tensors past the device checks: a call that is not refused
    before the library would be, by its own checks, or fail to launch."""
    monkeypatch.setattr(lo, "_device", lambda t, name: -1)
    monkeypatch.setattr(lo, "_stream", lambda s, d: 0)


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def test_cpu_tensors_are_refused():
    with pytest.raises(TypeError, match="current device"):
        pg.linear(z(2, 3), z(3, 4), z(2, 4))


@pytest.mark.parametrize("change,error", [
    (dict(W=z(3, 5)), ValueError), (dict(W=z(3, 4, dtype=F32)), TypeError),
    (dict(Y=z(2, 4, dtype=torch.float16)), TypeError), (dict(Y=z(3, 4)), ValueError),
    (dict(X=z(2, 3, dtype=torch.float64)), TypeError), (dict(X=z(3, 2).t()), ValueError),
    (dict(X=z(1, 3).expand(2, 3)), ValueError), (dict(W=z(3, 8)[:, ::2]), ValueError),
    (dict(bias=z(5)), ValueError), (dict(bias=z(8)[::2]), ValueError),
    (dict(residual=z(2, 4, dtype=F32)), TypeError), (dict(Z=z(2, 5)), ValueError),
    (dict(act="tanh"), ValueError), (dict(W=z(1, 3, 4)), ValueError), (dict(X=z(3)), ValueError)])
def test_linear_refusals(anywhere, change, error):
    args = dict(X=z(2, 3), W=z(3, 4), Y=z(2, 4))
    args.update(change)
    with pytest.raises(error):
        pg.linear(args.pop("X"), args.pop("W"), args.pop("Y"), **args)


def test_other_refusals(anywhere):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    f = lambda *s: torch.zeros(*s)
    with pytest.raises(TypeError):       # one dtype for dW and dbias
        pg.linear_backward(z(2, 4), z(2, 3), z(3, 4), dW=z(3, 4), dbias=f(4))
    with pytest.raises(TypeError):
        pg.linear_backward(z(2, 4), z(2, 3), z(3, 4), dW=z(3, 4, dtype=torch.float16))
    with pytest.raises(pg.PgemmError) as e:   # the workspace is required
        pg.linear_backward(z(2, 4), z(2, 3), z(3, 4), dbias=z(4))
    assert e.value.status == -12
    with pytest.raises(pg.PgemmError) as e:   # Z is needed with an activation
        pg.linear_backward(z(2, 4), z(2, 3), z(3, 4), act="silu", dX=z(2, 3))
    assert e.value.status == -6
    good = dict(weights=f(5, 2), experts=i(5, 2), offsets=i(9), tokens=i(10), slots=i(5, 2))
    for name, bad, err in (("weights", f(4, 2), ValueError), ("experts", f(5, 2), TypeError),
                           ("offsets", i(8), ValueError), ("tokens", i(9), ValueError),
                           ("slots", i(5, 4)[:, ::2], ValueError)):
        with pytest.raises(err):
            pg.route(f(5, 8), *dict(good, **{name: bad}).values())
    with pytest.raises(ValueError):
        pg.route(f(5, 8), *good.values(), score="other")
    with pytest.raises(pg.PgemmError) as e:   # three of eight experts' groups
        pg.route(f(5, 8), *good.values(), groups=3)
    assert e.value.status == -6
    with pytest.raises(ValueError):           # 2-D expert weights
        pg.expert_linear(z(4, 3), z(3, 4), z(4, 4), i(3))
    with pytest.raises(ValueError):           # overlapping experts
        pg.expert_linear(z(4, 3), z(1, 3, 4).expand(2, 3, 4), z(4, 4), i(3))
    with pytest.raises(pg.PgemmError) as e:   # fewer rows than Y without tokens
        pg.expert_linear(z(3, 3), z(2, 3, 4), z(4, 4), i(3))
    assert e.value.status == -5
    with pytest.raises(ValueError):
        pg.combine(z(4, 3), i(2, 2), z(2, 4))
    with pytest.raises(TypeError):
        pg.combine(z(4, 3), torch.zeros(2, 2, dtype=torch.int64), z(2, 3))
    with pytest.raises(ValueError):
        pg.combine_backward(z(2, 3), None, i(2, 2), None, dweights=f(2, 2))


def test_status_of_late_arguments_reads_as_an_argument():
    assert "argument" in pg.status_string(-14)


def test_expert_gradient_refusals(anywhere):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    dY, X, W, off = z(4, 5), z(4, 3), z(2, 3, 5), i(3)
    for args, kw in (((dY, X, W[0], off), {}), ((dY, X, z(3, 3, 5), off), {}),
                     ((dY, X, z(2, 4, 5), off), {}), ((dY, X, W, i(1)), {}), ((dY, X, W, i(3, 1)), {}),
                     ((dY, None, W, off), dict(dX=z(4, 4))), ((dY, None, W, off), dict(dX=z(3, 3))),
                     ((dY, X, None, off), dict(dW=z(2, 5, 3))), ((dY, X, None, off), dict(dW=z(3, 5)))):
        with pytest.raises(ValueError):
            pg.expert_linear_backward(*args, **kw)
    for kw in (dict(dX=z(4, 3)), dict(dW=z(2, 3, 5))):       # each needs the other operand
        with pytest.raises(pg.PgemmError) as e:
            pg.expert_linear_backward(dY, X if "dX" in kw else None, W if "dW" in kw else None, off,
                                      **kw)
        assert e.value.status == (-9 if "dX" in kw else -8)
