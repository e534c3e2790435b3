"""Layer operators on GPU tensors: linear, routing to experts, the experts'
products and their combination, each with its gradients.

Thin ctypes binding over the entry points of ``include/pgemm_layers.h``.
Tensors are float32, float16 or bfloat16 on the current device; their rows
are contiguous (any row stride that is at least the row's length).  Weights
are k x n tensors in either order: contiguous rows, or the transposed view of a
weight kept as n x k.  Results go to tensors that the caller passes; nothing
is allocated here, and workspaces are the caller's (uint8 tensors of at least
the number of bytes that the ``*_workspace`` functions return).  Every call is
enqueued on ``stream`` (default: torch's current stream) and returns at once.
"""
from __future__ import annotations

import ctypes
import struct

import torch

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
_ACTS = {"none": 0, None: 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
_SCORES = {"softmax": 0, "sigmoid": 1}
_KN, _NK = 0, 1


class _Rows(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_longlong)]


class _Weight(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_longlong), ("order", ctypes.c_int),
                ("stride", ctypes.c_longlong)]


class _Kind(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("out_dtype", ctypes.c_int), ("act", ctypes.c_int)]


class _RouteOut(ctypes.Structure):
    _fields_ = [(x, ctypes.c_void_p)
                for x in ("weights", "expert_index", "offsets", "tokens", "slots")]


class _Plan(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_int), ("offsets", ctypes.c_void_p),
                ("tokens", ctypes.c_void_p), ("x_rows", ctypes.c_int)]


# every entry point include/pgemm_layers.h declares
EXPORTS = ("pgemm_linear", "pgemm_linear_workspace", "pgemm_linear_backward",
           "pgemm_linear_backward_workspace", "pgemm_route", "pgemm_route_workspace",
           "pgemm_route_backward", "pgemm_expert_linear", "pgemm_expert_linear_backward",
           "pgemm_expert_linear_backward_workspace", "pgemm_combine", "pgemm_combine_backward",
           "pgemm_layer_call")

_lib = None
_check = None
_call = None            # pgemm_layer_call

# The arguments of pgemm_layer_call, by op: a call's parameters in order (P
# pointers, q and N 64-bit sizes, each at its natural alignment).  Packed
# arguments cost a call about 4 us less than structures built one by one.
_KIND, _ROWS, _WEIGHT, _PLAN = "3i", "Pq", "Pqiq", "iPPi"


def _struct(*parts):
    """A struct of nested C structs, each padded to its alignment."""
    fmt = "@"
    for p in parts:
        fmt += p + ("0q" if p in (_PLAN, _WEIGHT) else "")
    return struct.Struct(fmt).pack


_PACK = (
    _struct(_KIND, "3i", _ROWS, _WEIGHT, "P", _ROWS, _ROWS, _ROWS, "PNP"),
    _struct(_KIND, "3i", _ROWS, _ROWS, _ROWS, _WEIGHT, _ROWS, _WEIGHT, "PPNP"),
    _struct("8if", "0q", _ROWS, "P", "5P", "PNP"),
    _struct("6if", "P", _ROWS, "P", _ROWS, "P"),
    _struct(_KIND, "3i", _PLAN, _ROWS, _WEIGHT, "P", _ROWS, _ROWS, "P"),
    _struct(_KIND, "3i", _PLAN, _ROWS, _ROWS, _ROWS, _WEIGHT, _ROWS, _WEIGHT, "PPNP"),
    _struct("5i", "0q", _ROWS, "PP", _ROWS, _ROWS, "P"),
    _struct("5i", "0q", _ROWS, _ROWS, "PP", _ROWS, "PP"),
)
(_LINEAR, _LINEAR_BACKWARD, _ROUTE, _ROUTE_BACKWARD, _EXPERT_LINEAR, _EXPERT_LINEAR_BACKWARD,
 _COMBINE, _COMBINE_BACKWARD) = range(8)

_NO_ROWS = (0, 1)
_NO_WEIGHT = (0, 1, _KN, 0)


def _bind(lib, check):
    """Declare the entry points' types (called once, by the package)."""
    global _lib, _check, _call
    missing = [n for n in EXPORTS if not hasattr(lib, n)]
    if missing:
        raise ImportError("libpgemm.so is older than this binding (no %s); rebuild it with "
                          "`python precision_gemm_02_amd/build.py`" % ", ".join(missing))
    i, f, p, z = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
    types = {
        "pgemm_linear": [_Kind, i, i, i, _Rows, _Weight, p, _Rows, _Rows, _Rows, p, z, p],
        "pgemm_linear_workspace": [i, i, i, i],
        "pgemm_linear_backward": [_Kind, i, i, i, _Rows, _Rows, _Rows, _Weight, _Rows, _Weight, p,
                                  p, z, p],
        "pgemm_linear_backward_workspace": [_Kind, i, i, i],
        "pgemm_route": [i, i, i, i, i, i, i, i, f, _Rows, p, _RouteOut, p, z, p],
        "pgemm_route_workspace": [i, i, i],
        "pgemm_route_backward": [i, i, i, i, i, i, f, p, _Rows, p, _Rows, p],
        "pgemm_expert_linear": [_Kind, i, i, i, _Plan, _Rows, _Weight, p, _Rows, _Rows, p],
        "pgemm_expert_linear_backward": [_Kind, i, i, i, _Plan, _Rows, _Rows, _Rows, _Weight,
                                         _Rows, _Weight, p, p, z, p],
        "pgemm_expert_linear_backward_workspace": [_Kind, i, i, i, i],
        "pgemm_combine": [i, i, i, i, i, _Rows, p, p, _Rows, _Rows, p],
        "pgemm_combine_backward": [i, i, i, i, i, _Rows, _Rows, p, p, _Rows, p, p],
    }
    for name, args in types.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = z if name.endswith("_workspace") else i
    lib.pgemm_layer_call.argtypes = [i, ctypes.c_char_p]
    lib.pgemm_layer_call.restype = i
    _lib, _check, _call = lib, check, lib.pgemm_layer_call


# ---- arguments -----------------------------------------------------------------

def _device(t, name):
    """The current device's index, which must be the tensor's (an address
    elsewhere would be a fault on the GPU, not an error code)."""
    device = t.get_device()
    if device < 0 or device != torch._C._cuda_getDevice():
        raise TypeError("%s is on %s; pgemm needs memory of the current device" % (name, t.device))
    return device


def _wrong(t, name, dtype, shape, device):
    """Raise for the first thing that is not as expected."""
    if t.dtype is not dtype:
        raise TypeError("%s is %s, expected %s" % (name, t.dtype, dtype))
    if tuple(t.shape) != tuple(shape):
        raise ValueError("%s is %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    raise TypeError("%s is on %s; pgemm needs memory of the current device (cuda:%d)"
                    % (name, t.device, device))


def _rows(t, name, rows, cols, dtype, device):
    """(address, row stride) of a matrix with contiguous rows (None: none)."""
    if t is None:
        return _NO_ROWS
    if t.dtype is not dtype or t.shape != (rows, cols) or t.get_device() != device:
        _wrong(t, name, dtype, (rows, cols), device)
    s0, s1 = t.stride()
    if s1 == 1 and s0 >= cols and rows > 1:
        return t.data_ptr(), s0 or 1
    if rows == 0 or cols == 0:
        return t.data_ptr(), max(1, cols)
    if cols > 1 and s1 != 1:
        raise ValueError("%s must have contiguous rows (strides %s)" % (name, (s0, s1)))
    if rows == 1:
        s0 = cols
    if s0 < cols:
        raise ValueError("%s has overlapping rows (strides %s)" % (name, (s0, s1)))
    return t.data_ptr(), s0


def _weight(t, name, experts, k, n, dtype, device):
    """(address, ld, order, expert stride) of a k x n weight, or `experts` of
    them (experts None: one, 2-D)."""
    if t is None:
        return _NO_WEIGHT
    shape = (k, n) if experts is None else (experts, k, n)
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        _wrong(t, name, dtype, shape, device)
    if experts is None:
        stride, (sk, sn) = 0, t.stride()
    else:
        stride, sk, sn = t.stride()
    if k == 0 or n == 0 or experts == 0:
        return t.data_ptr(), max(1, n), _KN, max(1, k) * max(1, n)
    if (n == 1 or sn == 1) and (k == 1 or sk >= n):
        order, ld = _KN, (sk if k > 1 else n)
        span = (k - 1) * ld + n
    elif (k == 1 or sk == 1) and (n == 1 or sn >= k):
        order, ld = _NK, (sn if n > 1 else k)
        span = (n - 1) * ld + k
    else:
        raise ValueError("%s with strides %s has neither contiguous rows nor contiguous columns"
                         % (name, t.stride()))
    if experts is not None and experts > 1 and stride < span:
        raise ValueError("%s: the experts' weights overlap (strides %s)" % (name, t.stride()))
    return t.data_ptr(), ld, order, stride


def _flat(t, name, shape, dtype, device):
    """A contiguous tensor's address (None: 0)."""
    if t is None:
        return 0
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device:
        _wrong(t, name, dtype, shape, device)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _space(ws, device):
    if ws is None:
        return 0, 0
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    if ws.get_device() != device:
        raise TypeError("ws is on %s; pgemm needs memory of the current device" % ws.device)
    return ws.data_ptr(), ws.nbytes


def _stream(stream, device):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _dtype(t, name):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("%s is %s; the layer operators take float32, float16 and bfloat16"
                        % (name, t.dtype))
    return code


def _out(t, name, dtype):
    """A result's type: the inputs' or float32."""
    if t.dtype is not dtype and t.dtype is not torch.float32:
        raise TypeError("%s is %s, expected %s or float32" % (name, t.dtype, dtype))
    return _DTYPES[t.dtype]


def _act(act):
    code = _ACTS.get(act)
    if code is None:
        raise ValueError("act is %r, expected one of none, relu, gelu, gelu_tanh, silu" % (act,))
    return code


def _shape2(t, name):
    if t.dim() != 2:
        raise ValueError("%s must be 2-D" % name)
    return t.shape


# ---- the operators -------------------------------------------------------------

def linear(X, W, Y, *, bias=None, act="none", residual=None, Z=None, ws=None, stream=None):
    """Y <- act(X @ W + bias) + residual, in place; returns Y.

    X (m, k), W (k, n) in either order, bias (n,) and Z (m, n) have one dtype;
    Y and residual (m, n) have that dtype or float32.  Z, if given, receives X @
    W + bias for ``linear_backward``.  residual may be Y itself.  ``ws``
    (``linear_workspace`` bytes) lets few rows share a long k over more
    workgroups."""
    dev = _device(X, "X")
    m, k = _shape2(X, "X")
    n = _shape2(Y, "Y")[1]
    T = X.dtype
    out = Y.dtype
    st = _call(_LINEAR, _PACK[_LINEAR](
        _dtype(X, "X"), _out(Y, "Y", T), _act(act), m, n, k, *_rows(X, "X", m, k, T, dev),
        *_weight(W, "W", None, k, n, T, dev), _flat(bias, "bias", (n,), T, dev),
        *_rows(residual, "residual", m, n, out, dev), *_rows(Z, "Z", m, n, T, dev),
        *_rows(Y, "Y", m, n, out, dev), *_space(ws, dev), _stream(stream, dev)))
    if st != 0:
        _check(st, "linear")
    return Y


def linear_workspace(m, n, k, dtype) -> int:
    """Workspace bytes ``linear`` can use for this shape (0: none)."""
    return _lib.pgemm_linear_workspace(_DTYPES[dtype], m, n, k)


def _grad_type(dW, dbias, T):
    """The type of the weight's and bias's gradients: one of T and float32."""
    out = [x for x in (dW, dbias) if x is not None]
    if len(out) == 2 and dW.dtype is not dbias.dtype:
        raise TypeError("dW is %s and dbias %s; they share one dtype" % (dW.dtype, dbias.dtype))
    return out[0].dtype if out else T


def linear_backward(dY, X, W, *, Z=None, act="none", dX=None, dW=None, dbias=None, ws=None,
                    stream=None):
    """Gradients of ``linear``: with dZ = dY * act'(Z), dX <- dZ @ W^T, dW <-
    X^T @ dZ, dbias <- the sum of dZ's rows; those given are written.

    Z is what ``linear`` kept (needed unless act is none).  dX has the inputs'
    dtype; dW (in either order, not necessarily W's) and dbias have it or
    float32.  W may be None without dX, X without dW.  ``ws`` has
    ``linear_backward_workspace`` bytes."""
    dev = _device(dY, "dY")
    m, n = _shape2(dY, "dY")
    some = dX if dX is not None else X
    if some is not None:
        k = _shape2(some, "dX" if dX is not None else "X")[1]
    elif dW is not None or W is not None:
        k = (dW if dW is not None else W).shape[0]
    else:
        k = 0
    T = dY.dtype
    out = _grad_type(dW, dbias, T)
    code = _dtype(dY, "dY")
    if out is not T and out is not torch.float32:
        raise TypeError("dW and dbias are %s, expected %s or float32" % (out, T))
    st = _call(_LINEAR_BACKWARD, _PACK[_LINEAR_BACKWARD](
        code, _DTYPES[out], _act(act), m, n, k, *_rows(dY, "dY", m, n, T, dev),
        *_rows(Z, "Z", m, n, T, dev), *_rows(X, "X", m, k, T, dev),
        *_weight(W, "W", None, k, n, T, dev), *_rows(dX, "dX", m, k, T, dev),
        *_weight(dW, "dW", None, k, n, out, dev), _flat(dbias, "dbias", (n,), out, dev),
        *_space(ws, dev), _stream(stream, dev)))
    if st != 0:
        _check(st, "linear_backward")


def linear_backward_workspace(m, n, k, dtype, act="none") -> int:
    """Workspace bytes ``linear_backward`` needs."""
    d = _DTYPES[dtype]
    return _lib.pgemm_linear_backward_workspace(_Kind(d, d, _act(act)), m, n, k)


def _score(score):
    code = _SCORES.get(score)
    if code is None:
        raise ValueError("score is %r, expected softmax or sigmoid" % (score,))
    return code


def route(logits, weights, experts, offsets, tokens, slots, *, bias=None, score="softmax",
          groups=1, top_groups=1, renorm=True, scale=1.0, ws=None, stream=None):
    """The best experts of each token, their weights, and the plan that the
    experts' products read.

    logits (m, E).  Written: weights (m, top) float32, experts (m, top) int32
    (-1: none left), offsets (E + 1,) int32 (rows [offsets[e], offsets[e+1])
    are expert e's), tokens (m * top,) int32 (each row's token; entries
    behind the last row stay as they were) and slots (m, top) int32 (each
    choice's row, -1: none).  bias (E,) float32 is added to the scores for the
    choice alone; with ``groups`` the experts of the ``top_groups`` best groups
    compete.  Logits of -inf, of the dtype's lowest value and NaN are masked.
    ``ws`` has ``route_workspace`` bytes."""
    dev = _device(logits, "logits")
    m, E = _shape2(logits, "logits")
    top = _shape2(weights, "weights")[1]
    i32, f32 = torch.int32, torch.float32
    st = _call(_ROUTE, _PACK[_ROUTE](
        _dtype(logits, "logits"), m, E, top, _score(score), groups, top_groups, bool(renorm),
        scale, *_rows(logits, "logits", m, E, logits.dtype, dev),
        _flat(bias, "bias", (E,), f32, dev), _flat(weights, "weights", (m, top), f32, dev),
        _flat(experts, "experts", (m, top), i32, dev),
        _flat(offsets, "offsets", (E + 1,), i32, dev),
        _flat(tokens, "tokens", (m * top,), i32, dev), _flat(slots, "slots", (m, top), i32, dev),
        *_space(ws, dev), _stream(stream, dev)))
    if st != 0:
        _check(st, "route")


def route_workspace(m, experts, top) -> int:
    """Workspace bytes ``route`` needs (0 for up to 64 tokens)."""
    return _lib.pgemm_route_workspace(m, experts, top)


def route_backward(dweights, logits, experts, dlogits, *, score="softmax", renorm=True, scale=1.0,
                   stream=None):
    """dlogits (m, E) <- the gradient of ``route``'s weights, given theirs,
    for the choice that it made (experts).  No gradient reaches the bias."""
    dev = _device(logits, "logits")
    m, E = _shape2(logits, "logits")
    top = _shape2(experts, "experts")[1]
    T = logits.dtype
    st = _call(_ROUTE_BACKWARD, _PACK[_ROUTE_BACKWARD](
        _dtype(logits, "logits"), m, E, top, _score(score), bool(renorm), scale,
        _flat(dweights, "dweights", (m, top), torch.float32, dev),
        *_rows(logits, "logits", m, E, T, dev),
        _flat(experts, "experts", (m, top), torch.int32, dev),
        *_rows(dlogits, "dlogits", m, E, T, dev), _stream(stream, dev)))
    if st != 0:
        _check(st, "route_backward")
    return dlogits


def _plan(E, offsets, tokens, rows, x_rows, device):
    return (E, _flat(offsets, "offsets", (E + 1,), torch.int32, device),
            _flat(tokens, "tokens", (rows,), torch.int32, device), x_rows)


def expert_linear(X, W, Y, offsets, *, tokens=None, bias=None, act="none", Z=None, stream=None):
    """Y[r] <- act(X[src(r)] @ W[e] + bias[e]) for the rows r in [offsets[e],
    offsets[e+1]) of each expert e; returns Y.

    W (E, k, n), each in either order; bias (E, n).  With ``tokens`` src(r) is
    tokens[r], a row of X (m, k); without, X is (rows, k) and src(r) is r.
    Rows of Y (and Z) behind offsets[E] stay as they were."""
    dev = _device(X, "X")
    rows, n = _shape2(Y, "Y")
    xr, k = _shape2(X, "X")
    if W.dim() != 3:
        raise ValueError("W must be 3-D")
    E = W.shape[0]
    T = X.dtype
    st = _call(_EXPERT_LINEAR, _PACK[_EXPERT_LINEAR](
        _dtype(X, "X"), _out(Y, "Y", T), _act(act), rows, n, k,
        *_plan(E, offsets, tokens, rows, xr, dev), *_rows(X, "X", xr, k, T, dev),
        *_weight(W, "W", E, k, n, T, dev), _flat(bias, "bias", (E, n), T, dev),
        *_rows(Z, "Z", rows, n, T, dev), *_rows(Y, "Y", rows, n, Y.dtype, dev),
        _stream(stream, dev)))
    if st != 0:
        _check(st, "expert_linear")
    return Y


def expert_linear_backward(dY, X, W, offsets, *, tokens=None, Z=None, act="none", dX=None, dW=None,
                           dbias=None, ws=None, stream=None):
    """Gradients of ``expert_linear``: dX (rows, k) per row (``combine`` sums
    them over a token's rows), dW (E, k, n), dbias (E, n); those given are
    written, zeros for experts without rows.  W may be None without dX, X without
    dW.  ``ws`` has ``expert_linear_backward_workspace`` bytes."""
    dev = _device(dY, "dY")
    rows, n = _shape2(dY, "dY")
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("offsets is %s, expected (experts + 1,)" % (tuple(offsets.shape),))
    E = offsets.shape[0] - 1
    xr, k = rows, 0
    if X is not None:
        xr, k = _shape2(X, "X")
    elif dX is not None:
        k = _shape2(dX, "dX")[1]
    for t, name in ((W, "W"), (dW, "dW")):
        if t is not None:
            if t.dim() != 3:
                raise ValueError("%s must be 3-D" % name)
            if X is None and dX is None:
                k = t.shape[1]
    T = dY.dtype
    out = _grad_type(dW, dbias, T)
    code = _dtype(dY, "dY")
    if out is not T and out is not torch.float32:
        raise TypeError("dW and dbias are %s, expected %s or float32" % (out, T))
    st = _call(_EXPERT_LINEAR_BACKWARD, _PACK[_EXPERT_LINEAR_BACKWARD](
        code, _DTYPES[out], _act(act), rows, n, k, *_plan(E, offsets, tokens, rows, xr, dev),
        *_rows(dY, "dY", rows, n, T, dev), *_rows(Z, "Z", rows, n, T, dev),
        *_rows(X, "X", xr, k, T, dev), *_weight(W, "W", E, k, n, T, dev),
        *_rows(dX, "dX", rows, k, T, dev), *_weight(dW, "dW", E, k, n, out, dev),
        _flat(dbias, "dbias", (E, n), out, dev), *_space(ws, dev), _stream(stream, dev)))
    if st != 0:
        _check(st, "expert_linear_backward")


def expert_linear_backward_workspace(rows, n, k, experts, dtype, act="none") -> int:
    """Workspace bytes ``expert_linear_backward`` needs."""
    d = _DTYPES[dtype]
    return _lib.pgemm_expert_linear_backward_workspace(_Kind(d, d, _act(act)), rows, n, k, experts)


def combine(Y, slots, out, *, weights=None, residual=None, stream=None):
    """out[t] <- residual[t] + sum over j of weights[t, j] * Y[slots[t, j]];
    returns out.

    Y (rows, n), out and residual (m, n), slots (m, top) int32 (outside the
    rows, -1: none), weights (m, top) float32 (None: ones).  residual may be
    out itself."""
    dev = _device(Y, "Y")
    rows, n = _shape2(Y, "Y")
    m, top = _shape2(slots, "slots")
    T = Y.dtype
    st = _call(_COMBINE, _PACK[_COMBINE](
        _dtype(Y, "Y"), m, n, top, rows, *_rows(Y, "Y", rows, n, T, dev),
        _flat(slots, "slots", (m, top), torch.int32, dev),
        _flat(weights, "weights", (m, top), torch.float32, dev),
        *_rows(residual, "residual", m, n, T, dev), *_rows(out, "out", m, n, T, dev),
        _stream(stream, dev)))
    if st != 0:
        _check(st, "combine")
    return out


def combine_backward(dout, Y, slots, weights, *, dY=None, dweights=None, stream=None):
    """Gradients of ``combine``: dY[slots[t, j]] <- weights[t, j] * dout[t]
    (rows that no slot names stay as they were) and dweights[t, j] <-
    <dout[t], Y[slots[t, j]]>; those given are written (Y may be None without
    dweights).  The residual's gradient is dout.  A row belongs to one (token,
    choice) at most, as ``route`` gives them."""
    dev = _device(dout, "dout")
    m, n = _shape2(dout, "dout")
    top = _shape2(slots, "slots")[1]
    T = dout.dtype
    if dweights is not None and Y is None:
        raise ValueError("dweights needs Y")
    some = Y if Y is not None else dY
    rows = 0 if some is None else _shape2(some, "Y")[0]
    st = _call(_COMBINE_BACKWARD, _PACK[_COMBINE_BACKWARD](
        _dtype(dout, "dout"), m, n, top, rows, *_rows(dout, "dout", m, n, T, dev),
        *_rows(Y, "Y", rows, n, T, dev), _flat(slots, "slots", (m, top), torch.int32, dev),
        _flat(weights, "weights", (m, top), torch.float32, dev),
        *_rows(dY, "dY", rows, n, T, dev),
        _flat(dweights, "dweights", (m, top), torch.float32, dev), _stream(stream, dev)))
    if st != 0:
        _check(st, "combine_backward")
