"""Operators of a feed-forward block on GPU tensors: layer norm and gated
products with their gradients, products of 8-bit operands and their quantization.

Thin ctypes binding over the entry points of ``include/pgemm_blocks.h``, with the
conventions of ``layer_ops``: tensors on the current device with contiguous
rows, results in tensors that the caller passes, workspaces of the caller
(uint8 tensors of at least the number of bytes that the ``*_workspace``
functions return), every call enqueued on ``stream`` (default: torch's current
stream) and returning at once.
"""
from __future__ import annotations

import ctypes

import torch

from .layer_ops import (_DTYPES, _KIND, _NO_WEIGHT, _ROWS, _WEIGHT, _act, _device, _dtype, _flat,
                        _grad_type, _Kind, _out, _Rows, _rows, _shape2, _space, _stream, _struct,
                        _Weight, _weight, _wrong)

# every entry point include/pgemm_blocks.h declares
EXPORTS = ("pgemm_layer_norm", "pgemm_layer_norm_backward", "pgemm_layer_norm_backward_workspace",
           "pgemm_gated_linear", "pgemm_gated_linear_workspace", "pgemm_gated_linear_backward",
           "pgemm_gated_linear_backward_workspace", "pgemm_quantize", "pgemm_linear_fp8",
           "pgemm_linear_fp8_workspace", "pgemm_block_call")

_FP8 = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}
_BLOCK = 128            # columns (and rows) of a block with one scale


class _Scales(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("row_stride", ctypes.c_longlong),
                ("block_stride", ctypes.c_longlong), ("rows", ctypes.c_int)]


def _pair(name, kind):
    return type(name, (ctypes.Structure,), {"_fields_": [("gate", kind), ("up", kind)]})


_GateWeights, _GateRows = _pair("_GateWeights", _Weight), _pair("_GateRows", _Rows)
_GateBias = _pair("_GateBias", ctypes.c_void_p)


class _Fp8Kind(ctypes.Structure):
    _fields_ = [("x_type", ctypes.c_int), ("w_type", ctypes.c_int), ("out_dtype", ctypes.c_int),
                ("act", ctypes.c_int)]

_lib = None
_check = None
_call = None            # pgemm_block_call

# The arguments of pgemm_block_call, by op (see layer_ops)
_SCALES = "Pqqi0q"
_PACK = (
    _struct("3i", "0q", _ROWS, "PPf", "0q", "PP", _ROWS, "P"),
    _struct(_KIND, "2i", "0q", _ROWS, _ROWS, "PPP", _ROWS, _ROWS, "PPPNP"),
    _struct("4i", _WEIGHT, _ROWS, _SCALES, "P"),
    _struct("7i", "0q", _ROWS, _SCALES, _ROWS, _SCALES, "P", _ROWS, _ROWS, _ROWS, "PNP"),
    _struct(_KIND, "3i", _ROWS, _WEIGHT, _WEIGHT, "PP", _ROWS, _ROWS, _ROWS, "PNP"),
    _struct(_KIND, "3i", _ROWS, _ROWS, _ROWS, _ROWS, _WEIGHT, _WEIGHT, _ROWS, _WEIGHT, _WEIGHT, "PP",
            "PNP"),
)
(_LAYER_NORM, _LAYER_NORM_BACKWARD, _QUANTIZE, _LINEAR_FP8, _GATED_LINEAR,
 _GATED_LINEAR_BACKWARD) = range(6)


def _bind(lib, check):
    """Declare the entry points' types (called once, by the package)."""
    global _lib, _check, _call
    missing = [n for n in EXPORTS if not hasattr(lib, n)]
    if missing:
        raise ImportError("libpgemm.so is older than this binding (no %s); rebuild it with "
                          "`python precision_gemm_02_amd/build.py`" % ", ".join(missing))
    i, f, p, z = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
    types = {
        "pgemm_layer_norm": [i, i, i, _Rows, p, p, f, p, p, _Rows, p],
        "pgemm_layer_norm_backward": [_Kind, i, i, _Rows, _Rows, p, p, p, _Rows, _Rows, p, p, p, z, p],
        "pgemm_layer_norm_backward_workspace": [i, i],
        "pgemm_gated_linear": [_Kind, i, i, i, _Rows, _GateWeights, _GateBias, _GateRows, _Rows, p, z,
                               p],
        "pgemm_gated_linear_workspace": [i, i, i, i],
        "pgemm_gated_linear_backward": [_Kind, i, i, i, _Rows, _GateRows, _Rows, _GateWeights, _Rows,
                                        _GateWeights, _GateBias, p, z, p],
        "pgemm_gated_linear_backward_workspace": [_Kind, i, i, i],
        "pgemm_quantize": [i, i, i, i, _Weight, _Rows, _Scales, p],
        "pgemm_linear_fp8": [_Fp8Kind, i, i, i, _Rows, _Scales, _Rows, _Scales, p, _Rows, _Rows, _Rows,
                             p, z, p],
        "pgemm_linear_fp8_workspace": [i, i, i],
    }
    for name, args in types.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = z if name.endswith("_workspace") else i
    lib.pgemm_block_call.argtypes = [i, ctypes.c_char_p]
    lib.pgemm_block_call.restype = i
    _lib, _check, _call = lib, check, lib.pgemm_block_call


# ---- layer norm ------------------------------------------------------------------

def layer_norm(X, Y, *, weight=None, bias=None, eps=1e-5, mean=None, rstd=None, stream=None):
    """Y <- (X - mean) * rstd * weight + bias for each row, in place; returns Y.

    X and Y (m, n), weight and bias (n,) have one dtype.  mean and rstd (m,)
    float32, if given, receive the rows' statistics for
    ``layer_norm_backward``: rstd is 1 / sqrt(variance + eps)."""
    dev = _device(X, "X")
    m, n = _shape2(X, "X")
    T, f32 = X.dtype, torch.float32
    st = _call(_LAYER_NORM, _PACK[_LAYER_NORM](
        _dtype(X, "X"), m, n, *_rows(X, "X", m, n, T, dev), _flat(weight, "weight", (n,), T, dev),
        _flat(bias, "bias", (n,), T, dev), eps, _flat(mean, "mean", (m,), f32, dev),
        _flat(rstd, "rstd", (m,), f32, dev), *_rows(Y, "Y", m, n, T, dev), _stream(stream, dev)))
    if st != 0:
        _check(st, "layer_norm")
    return Y


def layer_norm_backward(dY, X, mean, rstd, *, weight=None, residual=None, dX=None, dweight=None,
                        dbias=None, ws=None, stream=None):
    """Gradients of ``layer_norm``: dX (m, n), dweight and dbias (n,); those given are
    written.

    mean and rstd are what ``layer_norm`` kept.  residual (m, n), the gradient that
    reaches X past the norm, is added to dX and may be dX itself.  dX and
    residual have the inputs' dtype; dweight and dbias have it or float32.
    ``ws`` has ``layer_norm_backward_workspace`` bytes (needed for dweight and
    dbias)."""
    dev = _device(X, "X")
    m, n = _shape2(X, "X")
    T, f32 = X.dtype, torch.float32
    out = _grad_type(dweight, dbias, T)
    code = _dtype(X, "X")
    if out is not T and out is not f32:
        raise TypeError("dweight and dbias are %s, expected %s or float32" % (out, T))
    if mean is None or rstd is None:
        raise ValueError("mean and rstd are needed")
    st = _call(_LAYER_NORM_BACKWARD, _PACK[_LAYER_NORM_BACKWARD](
        code, _DTYPES[out], 0, m, n, *_rows(dY, "dY", m, n, T, dev), *_rows(X, "X", m, n, T, dev),
        _flat(mean, "mean", (m,), f32, dev), _flat(rstd, "rstd", (m,), f32, dev),
        _flat(weight, "weight", (n,), T, dev), *_rows(residual, "residual", m, n, T, dev),
        *_rows(dX, "dX", m, n, T, dev), _flat(dweight, "dweight", (n,), out, dev),
        _flat(dbias, "dbias", (n,), out, dev), *_space(ws, dev), _stream(stream, dev)))
    if st != 0:
        _check(st, "layer_norm_backward")


def layer_norm_backward_workspace(m, n) -> int:
    """Workspace bytes ``layer_norm_backward`` needs for dweight or dbias."""
    return _lib.pgemm_layer_norm_backward_workspace(m, n)


# ---- gated products ----------------------------------------------------------------

def _gate_weights(gate, up, k, n, dtype, device):
    """Both weights' members: in one order and with one stride."""
    g = _weight(gate, "W_gate", None, k, n, dtype, device)
    u = _weight(up, "W_up", None, k, n, dtype, device)
    if g[1:3] != u[1:3] and k > 0 and n > 0:
        raise ValueError("W_gate with strides %s and W_up with strides %s must have the same"
                         % (gate.stride(), up.stride()))
    return g + u


def gated_linear(X, W_gate, W_up, Y, *, bias_gate=None, bias_up=None, act="silu", Z_gate=None,
                 Z_up=None, ws=None, stream=None):
    """Y <- act(X @ W_gate + bias_gate) * (X @ W_up + bias_up), in place; returns Y.

    X (m, k), the weights (k, n) in either order but both with the same strides, the
    biases (n,) and Z (m, n) have one dtype; Y (m, n) has that dtype or float32.
    Z_gate and Z_up, if given, receive X @ W + bias of each for
    ``gated_linear_backward``.  ``ws`` (``gated_linear_workspace`` bytes) lets
    workgroups share a long k, and rows that are not whole chunks of 16 bytes be
    copied into such."""
    dev = _device(X, "X")
    m, k = _shape2(X, "X")
    n = _shape2(Y, "Y")[1]
    T = X.dtype
    if W_gate is None or W_up is None:
        raise ValueError("both weights are needed")
    st = _call(_GATED_LINEAR, _PACK[_GATED_LINEAR](
        _dtype(X, "X"), _out(Y, "Y", T), _act(act), m, n, k, *_rows(X, "X", m, k, T, dev),
        *_gate_weights(W_gate, W_up, k, n, T, dev), _flat(bias_gate, "bias_gate", (n,), T, dev),
        _flat(bias_up, "bias_up", (n,), T, dev), *_rows(Z_gate, "Z_gate", m, n, T, dev),
        *_rows(Z_up, "Z_up", m, n, T, dev), *_rows(Y, "Y", m, n, Y.dtype, dev), *_space(ws, dev),
        _stream(stream, dev)))
    if st != 0:
        _check(st, "gated_linear")
    return Y


def gated_linear_workspace(m, n, k, dtype) -> int:
    """Workspace bytes ``gated_linear`` can use for this shape (0: none)."""
    return _lib.pgemm_gated_linear_workspace(_DTYPES[dtype], m, n, k)


def gated_linear_backward(dY, X, W_gate, W_up, Z_gate, Z_up, *, act="silu", dX=None, dW_gate=None,
                          dW_up=None, dbias_gate=None, dbias_up=None, ws=None, stream=None):
    """Gradients of ``gated_linear``: with dZ_gate = dY * Z_up * act'(Z_gate) and dZ_up
    = dY * act(Z_gate), dX <- dZ_gate @ W_gate^T + dZ_up @ W_up^T, dW <- X^T @ dZ and
    dbias <- the sum of dZ's rows of each; those given are written.

    Z_gate and Z_up are what ``gated_linear`` kept.  dX has the inputs' dtype; the
    dW (each in either order) and dbias have one dtype, the inputs' or float32.  The
    weights may be None without dX, X without a dW.  ``ws`` has
    ``gated_linear_backward_workspace`` bytes."""
    dev = _device(dY, "dY")
    m, n = _shape2(dY, "dY")
    some = dX if dX is not None else X
    if some is not None:
        k = _shape2(some, "dX" if dX is not None else "X")[1]
    else:
        k = next((w.shape[0] for w in (dW_gate, dW_up, W_gate, W_up) if w is not None), 0)
    T = dY.dtype
    given = [t for t in (dW_gate, dW_up, dbias_gate, dbias_up) if t is not None]
    out = given[0].dtype if given else T
    code = _dtype(dY, "dY")
    if any(t.dtype is not out for t in given) or (out is not T and out is not torch.float32):
        raise TypeError("dW and dbias are %s, expected all %s or all float32"
                        % (", ".join(str(t.dtype) for t in given), T))
    if Z_gate is None or Z_up is None:
        raise ValueError("Z_gate and Z_up are needed")
    if W_gate is None or W_up is None:
        if dX is not None:
            raise ValueError("dX needs both weights")
        W = _NO_WEIGHT + _NO_WEIGHT
    else:
        W = _gate_weights(W_gate, W_up, k, n, T, dev)
    if X is None and (dW_gate is not None or dW_up is not None):
        raise ValueError("a dW needs X")
    st = _call(_GATED_LINEAR_BACKWARD, _PACK[_GATED_LINEAR_BACKWARD](
        code, _DTYPES[out], _act(act), m, n, k, *_rows(dY, "dY", m, n, T, dev),
        *_rows(Z_gate, "Z_gate", m, n, T, dev), *_rows(Z_up, "Z_up", m, n, T, dev),
        *_rows(X, "X", m, k, T, dev), *W, *_rows(dX, "dX", m, k, T, dev),
        *_weight(dW_gate, "dW_gate", None, k, n, out, dev),
        *_weight(dW_up, "dW_up", None, k, n, out, dev),
        _flat(dbias_gate, "dbias_gate", (n,), out, dev), _flat(dbias_up, "dbias_up", (n,), out, dev),
        *_space(ws, dev), _stream(stream, dev)))
    if st != 0:
        _check(st, "gated_linear_backward")


def gated_linear_backward_workspace(m, n, k, dtype) -> int:
    """Workspace bytes ``gated_linear_backward`` needs."""
    d = _DTYPES[dtype]
    return _lib.pgemm_gated_linear_backward_workspace(_Kind(d, d, 0), m, n, k)


# ---- 8-bit products ----------------------------------------------------------------

def _fp8(t, name):
    code = _FP8.get(t.dtype)
    if code is None:
        raise TypeError("%s is %s, expected float8_e4m3fn or float8_e5m2" % (name, t.dtype))
    return code


def _columns(t, name, rows, cols, device):
    """(address, column stride) of a matrix with contiguous columns."""
    if t.shape != (rows, cols) or t.get_device() != device:
        _wrong(t, name, t.dtype, (rows, cols), device)
    s0, s1 = t.stride()
    if s0 == 1 and s1 >= rows and cols > 1:
        return t.data_ptr(), s1 or 1
    if rows == 0 or cols == 0:
        return t.data_ptr(), max(1, rows)
    if rows > 1 and s0 != 1:
        raise ValueError("%s must have contiguous columns (strides %s): the transposed view of a weight "
                         "kept as n x k" % (name, (s0, s1)))
    if cols == 1:
        s1 = rows
    if s1 < rows:
        raise ValueError("%s has overlapping columns (strides %s)" % (name, (s0, s1)))
    return t.data_ptr(), s1


def _scales(t, name, rows, cols, device, turned=False, by_row=False, written=False):
    """(address, row stride, block stride, rows per scale) of the scales of a (rows,
    cols) matrix: one for 128 columns of each row, or of 128 rows together.  turned:
    the tensor is transposed."""
    blocks = (cols + 127) // 128
    if t.dtype is not torch.float32 or t.get_device() != device:
        _wrong(t, name, torch.float32, t.shape, device)
    if turned:
        n1, n0 = t.shape
        s1, s0 = t.stride()
    else:
        n0, n1 = t.shape
        s0, s1 = t.stride()
    by = 1 if n0 == rows else _BLOCK
    if n1 != blocks or (n0 != rows and (by_row or n0 != (rows + 127) // 128)):
        want = [(rows, blocks)] + ([] if by_row else [((rows + 127) // 128, blocks)])
        raise ValueError("%s is %s, expected %s" % (name, tuple(t.shape), " or ".join(
            str(w[::-1] if turned else w) for w in want)))
    if n0 <= 1:
        s0 = blocks
    if blocks <= 1:
        s1 = 1
    if written and n0 * blocks > 0 and not (
            (n0 == 1 or s0 > 0) and (blocks == 1 or s1 > 0) and
            (n0 == 1 or blocks == 1 or s0 >= blocks * s1 or s1 >= n0 * s0)):
        raise ValueError("%s overlaps itself (strides %s)" % (name, t.stride()))
    return t.data_ptr(), s0, s1, by


def quantize(X, Q, scales, *, stream=None):
    """Q <- X / scale in 8 bits, scales <- a scale for each block of 128 columns;
    returns Q.

    X (r, c) has contiguous rows or contiguous columns (a transposed view), Q (r, c)
    float8_e4m3fn or float8_e5m2 contiguous rows.  scales, float32, is (r, c / 128)
    for a scale of each row's block or (r / 128, c / 128) for one of 128 rows
    together, sizes rounded up, with any strides.  The largest magnitude of a
    block becomes the type's largest number; Q * scale stands for X.  A block
    that holds an infinity or a NaN becomes NaN."""
    dev = _device(X, "X")
    r, c = _shape2(X, "X")
    _shape2(scales, "scales")
    code, q = _dtype(X, "X"), _fp8(Q, "Q")
    st = _call(_QUANTIZE, _PACK[_QUANTIZE](
        code, q, r, c, *_weight(X, "X", None, r, c, X.dtype, dev),
        *_rows(Q, "Q", r, c, Q.dtype, dev), *_scales(scales, "scales", r, c, dev, written=True),
        _stream(stream, dev)))
    if st != 0:
        _check(st, "quantize")
    return Q


def linear_fp8(X, x_scales, W, w_scales, Y, *, bias=None, act="none", residual=None, Z=None, ws=None,
               stream=None):
    """Y <- act(X @ W + bias) + residual for 8-bit X and W with scales, in place;
    returns Y.

    X (m, k) has contiguous rows; W (k, n) contiguous columns: the transposed view
    of a weight kept as n x k.  Each is float8_e4m3fn or float8_e5m2.  x_scales
    (m, k / 128) and w_scales (k / 128, n) or (k / 128, n / 128), sizes rounded up,
    are float32 with any strides: ``quantize`` of the n x k weight gives W and
    w_scales transposed.  Y, residual, Z (m, n) and bias (n,) have one dtype; Z, if
    given, receives X @ W + bias.  ``ws`` (``linear_fp8_workspace`` bytes) lets
    several workgroups share a long k."""
    dev = _device(X, "X")
    m, k = _shape2(X, "X")
    n = _shape2(Y, "Y")[1]
    T = Y.dtype
    x, w, out = _fp8(X, "X"), _fp8(W, "W"), _dtype(Y, "Y")
    _shape2(W, "W")
    if x_scales.dim() != 2 or w_scales.dim() != 2:
        raise ValueError("x_scales and w_scales must be 2-D")
    st = _call(_LINEAR_FP8, _PACK[_LINEAR_FP8](
        x, w, out, _act(act), m, n, k, *_rows(X, "X", m, k, X.dtype, dev),
        *_scales(x_scales, "x_scales", m, k, dev, by_row=True),
        *_columns(W, "W", k, n, dev), *_scales(w_scales, "w_scales", n, k, dev, turned=True),
        _flat(bias, "bias", (n,), T, dev),
        *_rows(residual, "residual", m, n, T, dev), *_rows(Z, "Z", m, n, T, dev),
        *_rows(Y, "Y", m, n, T, dev), *_space(ws, dev), _stream(stream, dev)))
    if st != 0:
        _check(st, "linear_fp8")
    return Y


def linear_fp8_workspace(m, n, k) -> int:
    """Workspace bytes ``linear_fp8`` can use for this shape (0: none)."""
    return _lib.pgemm_linear_fp8_workspace(m, n, k)
