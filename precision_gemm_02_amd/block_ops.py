"""Operators of a feed-forward block on GPU tensors: layer norm with its gradients.

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

from .layer_ops import (_DTYPES, _ROWS, _device, _dtype, _flat, _grad_type, _Rows, _rows, _shape2,
                        _space, _stream, _struct)

# every entry point include/pgemm_blocks.h declares
EXPORTS = ("pgemm_layer_norm", "pgemm_layer_norm_backward", "pgemm_layer_norm_backward_workspace",
           "pgemm_block_call")

_lib = None
_check = None
_call = None            # pgemm_block_call

# The arguments of pgemm_block_call, by op (see layer_ops)
_PACK = (
    _struct("3i", "0q", _ROWS, "PPf", "0q", "PP", _ROWS, "P"),
    _struct("4i", _ROWS, _ROWS, "PPP", _ROWS, _ROWS, "PPPNP"),
)
_LAYER_NORM, _LAYER_NORM_BACKWARD = range(2)


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
        "pgemm_layer_norm_backward": [i, i, i, i, _Rows, _Rows, p, p, p, _Rows, _Rows, p, p, p, z, p],
        "pgemm_layer_norm_backward_workspace": [i, i],
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
        code, _DTYPES[out], m, n, *_rows(dY, "dY", m, n, T, dev), *_rows(X, "X", m, n, T, dev),
        _flat(mean, "mean", (m,), f32, dev), _flat(rstd, "rstd", (m,), f32, dev),
        _flat(weight, "weight", (n,), T, dev), *_rows(residual, "residual", m, n, T, dev),
        *_rows(dX, "dX", m, n, T, dev), _flat(dweight, "dweight", (n,), out, dev),
        _flat(dbias, "dbias", (n,), out, dev), *_space(ws, dev), _stream(stream, dev)))
    if st != 0:
        _check(st, "layer_norm_backward")


def layer_norm_backward_workspace(m, n) -> int:
    """Workspace bytes ``layer_norm_backward`` needs for dweight or dbias."""
    return _lib.pgemm_layer_norm_backward_workspace(m, n)
