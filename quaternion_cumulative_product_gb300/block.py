"""Operators of a residual block around the sequence mixer (C ABI: ``include/quat_block.h``).

* :func:`quat_layer_norm_fwd` / :func:`quat_layer_norm_bwd`: layer norm over the last
  dimension, and its backward with the weights' gradients;
* :func:`quat_dropout_fwd` / :func:`quat_dropout_bwd`: dropout from a counter-based
  generator, added on a residual, and its gradient; no mask is stored.

As in :mod:`quaternion_cumulative_product_gb300.mixer`, the calls check and marshal
arguments only, run on the current torch stream (or ``stream``), and have no CPU path.
The differentiable forms are in :mod:`quaternion_cumulative_product_gb300.autograd`.
"""
from __future__ import annotations

import ctypes

import torch

from . import load_library
from .mixer import _code, _empty, _need, _ptr, _run, _with_stream

__all__ = ["QS_NORM_MAX_D", "quat_layer_norm_fwd", "quat_layer_norm_bwd", "quat_dropout_fwd", "quat_dropout_bwd"]

QS_NORM_MAX_D = 16384   # longest row of quat_layer_norm_*

_ready = None


def _lib():
    """The library with the argument types of this module's calls set."""
    global _ready
    if _ready is None:
        lib = load_library()
        vp, i64, c_int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        for name, head, pointers, sizes in (("quat_layer_norm_fwd", [c_int, ctypes.c_float], 4, 3),
                                            ("quat_layer_norm_bwd", [c_int, ctypes.c_float], 6, 3),
                                            ("quat_dropout_fwd", [c_int, ctypes.c_double], 4, 1),
                                            ("quat_dropout_bwd", [c_int, ctypes.c_double], 3, 1)):
            fn = getattr(lib, name)
            fn.argtypes = head + [vp] * pointers + [i64] * sizes + [vp]
            fn.restype = c_int
        _ready = lib
    return _ready


def _cuda(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    return t.device


def _rows(x):
    """(rows, values of a row, distance between rows) of a tensor whose rows lie at one distance."""
    D = x.shape[-1]
    if x.is_contiguous():
        return x.numel() // D if D else 0, D, D
    if x.stride(-1) != 1 and D > 1:
        raise ValueError("the last dimension of x must be contiguous")
    rows, apart = 1, None
    for n, s in zip(reversed(x.shape[:-1]), reversed(x.stride()[:-1])):
        if n == 1:
            continue
        if apart is None:
            apart = s
        elif s != apart * rows:
            raise ValueError(f"the rows of x must lie at one distance (shape {tuple(x.shape)}, strides {x.stride()})")
        rows *= n
    return rows, D, D if apart is None else apart


def _norm_args(x, w, b):
    device = _cuda("x", x)
    if x.dim() < 1:
        raise ValueError("x must have at least one dimension")
    code = _code(x, "x")
    R, D, ld = _rows(x)
    if D > QS_NORM_MAX_D:
        raise ValueError(f"rows must hold at most {QS_NORM_MAX_D} values, got {D}")
    for name, t in (("w", w), ("b", b)):
        if t is not None:
            _need(name, t, (D,), device, torch.float32)
    return device, code, R, D, ld


@_with_stream
def quat_layer_norm_fwd(x, w=None, b=None, *, eps=1e-5, y=None):
    """Layer norm over the last dimension: ``(x - mean) / sqrt(var + eps) * w + b``.

    ``x`` [..,D]: float32 or bfloat16 CUDA, at most ``QS_NORM_MAX_D`` values to a row,
    rows contiguous and at one distance from each other (a slice of a joint projection
    needs no copy).  ``w``, ``b``: float32 [D] or None.  Returns a contiguous tensor.
    """
    device, code, R, D, ld = _norm_args(x, w, b)
    if y is None:
        y = _empty(x)
    else:
        _need("y", y, x.shape, device, x.dtype)
    _run(_lib().quat_layer_norm_fwd, "quat_layer_norm_fwd", device, code, eps, x.data_ptr(), _ptr(w), _ptr(b), y.data_ptr(), R, D, ld)
    return y


@_with_stream
def quat_layer_norm_bwd(x, d_y, w=None, b=None, *, eps=1e-5):
    """``(d_x, d_w, d_b)`` of :func:`quat_layer_norm_fwd` for a cotangent ``d_y`` (contiguous).

    Recomputed from ``x``.  ``d_w`` and ``d_b`` are float32, the sums over all rows in a
    fixed order, None where there is no weight or bias.
    """
    device, code, R, D, ld = _norm_args(x, w, b)
    _need("d_y", d_y, x.shape, device, x.dtype)
    d_x = _empty(x)
    d_w = None if w is None else torch.empty_like(w)
    d_b = None if b is None else torch.empty_like(b)
    _run(_lib().quat_layer_norm_bwd, "quat_layer_norm_bwd", device, code, eps, x.data_ptr(), _ptr(w), d_y.data_ptr(),
         d_x.data_ptr(), _ptr(d_w), _ptr(d_b), R, D, ld)
    return d_x, d_w, d_b


def _dropout_args(name, x, key, p):
    device = _cuda(name, x)
    code = _code(x, name)
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if not 0.0 <= p <= 1.0:
        raise ValueError(f"p must be between 0 and 1, got {p}")
    _need("key", key, (2,), device, torch.int64)
    return device, code


@_with_stream
def quat_dropout_fwd(x, key, p, residual=None, *, y=None):
    """``residual + dropout(x)``: each value is dropped with probability ``p``, the others are divided by ``1 - p``.

    ``x``: float32 or bfloat16 CUDA, contiguous; ``residual``: like ``x``, or None.  ``key``
    (int64 [2] CUDA: seed, offset) gives the random words: value ``i`` (in memory order) is
    kept where word ``i % 4`` of Philox4x32-10 at the counter ``(i // 4, offset)`` under
    ``seed`` is at least ``floor(p * 2**32)``.  The key is read when the work runs: count
    the offset up from call to call, and keep it for the backward.
    """
    device, code = _dropout_args("x", x, key, p)
    if residual is not None:
        _need("residual", residual, x.shape, device, x.dtype)
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    else:
        _need("y", y, x.shape, device, x.dtype)
    _run(_lib().quat_dropout_fwd, "quat_dropout_fwd", device, code, p, key.data_ptr(), x.data_ptr(), _ptr(residual), y.data_ptr(), x.numel())
    return y


@_with_stream
def quat_dropout_bwd(d_y, key, p):
    """``d_x`` of :func:`quat_dropout_fwd` (the residual's gradient is ``d_y`` itself), from the same ``key`` and ``p``."""
    device, code = _dropout_args("d_y", d_y, key, p)
    d_x = torch.empty_like(d_y, memory_format=torch.contiguous_format)
    _run(_lib().quat_dropout_bwd, "quat_dropout_bwd", device, code, p, key.data_ptr(), d_y.data_ptr(), d_x.data_ptr(), d_y.numel())
    return d_x
