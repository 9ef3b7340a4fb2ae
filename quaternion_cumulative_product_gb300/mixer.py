"""Sequence-mixer operators around the quaternion scan (C ABI: ``include/quat_mixer.h``).

* :func:`quat_norm_rotate_fwd` / :func:`quat_norm_rotate_bwd`: the per-head norm of
  queries and keys, then their rotation by ``conj(cum)``, in one pass;
* :func:`quat_delta_fwd`, :func:`quat_delta_fwd_carries`, :func:`quat_delta_bwd`: the
  gated delta rule over whole sequences (equal or packed), and its backward from
  the forward's carries and errors;
* :func:`quat_delta_step`: the gated delta rule for single tokens, on a pool of states
  updated in place.

As in the rest of the binding, the calls check and marshal arguments only; the
work runs in the library's CUDA kernels on the current torch stream (or
``stream``, whose memory the outputs then come from), and there is no CPU path.
The differentiable forms are in :mod:`quaternion_cumulative_product_gb300.autograd`.
"""
from __future__ import annotations

import ctypes
import functools
import inspect

import torch

from . import QS_OK, QuatScanError, _on_device, _stream_handle, load_library

__all__ = ["QS_DELTA_STEPS", "QS_DELTA_MAX_D", "QS_ROTATE_MAX_D", "quat_norm_rotate_fwd", "quat_norm_rotate_bwd",
           "quat_delta_fwd", "quat_delta_fwd_carries", "quat_delta_bwd", "quat_delta_step"]

QS_DELTA_STEPS = 64     # steps per chunk of the delta rule's carries
QS_DELTA_MAX_D = 128    # largest head dimensions of the delta rule
QS_ROTATE_MAX_D = 256   # largest head dimension of quat_norm_rotate_*

_NORMS = {"rms": 0, "l2": 1}
_F32, _BF16 = torch.float32, torch.bfloat16
_get_device = getattr(torch._C, "_cuda_getDevice", lambda: None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:
    _get_device = lambda: None  # noqa: E731  (then always through a Stream object)
_ready = None


def _lib():
    """The library with the argument types of this module's calls set."""
    global _ready
    if _ready is None:
        lib = load_library()
        vp, i64, c_int, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        for name, head, pointers, sizes in (("quat_norm_rotate_fwd", [c_int, c_int, c_int, f32], 8, 7),
                                            ("quat_norm_rotate_bwd", [c_int, c_int, c_int, f32], 13, 7),
                                            ("quat_delta_fwd", [c_int, c_int, f32], 12, 7),
                                            ("quat_delta_bwd", [c_int, c_int, f32], 17, 7),
                                            ("quat_delta_step", [c_int, c_int, f32], 9, 7)):
            fn = getattr(lib, name)
            fn.argtypes = head + [vp] * pointers + [i64] * sizes + [vp]
            fn.restype = c_int
        _ready = lib
    return _ready


def _code(t, name):
    dtype = t.dtype
    if dtype is _BF16:
        return 1
    if dtype is _F32:
        return 0
    raise TypeError(f"{name} must be torch.float32 or torch.bfloat16, got {dtype}")


def _need(name, t, shape, device, dtype, contiguous=True):
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}" if t.is_cuda
                         else f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _first(name, t, dims):
    """The first tensor of a call: CUDA, of the right number of dimensions; returns its device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {tuple(t.shape)}")
    return t.device


def _strides(*tensors):
    """The ``strides`` argument: NULL when all are contiguous."""
    for t in tensors:
        if not t.is_contiguous():
            break
    else:
        return None
    out = []
    for t in tensors:
        if t.stride(-1) != 1 and t.shape[-1] > 1:
            raise ValueError("the last dimension must be contiguous")
        # A dimension of one entry has no stride to speak of.
        out += [t.stride(i) if t.shape[i] > 1 else 0 for i in range(3)]
    return (ctypes.c_int64 * len(out))(*out)


def _no_expanded(**tensors):
    """bfloat16 rows of the delta rule come by tensor maps, which hold no stride of zero."""
    for name, t in tensors.items():
        if t.dtype is _BF16 and not t.is_contiguous() and any(n > 1 and s == 0 for n, s in zip(t.shape, t.stride())):
            raise ValueError(f"{name} is an expanded view, which a bfloat16 call does not take: pass {name}.contiguous()")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _empty(t):
    """A contiguous tensor like ``t``."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _with_stream(fn):
    """Adds the argument ``stream``: the call runs with it as the current stream.

    Outputs are then allocated on it too: from the current stream's memory they could still
    be in use there when the call writes them, or be handed out again before it has.
    """
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        q = args[0] if args else kw.get("q")
        if isinstance(q, torch.Tensor) and q.is_cuda and q.device != stream.device:
            raise ValueError(f"stream is on {stream.device}, expected {q.device}")
        with torch.cuda.stream(stream):
            return fn(*args, **kw)

    said = inspect.signature(fn)
    call.__signature__ = said.replace(parameters=[*said.parameters.values(),
                                                  inspect.Parameter("stream", inspect.Parameter.KEYWORD_ONLY, default=None)])
    return call


def _run(fn, where, device, *args):
    """Calls the library with the current stream on ``device``."""
    if _get_device() == device.index:   # the usual call, without a context or a Stream object
        rc = fn(*args, _raw_stream(device.index))
    else:
        with _on_device(device):
            rc = fn(*args, _stream_handle(None, device))
    if rc != QS_OK:
        raise QuatScanError(rc, where)


# ---------------------------------------------------------------------------
# Norm and rotation of queries and keys.
# ---------------------------------------------------------------------------
def _rotate_args(q, k, cum, w_q, w_k, norm):
    device = _first("q", q, 4)
    _first("k", k, 4)
    _first("cum", cum, 5)
    B, S, Hq, D = q.shape
    Hk = k.shape[2]
    H, J = cum.shape[2], cum.shape[3]
    code = _code(q, "q")
    _need("k", k, (B, S, Hk, D), device, q.dtype, contiguous=False)
    cum_code = _code(cum, "cum")
    _need("cum", cum, (B, S, H, J, 4), device, cum.dtype)
    for name, w in (("w_q", w_q), ("w_k", w_k)):
        if w is not None:
            _need(name, w, (D,), device, torch.float32)
    if H == 0 or Hq % H or Hk % H:
        raise ValueError(f"the heads of q ({Hq}) and k ({Hk}) must be multiples of cum's ({H})")
    if 4 * J > D:
        raise ValueError(f"{J} quaternions do not fit a head of {D}")
    if norm not in _NORMS:
        raise ValueError(f"norm must be 'rms' or 'l2', got {norm!r}")
    return device, code, cum_code, (B, S, H, J, Hq, Hk, D)


@_with_stream
def quat_norm_rotate_fwd(q, k, cum, w_q=None, w_k=None, *, norm="rms", eps=1e-6, q_out=None, k_out=None):
    """Norm of each head of ``q`` and ``k``, then the rotation of its quaternions by ``conj(cum)``.

    ``q`` [B,S,Hq,D] and ``k`` [B,S,Hk,D]: float32 or bfloat16 CUDA, the last
    dimension contiguous (views of a joint projection need no copy).  ``cum``
    [B,S,H,J,4]: the scan's output, float32 or bfloat16, ``H`` a divisor of both
    head counts, ``4J <= D``; values of a head past ``4J`` are not rotated.
    ``norm``: ``"rms"`` (mean of squares) or ``"l2"`` (sum of squares); ``w_q``,
    ``w_k``: float32 [D] weights or None.  Returns contiguous ``(q_out, k_out)``.
    """
    device, code, cum_code, dims = _rotate_args(q, k, cum, w_q, w_k, norm)
    if q_out is None:
        q_out = _empty(q)
    else:
        _need("q_out", q_out, q.shape, device, q.dtype)
    if k_out is None:
        k_out = _empty(k)
    else:
        _need("k_out", k_out, k.shape, device, k.dtype)
    _run(_lib().quat_norm_rotate_fwd, "quat_norm_rotate_fwd", device, code, cum_code, _NORMS[norm], eps,
         q.data_ptr(), k.data_ptr(), cum.data_ptr(), _ptr(w_q), _ptr(w_k), q_out.data_ptr(), k_out.data_ptr(),
         _strides(q, k), *dims)
    return q_out, k_out


@_with_stream
def quat_norm_rotate_bwd(q, k, cum, d_q_out, d_k_out, w_q=None, w_k=None, *, norm="rms", eps=1e-6):
    """``(d_q, d_k, d_cum, d_w_q, d_w_k)`` of :func:`quat_norm_rotate_fwd` for cotangents of its outputs.

    Recomputed from the inputs.  ``d_cum`` (in ``cum``'s type) sums over the heads
    that share a rotation and goes to the scan's backward as it is; the weights'
    gradients are float32, None where there is no weight.
    """
    device, code, cum_code, dims = _rotate_args(q, k, cum, w_q, w_k, norm)
    _need("d_q_out", d_q_out, q.shape, device, q.dtype)
    _need("d_k_out", d_k_out, k.shape, device, k.dtype)
    d_q = _empty(q)
    d_k = _empty(k)
    d_cum = torch.empty_like(cum)
    d_w_q = None if w_q is None else torch.empty_like(w_q)
    d_w_k = None if w_k is None else torch.empty_like(w_k)
    _run(_lib().quat_norm_rotate_bwd, "quat_norm_rotate_bwd", device, code, cum_code, _NORMS[norm], eps,
         q.data_ptr(), k.data_ptr(), cum.data_ptr(), _ptr(w_q), _ptr(w_k), d_q_out.data_ptr(), d_k_out.data_ptr(),
         d_q.data_ptr(), d_k.data_ptr(), d_cum.data_ptr(), _ptr(d_w_q), _ptr(d_w_k), _strides(q, k), *dims)
    return d_q, d_k, d_cum, d_w_q, d_w_k


# ---------------------------------------------------------------------------
# The gated delta rule.
# ---------------------------------------------------------------------------
def _delta_args(q, k, v, g, beta):
    device = _first("q", q, 4)
    _first("v", v, 4)
    B, S, Hk, Dk = q.shape
    Hv, Dv = v.shape[2:]
    code = _code(q, "q")
    _need("k", k, (B, S, Hk, Dk), device, q.dtype, contiguous=False)
    _need("v", v, (B, S, Hv, Dv), device, q.dtype, contiguous=False)
    gate = _code(g, "g")
    _need("g", g, (B, S, Hv), device, g.dtype)
    _need("beta", beta, (B, S, Hv), device, g.dtype)
    if Hk == 0 or Hv % Hk:
        raise ValueError(f"the heads of v ({Hv}) must be a multiple of those of q and k ({Hk})")
    for name, d in (("q and k", Dk), ("v", Dv)):
        if d == 0 or d % 8 or d > QS_DELTA_MAX_D:
            raise ValueError(f"heads of {name} must hold a multiple of 8 values, at most {QS_DELTA_MAX_D}, got {d}")
    return device, code, gate, (B, S, Hk, Hv, Dk, Dv)


def _sequences(offsets, B, S, device):
    """(number of sequences, carry slots' leading shape)."""
    if offsets is None:
        return B, (B, -(-S // QS_DELTA_STEPS))
    if offsets.dim() != 1 or offsets.shape[0] < 1:
        raise ValueError(f"offsets must be [N+1], got {tuple(offsets.shape)}")
    _need("offsets", offsets, offsets.shape, device, torch.int32)
    if B != 1:
        raise ValueError(f"packed sequences need a batch of 1, got {B}")
    N = offsets.shape[0] - 1
    return N, (S // QS_DELTA_STEPS + N,)


def _delta_fwd(q, k, v, g, beta, init, scale, offsets, keep):
    device, code, gate, (B, S, Hk, Hv, Dk, Dv) = _delta_args(q, k, v, g, beta)
    _no_expanded(q=q, k=k, v=v)
    N, slots = _sequences(offsets, B, S, device)
    if init is not None:
        _need("init", init, (N, Hv, Dk, Dv), device, torch.float32)
    o = _empty(v)
    final = torch.empty((N, Hv, Dk, Dv), dtype=torch.float32, device=device)
    carries = errors = None
    if keep:
        carries = torch.empty((*slots, Hv, Dk, Dv), dtype=torch.float32, device=device)
        errors = torch.empty((B, S, Hv, Dv), dtype=torch.float32, device=device)
    _run(_lib().quat_delta_fwd, "quat_delta_fwd", device, code, gate, Dk ** -0.5 if scale is None else scale,
         q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _ptr(init), o.data_ptr(),
         final.data_ptr(), _ptr(carries), _ptr(errors), _strides(q, k, v), _ptr(offsets), N, B, S, Hk, Hv, Dk, Dv)
    return o, final, carries, errors


@_with_stream
def quat_delta_fwd(q, k, v, g, beta, init=None, *, scale=None, offsets=None):
    """The gated delta rule over whole sequences: ``(o, final_state)``.

    ``M~ = exp(g_t) M_{t-1}``, ``e_t = v_t - M~^T k_t``, ``M_t = M~ + k_t (beta_t e_t)^T``,
    ``o_t = scale * M_t^T q_t`` for each value head, with the key head ``h // (Hv // Hk)``.
    ``q``, ``k`` [B,S,Hk,Dk], ``v`` [B,S,Hv,Dv]: float32 or bfloat16 CUDA (last
    dimension contiguous; expanded views in float32 only; keys are usually unit vectors); ``g`` (log decays, <= 0;
    -inf clears the state) and ``beta`` [B,S,Hv]: float32 or bfloat16, both alike.
    ``init`` [N,Hv,Dk,Dv] float32 or None (zeros).  ``scale`` defaults to
    ``Dk ** -0.5``.  ``offsets`` (int32 [N+1] CUDA, from 0 to S): a batch of 1 holds
    N packed sequences, some perhaps empty; else N = B.
    """
    return _delta_fwd(q, k, v, g, beta, init, scale, offsets, False)[:2]


@_with_stream
def quat_delta_fwd_carries(q, k, v, g, beta, init=None, *, scale=None, offsets=None):
    """:func:`quat_delta_fwd` that keeps what the backward needs: ``(o, final_state, carries, errors)``.

    ``carries``: the state entering every 64-step chunk, float32 [B,ceil(S/64),Hv,Dk,Dv]
    (packed: [S//64 + N, Hv, Dk, Dv]); ``errors``: the ``e_t``, float32 [B,S,Hv,Dv].
    """
    return _delta_fwd(q, k, v, g, beta, init, scale, offsets, True)


@_with_stream
def quat_delta_bwd(q, k, v, g, beta, carries, errors, d_o, d_final=None, *, scale=None, offsets=None):
    """``(d_q, d_k, d_v, d_g, d_beta, d_init)`` from the forward's carries and errors.

    ``d_o``: cotangent of ``o`` (contiguous), ``d_final``: of the final state or None.
    """
    device, code, gate, (B, S, Hk, Hv, Dk, Dv) = _delta_args(q, k, v, g, beta)
    _no_expanded(q=q, k=k, v=v)
    N, slots = _sequences(offsets, B, S, device)
    _need("carries", carries, (*slots, Hv, Dk, Dv), device, torch.float32)
    _need("errors", errors, (B, S, Hv, Dv), device, torch.float32)
    _need("d_o", d_o, (B, S, Hv, Dv), device, v.dtype)
    if d_final is not None:
        _need("d_final", d_final, (N, Hv, Dk, Dv), device, torch.float32)
    d_q, d_k = _empty(q), _empty(k)
    d_v = _empty(v)
    d_g, d_beta = torch.empty_like(g), torch.empty_like(beta)
    d_init = torch.empty((N, Hv, Dk, Dv), dtype=torch.float32, device=device)
    _run(_lib().quat_delta_bwd, "quat_delta_bwd", device, code, gate, Dk ** -0.5 if scale is None else scale,
         q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), carries.data_ptr(), errors.data_ptr(),
         d_o.data_ptr(), _ptr(d_final), d_q.data_ptr(), d_k.data_ptr(), d_v.data_ptr(), d_g.data_ptr(), d_beta.data_ptr(),
         d_init.data_ptr(), _strides(q, k, v), _ptr(offsets), N, B, S, Hk, Hv, Dk, Dv)
    return d_q, d_k, d_v, d_g, d_beta, d_init


@_with_stream
def quat_delta_step(q, k, v, g, beta, state, *, slots=None, scale=None, o=None):
    """The gated delta rule for T new tokens (usually one) of N sequences: ``o``; ``state`` is updated in place.

    ``q``, ``k`` [N,T,Hk,Dk], ``v`` [N,T,Hv,Dv], ``g``, ``beta`` [N,T,Hv] as for
    :func:`quat_delta_fwd`; ``state`` float32 [P,Hv,Dk,Dv].  Row n uses
    ``state[slots[n]]`` (int32 [N]; None: ``state[n]``); a slot outside the pool
    (-1) marks an idle row, whose output is zero.  No two rows may share a slot.
    """
    device, code, gate, (N, T, Hk, Hv, Dk, Dv) = _delta_args(q, k, v, g, beta)
    _first("state", state, 4)
    P = state.shape[0]
    _need("state", state, (P, Hv, Dk, Dv), device, torch.float32)
    if slots is not None:
        _need("slots", slots, (N,), device, torch.int32)
    elif N > P:
        raise ValueError(f"{N} rows without slots need as many states, got {P}")
    if o is None:
        o = _empty(v)
    else:
        _need("o", o, (N, T, Hv, Dv), device, v.dtype)
    _run(_lib().quat_delta_step, "quat_delta_step", device, code, gate, Dk ** -0.5 if scale is None else scale,
         q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), state.data_ptr(), _ptr(slots),
         o.data_ptr(), _strides(q, k, v), P, N, T, Hk, Hv, Dk, Dv)
    return o
