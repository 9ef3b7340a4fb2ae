"""The sequence-mixer operators on the host: the formulas' own checks, and refusals (no GPU).

The 64-bit forms in ``mixer_reference.py``, which the GPU tests compare with, are
checked here against central differences; the C entry points' argument checks run
before any CUDA call and are called with pointers that nobody follows.
"""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

import mixer_reference as ref
import quaternion_cumulative_product_gb300 as qs
from quaternion_cumulative_product_gb300 import build as qbuild


def differences(loss, x, step=1e-6):
    """Central differences: the error is step^2 times a third derivative, and rounding over step, both below 1e-8 here."""
    out = np.zeros(x.shape)
    for i in np.ndindex(x.shape):
        keep = x[i]
        x[i] = keep + step
        hi = loss()
        x[i] = keep - step
        lo = loss()
        x[i] = keep
        out[i] = (hi - lo) / (2 * step)
    return out


@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_norm_rotate_gradient_by_differences(norm):
    rng = np.random.default_rng(0)
    x, cum, w = rng.standard_normal((1, 2, 4, 12)), rng.standard_normal((1, 2, 2, 2, 4)), rng.standard_normal(12)
    dz = rng.standard_normal(x.shape)
    loss = lambda: float((ref.norm_rotate(x, cum, w, norm, 0.1) * dz).sum())  # noqa: E731
    for got, leaf in zip(ref.norm_rotate_grad(x, cum, w, norm, 0.1, dz), (x, cum, w)):
        assert np.abs(got - differences(loss, leaf)).max() < 1e-7


def test_delta_gradient_by_differences():
    rng = np.random.default_rng(1)
    S, Hk, Hv, Dk, Dv = 4, 1, 2, 3, 2
    q, k, v = (rng.standard_normal(s) for s in ((S, Hk, Dk), (S, Hk, Dk), (S, Hv, Dv)))
    g, beta, init = -rng.random((S, Hv)), rng.random((S, Hv)), rng.standard_normal((Hv, Dk, Dv))
    do, df = rng.standard_normal(v.shape), rng.standard_normal(init.shape)

    def loss():
        o, f = ref.delta(q, k, v, g, beta, init, 0.7)
        return float((o * do).sum() + (f * df).sum())

    for got, leaf in zip(ref.delta_grad(q, k, v, g, beta, init, 0.7, do, df), (q, k, v, g, beta, init)):
        assert np.abs(got - differences(loss, leaf)).max() < 1e-7


def test_rotation_by_the_conjugate_is_relative():
    """<conj(c_t) a, conj(c_s) b> depends on q_t .. q_{s+1} alone; <c_t a, c_s b> does not."""
    rng = np.random.default_rng(2)
    unit = lambda *s: (lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True))(rng.standard_normal((*s, 4)))  # noqa: E731
    turn, a, b = unit(6), unit(), unit()
    dots = {"conj": [], "plain": []}
    for start in (unit(), unit()):
        c, cs = start, []
        for t in turn:
            c = ref.quat_mul(t, c)
            cs.append(c)
        dots["conj"].append(ref.quat_mul(ref.conj(cs[5]), a) @ ref.quat_mul(ref.conj(cs[2]), b))
        dots["plain"].append(ref.quat_mul(cs[5], a) @ ref.quat_mul(cs[2], b))
    assert abs(dots["conj"][0] - dots["conj"][1]) < 1e-12
    assert abs(dots["plain"][0] - dots["plain"][1]) > 1e-3


# ---------------------------------------------------------------------------
# Refusals of the C entry points.
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def lib():
    pytest.importorskip("torch")
    qbuild.build()
    from quaternion_cumulative_product_gb300 import mixer
    return mixer._lib()


def at(i):
    return ctypes.c_void_p((i + 1) << 40)   # far apart: no two of them overlap


def strides(*v):
    return (ctypes.c_int64 * len(v))(*v)


ROT = dict(dtype=1, cum=0, norm=0, eps=1e-6, B=2, S=3, H=2, J=4, Hq=4, Hk=2, D=16)


def rotate(lib, ptrs=None, st=None, bwd=False, **kw):
    p = [at(i) for i in range(12 if bwd else 7)] if ptrs is None else ptrs
    a = dict(ROT, **kw)
    fn = lib.quat_norm_rotate_bwd if bwd else lib.quat_norm_rotate_fwd
    return fn(a["dtype"], a["cum"], a["norm"], a["eps"], *p, st, a["B"], a["S"], a["H"], a["J"], a["Hq"], a["Hk"], a["D"], None)


@pytest.mark.parametrize("bwd", [False, True])
def test_norm_rotate_refusals(lib, bwd):
    for bad in (dict(dtype=2), dict(cum=-1), dict(norm=2), dict(eps=-1.0), dict(eps=float("nan")), dict(B=-1), dict(S=1 << 31),
                dict(J=5), dict(D=18), dict(D=260), dict(D=132), dict(Hq=3), dict(Hk=1), dict(B=1 << 20, S=1 << 12)):
        assert rotate(lib, bwd=bwd, **bad) == qs.QS_ERR_DIMS, bad
    n = 12 if bwd else 7
    need = [0, 1, 2, *([5, 6, 7, 8, 9, 10, 11] if bwd else [5, 6])]
    for i in range(n):
        p = [at(j) for j in range(n)]
        p[i] = ctypes.c_void_p(p[i].value + 4)
        assert rotate(lib, p, bwd=bwd) == qs.QS_ERR_MISALIGNED, i
        if i in need:
            p[i] = None
            assert rotate(lib, p, bwd=bwd) == qs.QS_ERR_NULL, i
    p = [at(j) for j in range(n)]
    p[-1] = p[0]
    assert rotate(lib, p, bwd=bwd) == qs.QS_ERR_ALIAS
    p = [at(j) for j in range(n)]
    p[-1] = p[-2]
    assert rotate(lib, p, bwd=bwd) == qs.QS_ERR_ALIAS
    assert rotate(lib, st=strides(192, 64, 16, 192, 64, 4), bwd=bwd) == qs.QS_ERR_MISALIGNED
    assert rotate(lib, st=strides(-192, 64, 16, 192, 64, 16), bwd=bwd) == qs.QS_ERR_MISALIGNED
    if not bwd:
        assert rotate(lib, [None] * 7, S=0) == qs.QS_OK


DELTA = dict(dtype=1, gate=0, scale=0.1, N=2, B=2, S=70, Hk=2, Hv=4, Dk=64, Dv=128)


def delta(lib, ptrs=None, st=None, offsets=None, bwd=False, **kw):
    n = 15 if bwd else 10
    p = [at(i) for i in range(n)] if ptrs is None else ptrs
    a = dict(DELTA, **kw)
    fn = lib.quat_delta_bwd if bwd else lib.quat_delta_fwd
    return fn(a["dtype"], a["gate"], a["scale"], *p, st, offsets, a["N"], a["B"], a["S"], a["Hk"], a["Hv"], a["Dk"], a["Dv"], None)


@pytest.mark.parametrize("bwd", [False, True])
def test_delta_refusals(lib, bwd):
    for bad in (dict(dtype=2), dict(gate=3), dict(N=3), dict(B=-1), dict(S=1 << 31), dict(Hv=3), dict(Hk=0), dict(Dk=0), dict(Dk=12),
                dict(Dv=136), dict(offsets=at(30)), dict(N=1 << 30, B=1 << 30), dict(S=(1 << 31) - 1, Hv=1 << 12)):
        assert delta(lib, bwd=bwd, **bad) == qs.QS_ERR_DIMS, bad
    n = 15 if bwd else 10
    need = [i for i in range(14) if i != 8] if bwd else [0, 1, 2, 3, 4, 6, 8, 9]
    for i in range(n):
        p = [at(j) for j in range(n)]
        p[i] = ctypes.c_void_p(p[i].value + 8)
        assert delta(lib, p, bwd=bwd) == qs.QS_ERR_MISALIGNED, i
        p[i] = None
        if i in need:
            assert delta(lib, p, bwd=bwd) == qs.QS_ERR_NULL, i
    for other in (0, n - 2):
        p = [at(j) for j in range(n)]
        p[n - 1] = p[other]
        assert delta(lib, p, bwd=bwd) == qs.QS_ERR_ALIAS
    good = [70 * 128, 128, 64] * 2 + [70 * 512, 512, 128]
    for i, v in ((0, -8), (1, 4), (5, 0), (7, 0)):
        assert delta(lib, st=strides(*[v if j == i else g for j, g in enumerate(good)]), bwd=bwd) == qs.QS_ERR_MISALIGNED
    assert delta(lib, [None] * n, bwd=bwd, N=0, B=0) == qs.QS_OK


STEP = dict(dtype=0, gate=0, scale=0.1, P=5, N=3, T=1, Hk=1, Hv=2, Dk=8, Dv=16)


def step(lib, ptrs=None, st=None, **kw):
    p = [at(i) for i in range(8)] if ptrs is None else ptrs
    a = dict(STEP, **kw)
    return lib.quat_delta_step(a["dtype"], a["gate"], a["scale"], *p, st, a["P"], a["N"], a["T"], a["Hk"], a["Hv"], a["Dk"], a["Dv"], None)


def test_step_refusals(lib):
    for bad in (dict(dtype=5), dict(gate=-1), dict(N=-1), dict(Hv=3, Hk=2), dict(Hk=0), dict(Dk=4), dict(Dv=200), dict(Dk=0), dict(N=1 << 30, P=1 << 30)):
        assert step(lib, **bad) == qs.QS_ERR_DIMS, bad
    p = [at(j) for j in range(8)]
    p[6] = None
    assert step(lib, p, N=6) == qs.QS_ERR_DIMS   # no slots, more rows than states
    for i in (0, 1, 2, 3, 4, 5, 7):
        p = [at(j) for j in range(8)]
        p[i] = None
        assert step(lib, p) == qs.QS_ERR_NULL, i
        p[i] = ctypes.c_void_p(at(i).value + 4)
        assert step(lib, p) == qs.QS_ERR_MISALIGNED, i
    p = [at(j) for j in range(8)]
    p[7] = p[5]
    assert step(lib, p) == qs.QS_ERR_ALIAS
    assert step(lib, st=strides(8, 8, 2, 8, 8, 8, 32, 32, 16)) == qs.QS_ERR_MISALIGNED
    assert step(lib, [None] * 8, N=0) == qs.QS_OK


# ---------------------------------------------------------------------------
# Refusals of the Python calls.
# ---------------------------------------------------------------------------
def test_python_calls_refuse_cpu_tensors():
    torch = pytest.importorskip("torch")
    z = torch.zeros
    q, g, m = z(1, 4, 2, 8), z(1, 4, 2), z(1, 2, 8, 8)
    with pytest.raises(ValueError, match="no CPU path"):
        qs.quat_norm_rotate_fwd(q, q, z(1, 4, 2, 2, 4))
    with pytest.raises(ValueError, match="no CPU path"):
        qs.quat_norm_rotate_bwd(q, q, z(1, 4, 2, 2, 4), q, q)
    for call in (qs.quat_delta_fwd, qs.quat_delta_fwd_carries):
        with pytest.raises(ValueError, match="no CPU path"):
            call(q, q, q, g, g)
    with pytest.raises(ValueError, match="no CPU path"):
        qs.quat_delta_bwd(q, q, q, g, g, z(1, 1, 2, 8, 8), q, q)
    with pytest.raises(ValueError, match="no CPU path"):
        qs.quat_delta_step(q, q, q, g, g, m)
    with pytest.raises(TypeError, match="torch.Tensor"):
        qs.quat_delta_step(None, q, q, g, g, m)


def test_module_names():
    assert qs.QS_DELTA_STEPS == 64 == qs.QS_CARRY_STEPS and qs.QS_DELTA_MAX_D == 128 and qs.QS_ROTATE_MAX_D == 256
    assert all(hasattr(qs, n) for n in qs.__all__)
    with pytest.raises(AttributeError):
        qs.no_such_name


def test_step_table_of_headers(lib):
    """The header's constants are the binding's."""
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "quat_mixer.h")).read()
    for name in ("QS_DELTA_STEPS", "QS_DELTA_MAX_D", "QS_ROTATE_MAX_D"):
        assert int(re.search(rf"#define {name} (\d+)", text).group(1)) == getattr(qs, name)
