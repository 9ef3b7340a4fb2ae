"""Plain 64-bit forms of the sequence-mixer operators for the tests (numpy, CPU).

Written from the formulas token by token; nothing here is shared with the library.
"""
from __future__ import annotations

import numpy as np


def quat_mul(a, b):
    aw, ax, ay, az = np.moveaxis(a, -1, 0)
    bw, bx, by, bz = np.moveaxis(b, -1, 0)
    return np.stack([aw * bw - ax * bx - ay * by - az * bz, aw * bx + ax * bw + ay * bz - az * by,
                     aw * by - ax * bz + ay * bw + az * bx, aw * bz + ax * by - ay * bx + az * bw], -1)


def conj(a):
    return a * np.array([1.0, -1.0, -1.0, -1.0])


def _spread(cum, heads):
    return np.repeat(cum, heads // cum.shape[2], axis=2)


def norm_rotate(x, cum, w, norm, eps):
    """z [B,S,h,D] for x [B,S,h,D], cum [B,S,H,J,4]."""
    D, J = x.shape[-1], cum.shape[3]
    div = D if norm == "rms" else 1
    n = x / np.sqrt((x * x).sum(-1, keepdims=True) / div + eps)
    n = n * (1.0 if w is None else w)
    z = n.copy()
    turned = quat_mul(conj(_spread(cum, x.shape[2])), n[..., : 4 * J].reshape(*x.shape[:3], J, 4))
    z[..., : 4 * J] = turned.reshape(*x.shape[:3], 4 * J)
    return z


def norm_rotate_grad(x, cum, w, norm, eps, dz):
    """(d_x, d_cum, d_w)."""
    D, J, H = x.shape[-1], cum.shape[3], cum.shape[2]
    div = D if norm == "rms" else 1
    r = 1 / np.sqrt((x * x).sum(-1, keepdims=True) / div + eps)
    ww = np.ones(D) if w is None else w
    n = x * r * ww
    c = _spread(cum, x.shape[2])
    dzq = dz[..., : 4 * J].reshape(*x.shape[:3], J, 4)
    nq = n[..., : 4 * J].reshape(*x.shape[:3], J, 4)
    dn = dz.copy()
    dn[..., : 4 * J] = quat_mul(c, dzq).reshape(*x.shape[:3], 4 * J)
    dc = quat_mul(nq, conj(dzq)).reshape(*x.shape[:2], H, x.shape[2] // H, J, 4).sum(3)
    dm = dn * ww
    dx = dm * r - x * r ** 3 * (dm * x).sum(-1, keepdims=True) / div
    return dx, dc, (dn * x * r).sum((0, 1, 2))


def delta(q, k, v, g, beta, init, scale, keep=None):
    """(o, final) for q, k [S,Hk,Dk], v [S,Hv,Dv], g, beta [S,Hv], init [Hv,Dk,Dv]."""
    S, Hv = g.shape
    shared = Hv // q.shape[1]
    q, k = np.repeat(q, shared, 1), np.repeat(k, shared, 1)
    M = init.copy()
    o = np.zeros(v.shape)
    for t in range(S):
        before = M
        cleared = np.exp(g[t])[:, None, None] * M
        e = v[t] - np.einsum("hk,hkv->hv", k[t], cleared)
        M = cleared + k[t][:, :, None] * (beta[t][:, None] * e)[:, None, :]
        o[t] = scale * np.einsum("hk,hkv->hv", q[t], M)
        if keep is not None:
            keep.append((before, cleared, e, M))
    return o, M


def delta_grad(q, k, v, g, beta, init, scale, d_o, d_final):
    """(d_q, d_k, d_v, d_g, d_beta, d_init)."""
    keep = []
    delta(q, k, v, g, beta, init, scale, keep)
    S, Hv = g.shape
    Hk = q.shape[1]
    shared = Hv // Hk
    qr, kr = np.repeat(q, shared, 1), np.repeat(k, shared, 1)
    dq, dk, dv = np.zeros(qr.shape), np.zeros(kr.shape), np.zeros(v.shape)
    dg, dbeta = np.zeros(g.shape), np.zeros(beta.shape)
    dM = d_final.copy()
    for t in reversed(range(S)):
        before, cleared, e, M = keep[t]
        dq[t] = scale * np.einsum("hkv,hv->hk", M, d_o[t])
        dM = dM + scale * qr[t][:, :, None] * d_o[t][:, None, :]
        du = np.einsum("hkv,hk->hv", dM, kr[t])
        dbeta[t] = (du * e).sum(-1)
        de = beta[t][:, None] * du
        dk[t] = np.einsum("hkv,hv->hk", dM, beta[t][:, None] * e) - np.einsum("hkv,hv->hk", cleared, de)
        dv[t] = de
        dcl = dM - kr[t][:, :, None] * de[:, None, :]
        dg[t] = (dcl * cleared).sum((-1, -2))
        dM = np.exp(g[t])[:, None, None] * dcl
    fold = lambda d: d.reshape(S, Hk, shared, d.shape[2]).sum(2)  # noqa: E731
    return fold(dq), fold(dk), dv, dg, dbeta, dM
