"""Plain 64-bit forms of the residual block's operators and of linear attention with a decay (numpy, CPU).

Written from the formulas, step by step; nothing here is shared with the library.
"""
from __future__ import annotations

import numpy as np


def decay(q, k, v, g, init, scale):
    """(o, final) for q, k [S,Hk,Dk], v [S,Hv,Dv], g [S,Hv], init [Hv,Dk,Dv]."""
    S, Hv = g.shape
    shared = Hv // q.shape[1]
    q, k = np.repeat(q, shared, 1), np.repeat(k, shared, 1)
    M, o = init.copy(), np.zeros(v.shape)
    for t in range(S):
        M = np.exp(g[t])[:, None, None] * M + k[t][:, :, None] * v[t][:, None, :]
        o[t] = scale * np.einsum("hkv,hk->hv", M, q[t])
    return o, M


def decay_grad(q, k, v, g, init, scale, do, dfinal):
    """(d_q, d_k, d_v, d_g, d_init)."""
    S, Hv = g.shape
    Hk = q.shape[1]
    shared = Hv // Hk
    qh, kh = np.repeat(q, shared, 1), np.repeat(k, shared, 1)
    kept, M = [], init.copy()
    for t in range(S):
        before = np.exp(g[t])[:, None, None] * M
        M = before + kh[t][:, :, None] * v[t][:, None, :]
        kept.append((before, M))
    dq, dk, dv, dg, dM = np.zeros(qh.shape), np.zeros(kh.shape), np.zeros(v.shape), np.zeros(g.shape), dfinal.copy()
    for t in reversed(range(S)):
        before, M = kept[t]
        dM = dM + scale * qh[t][:, :, None] * do[t][:, None, :]
        dq[t] = scale * np.einsum("hkv,hv->hk", M, do[t])
        dk[t] = np.einsum("hkv,hv->hk", dM, v[t])
        dv[t] = np.einsum("hkv,hk->hv", dM, kh[t])
        dg[t] = (dM * before).sum((1, 2))
        dM = np.exp(g[t])[:, None, None] * dM
    fold = lambda x: x.reshape(S, Hk, shared, x.shape[-1]).sum(2)  # noqa: E731
    return fold(dq), fold(dk), dv, dg, dM


def layer_norm(x, w, b, eps):
    m = x.mean(-1, keepdims=True)
    n = (x - m) / np.sqrt(((x - m) ** 2).mean(-1, keepdims=True) + eps)
    return n * (1.0 if w is None else w) + (0.0 if b is None else b)


def layer_norm_grad(x, w, eps, dy):
    """(d_x, d_w, d_b) by the Jacobian of a row, d n_i / d x_j = r (delta_ij - 1/D - n_i n_j / D)."""
    D = x.shape[-1]
    rows, d = x.reshape(-1, D), dy.reshape(-1, D)
    m = rows.mean(-1, keepdims=True)
    r = 1 / np.sqrt(((rows - m) ** 2).mean(-1, keepdims=True) + eps)
    n = (rows - m) * r
    dn = d * (1.0 if w is None else w)
    dx = r * (dn - dn.sum(-1, keepdims=True) / D - n * (n * dn).sum(-1, keepdims=True) / D)
    return dx.reshape(x.shape), (d * n).sum(0), d.sum(0)


def philox_words(seed, offset, count):
    """Words 0 .. count-1 of Philox4x32-10 in Python integers."""
    out, low = [], 0xFFFFFFFF
    for block in range((count + 3) // 4):
        c = [block & low, block >> 32, offset & low, (offset >> 32) & low]
        k = [seed & low, (seed >> 32) & low]
        for _ in range(10):
            a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
            c = [(b >> 32) ^ c[1] ^ k[0], b & low, (a >> 32) ^ c[3] ^ k[1], a & low]
            k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
        out += c
    return np.array(out[:count], dtype=np.uint64)


def dropout(x, seed, offset, p, residual=None):
    keep = philox_words(seed, offset, x.size).reshape(x.shape) >= int(np.floor(p * 2.0 ** 32))
    y = np.where(keep, x / (1 - p) if p < 1 else 0.0, 0.0)
    return y if residual is None else residual + y
