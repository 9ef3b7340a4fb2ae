"""Plain torch forms (any type, CPU) that stand in for the operators inside the layers."""
from __future__ import annotations

import block_reference as ref
import torch


def mul(a, b):
    aw, ax, ay, az = a.unbind(-1)
    bw, bx, by, bz = b.unbind(-1)
    return torch.stack([aw * bw - ax * bx - ay * by - az * bz, aw * bx + ax * bw + ay * bz - az * by,
                        aw * by - ax * bz + ay * bw + az * bx, aw * bz + ax * by - ay * bx + az * bw], -1)


def cumprod(q, init, **_):
    out = []
    for t in range(q.shape[1]):
        init = mul(q[:, t], init)
        out.append(init)
    return torch.stack(out, 1)


def rotate(q, k, cum, w_q=None, w_k=None, **_):
    conj = cum * torch.tensor([1.0, -1.0, -1.0, -1.0], dtype=cum.dtype)

    def one(x, w):
        n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        return mul(conj.repeat_interleave(x.shape[2] // cum.shape[2], 2), n.unflatten(-1, (-1, 4))).flatten(-2)
    return one(q, w_q), one(k, w_k)


def decay(q, k, v, g, init=None, scale=1.0, **_):
    B, S, Hv, Dv = v.shape
    q, k = (x.repeat_interleave(Hv // x.shape[2], 2) for x in (q, k))
    m = torch.zeros(B, Hv, q.shape[-1], Dv, dtype=v.dtype) if init is None else init + 0
    out = []
    for t in range(S):
        m = m * g[:, t].exp()[..., None, None] + k[:, t, :, :, None] * v[:, t, :, None]
        out.append(scale * torch.einsum("bhk,bhkv->bhv", q[:, t], m))
    return torch.stack(out, 1), m


def decay_step(q, k, v, g, state, scale=1.0, **_):
    o, m = decay(q, k, v, g, state, scale)
    state.copy_(m)
    return o


def layer_norm(x, w, b, eps=1e-5):
    m = x.mean(-1, keepdim=True)
    return (x - m) / ((x - m).square().mean(-1, keepdim=True) + eps).sqrt() * w + b


def dropout(x, key, p, residual=None):
    seed, offset = (int(t) % 2 ** 64 for t in key.tolist())
    keep = torch.from_numpy((ref.philox_words(seed, offset, x.numel()) >= int(p * 2 ** 32)).reshape(tuple(x.shape)))
    y = torch.where(keep, x / (1 - p), torch.zeros((), dtype=x.dtype))
    return y if residual is None else residual + y


def install(monkeypatch, layer):
    """Puts these in place of the operators in the module `layer`."""
    for name, form in {"quat_cumprod": cumprod, "quat_cumprod_fwd": cumprod, "quat_norm_rotate": rotate, "quat_norm_rotate_fwd": rotate,
                       "quat_decay": decay, "quat_decay_step": decay_step, "quat_layer_norm": layer_norm,
                       "quat_layer_norm_fwd": layer_norm, "quat_dropout": dropout}.items():
        monkeypatch.setattr(layer, name, form)
