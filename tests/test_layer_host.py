"""The sequence-mixer layer's cache and the autograd wrappers' bookkeeping, on the CPU.

The operators need a GPU; here plain torch forms stand in for them, so that what the layer
and the wrappers do around them can be checked.
"""
from __future__ import annotations

import pytest

torch = pytest.importorskip("torch")

from quaternion_cumulative_product_gb300 import autograd as ag  # noqa: E402
from quaternion_cumulative_product_gb300 import layer as mixer_layer  # noqa: E402


def mul(a, b):
    aw, ax, ay, az = a.unbind(-1)
    bw, bx, by, bz = b.unbind(-1)
    return torch.stack([aw * bw - ax * bx - ay * by - az * bz, aw * bx + ax * bw + ay * bz - az * by,
                        aw * by - ax * bz + ay * bw + az * bx, aw * bz + ax * by - ay * bx + az * bw], -1)


def plain_cumprod(q, init, **_):
    out = []
    for t in range(q.shape[1]):
        init = mul(q[:, t], init)
        out.append(init)
    return torch.stack(out, 1) if out else torch.empty_like(q)


def plain_rotate(q, k, cum, w_q=None, w_k=None, **_):
    conj = cum * torch.tensor([1.0, -1.0, -1.0, -1.0])

    def one(x, w):
        n = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
        return mul(conj.repeat_interleave(x.shape[2] // cum.shape[2], 2), n.unflatten(-1, (-1, 4))).flatten(-2)
    return one(q, w_q), one(k, w_k)


def plain_delta(q, k, v, g, beta, init=None, scale=1.0, **_):
    B, S, Hv, Dv = v.shape
    q, k = (x.repeat_interleave(Hv // x.shape[2], 2) for x in (q, k))
    m = torch.zeros(B, Hv, q.shape[-1], Dv) if init is None else init + 0
    out = []
    for t in range(S):
        m = m * g[:, t].exp()[..., None, None]
        e = v[:, t] - torch.einsum("bhk,bhkv->bhv", k[:, t], m)
        m = m + k[:, t, :, :, None] * (beta[:, t, :, None] * e)[:, :, None]
        out.append(scale * torch.einsum("bhk,bhkv->bhv", q[:, t], m))
    return (torch.stack(out, 1) if out else torch.empty_like(v)), m.clone()   # (the library saves no final state)


def plain_step(q, k, v, g, beta, state, scale=1.0, **_):
    o, m = plain_delta(q, k, v, g, beta, state, scale)
    state.copy_(m)
    return o


@pytest.fixture
def layer(monkeypatch):
    for name, fn in (("quat_cumprod", plain_cumprod), ("quat_cumprod_fwd", plain_cumprod), ("quat_norm_rotate", plain_rotate),
                     ("quat_norm_rotate_fwd", plain_rotate), ("quat_delta", plain_delta), ("quat_delta_step", plain_step)):
        monkeypatch.setattr(mixer_layer, name, fn)
    torch.manual_seed(3)
    return mixer_layer.QuatDeltaMixer(12, 2, 8, groups=2, dtype=torch.float32, device="cpu")


@pytest.mark.parametrize("B,S", [(1, 5), (1, 1), (3, 1), (3, 5)])
def test_cache_owns_its_memory(layer, B, S):
    """The cache of a prefill holds one step's rotation, and tokens after it leave the prefill's graph as it was."""
    x = torch.randn(B, S + 2, 12)
    y, cache = layer(x[:, :S])
    assert cache.turn.untyped_storage().nbytes() == cache.turn.numel() * 4
    tokens = [layer.step(x[:, t : t + 1], cache) for t in (S, S + 1)]
    y.square().sum().backward()   # (an in-place change of what the prefill saved is an error here)
    assert all(torch.isfinite(p.grad).all() for p in layer.parameters())
    with torch.no_grad():
        whole, end = layer(x)
    assert torch.allclose(torch.cat([y.detach(), *tokens], 1), whole, atol=1e-5)
    assert torch.allclose(cache.turn, end.turn, atol=1e-5) and torch.allclose(cache.state, end.state, atol=1e-5)


def test_empty_prefill_leaves_the_old_cache_alone(layer):
    x = torch.randn(2, 6, 12)
    with torch.no_grad():
        _, old = layer(x[:, :4])
        kept = old.turn.clone(), old.state.clone()
        y, new = layer(x[:, :0], old)
    assert y.shape == (2, 0, 12) and torch.equal(new.turn, kept[0]) and torch.equal(new.state, kept[1])
    layer.step(x[:, 4:5], new)
    assert torch.equal(old.turn, kept[0]) and torch.equal(old.state, kept[1])


# ---------------------------------------------------------------------------
# The autograd wrappers.
# ---------------------------------------------------------------------------
@pytest.fixture
def wrapped(monkeypatch):
    """The wrappers over plain forms; returns the arguments of the delta backward's last call."""
    seen = {}

    def delta_fwd(q, k, v, g, beta, init=None, *, scale=None, offsets=None):
        return plain_delta(q, k, v, g, beta, init, scale or 1.0)

    def delta_fwd_carries(*a, **kw):
        return (*delta_fwd(*a, **kw), torch.zeros(1), torch.zeros(1))

    def delta_bwd(q, k, v, g, beta, carries, errors, d_o, d_final=None, *, scale=None, offsets=None):
        seen.update(q=q, k=k, v=v, d_o=d_o, d_final=d_final)
        with torch.enable_grad():
            five = [t.detach().requires_grad_() for t in (q, k, v, g, beta)]
            o, fin = plain_delta(*five, None, scale or 1.0)
            outs, cots = ([o, fin], [d_o, d_final]) if d_final is not None else ([o], [d_o])
            return (*torch.autograd.grad(outs, five, cots), torch.zeros(q.shape[0], v.shape[2], q.shape[3], v.shape[3]))

    def rotate_fwd(q, k, cum, w_q=None, w_k=None, *, norm="rms", eps=1e-6):
        return plain_rotate(q, k, cum, w_q, w_k)

    def rotate_bwd(q, k, cum, d_q, d_k, w_q=None, w_k=None, *, norm="rms", eps=1e-6):
        with torch.enable_grad():
            five = [t.detach().requires_grad_() for t in (q, k, cum, w_q, w_k)]
            return torch.autograd.grad(plain_rotate(*five), five, [d_q, d_k])

    for name, fn in (("quat_delta_fwd", delta_fwd), ("quat_delta_fwd_carries", delta_fwd_carries), ("quat_delta_bwd", delta_bwd),
                     ("quat_norm_rotate_fwd", rotate_fwd), ("quat_norm_rotate_bwd", rotate_bwd)):
        monkeypatch.setattr(ag, name, fn)
    return seen


def delta_leaves(B=2, S=3, H=1, D=8):
    torch.manual_seed(4)
    x = [torch.randn(B, S, H, D), torch.randn(B, S, H, D), torch.randn(B, S, H, D), -torch.rand(B, S, H), torch.rand(B, S, H)]
    return [t.requires_grad_() for t in x]


def test_second_derivatives_are_refused(wrapped):
    """The gradients carry no graph of their own: asking for theirs is an error, not a silent zero."""
    x = delta_leaves()
    o, _ = ag.quat_delta(*x)
    d_v, = torch.autograd.grad(o.square().sum(), x[2], create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        d_v.sum().backward()
    w = torch.ones(8, requires_grad=True)
    q, k = ag.quat_norm_rotate(x[0], x[1], torch.randn(2, 3, 1, 2, 4), w, w)
    d_w, = torch.autograd.grad(q.square().sum() + k.sum(), w, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        d_w.sum().backward()


def test_delta_cotangents_that_nobody_has(wrapped):
    """A loss of o alone sends no cotangent of the final state; one of the state alone counts o's as zero."""
    x = delta_leaves()
    o, fin = ag.quat_delta(*x)
    want = torch.autograd.grad(plain_delta(*x)[0].square().sum(), x)
    got = torch.autograd.grad(o.square().sum(), x, retain_graph=True)
    assert wrapped["d_final"] is None and all(torch.allclose(a, b, atol=1e-5) for a, b in zip(got, want))
    want = torch.autograd.grad(plain_delta(*x)[1].square().sum(), x[1:])
    got = torch.autograd.grad(fin.square().sum(), x[1:])
    assert (wrapped["d_o"] == 0).all() and all(torch.allclose(a, b, atol=1e-5) for a, b in zip(got, want))
