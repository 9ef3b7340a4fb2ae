"""A small sequence-mixer layer that runs the framework's operators together.

Per step: queries, keys, values, gates and one quaternion per four values of a head
are projected from the input; the quaternions' cumulative product
(:func:`.autograd.quat_cumprod`) is the position; the norm and rotation of queries
and keys (:func:`.autograd.quat_norm_rotate`) and the gated delta rule
(:func:`.autograd.quat_delta`) follow, and an output projection.  The same layer
trains on whole sequences, prefills a cache and continues it token by token
(:func:`.quat_delta_step` on the cache's states in place).
"""
from __future__ import annotations

import dataclasses

import torch

from . import quat_cumprod_fwd, quat_delta_step, quat_norm_rotate_fwd
from .autograd import quat_cumprod, quat_delta, quat_norm_rotate

__all__ = ["QuatDeltaMixer", "MixerCache"]


@dataclasses.dataclass
class MixerCache:
    """What single tokens continue from: the last cumulative quaternion and the state."""
    turn: torch.Tensor    # [B, H, J, 4] float32
    state: torch.Tensor   # [B, Hv, D, D] float32


class QuatDeltaMixer(torch.nn.Module):
    """``width`` -> ``width``, with ``heads`` key heads of ``dim`` values shared by ``groups`` value heads each."""

    def __init__(self, width, heads, dim, groups=1, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        if dim % 8:
            raise ValueError(f"dim must be a multiple of 8, got {dim}")
        self.heads, self.dim, self.groups, self.dtype = heads, dim, groups, dtype
        hv = heads * groups
        kw = {"bias": False, "dtype": dtype, "device": device}
        self.qkv = torch.nn.Linear(width, (2 * heads + hv) * dim, **kw)
        self.turn = torch.nn.Linear(width, heads * dim, **kw)
        self.gates = torch.nn.Linear(width, 2 * hv, **kw)
        self.out = torch.nn.Linear(hv * dim, width, **kw)
        self.w_q = torch.nn.Parameter(torch.full((dim,), dim ** -0.5, device=device))   # unit vectors to start from
        self.w_k = torch.nn.Parameter(torch.full((dim,), dim ** -0.5, device=device))
        self.rate = torch.nn.Parameter(torch.linspace(-4.0, 0.0, hv, device=device))

    def _project(self, x):
        """q, k, v (views of one projection), log decays, beta, unit quaternions near the identity."""
        B, S, _ = x.shape
        H, hv = self.heads, self.heads * self.groups
        q, k, v = self.qkv(x).view(B, S, 2 * H + hv, self.dim).split([H, H, hv], dim=2)
        a, b = self.gates(x).float().chunk(2, dim=-1)
        g = -self.rate.exp() * torch.nn.functional.softplus(a)
        turn = self.turn(x).float().view(B, S, H, self.dim // 4, 4)
        turn = torch.cat([1 + 0.1 * turn[..., :1], 0.1 * turn[..., 1:]], -1)
        turn = turn / turn.norm(dim=-1, keepdim=True)
        return q, k, v, g.contiguous(), torch.sigmoid(b).contiguous(), turn.contiguous()

    def _identity(self, B, device):
        turn = torch.zeros(B, self.heads, self.dim // 4, 4, device=device)
        turn[..., 0] = 1
        return turn

    def forward(self, x, cache: MixerCache | None = None):
        """``x`` [B,S,width] -> (y [B,S,width], cache): training, or prefill after ``cache``."""
        B, S, _ = x.shape
        q, k, v, g, beta, turn = self._project(x)
        start = self._identity(B, x.device) if cache is None else cache.turn
        cum = quat_cumprod(turn, start, save_carries=True)
        q, k = quat_norm_rotate(q, k, cum, self.w_q, self.w_k)
        o, state = quat_delta(q, k, v, g, beta, None if cache is None else cache.state, scale=1.0)
        # A copy: a view would keep all of cum, and step() would write into what autograd has saved.
        last = (cum[:, -1] if S else start).detach().clone(memory_format=torch.contiguous_format)
        return self.out(o.flatten(2)), MixerCache(last, state.detach())

    @torch.no_grad()
    def step(self, x, cache: MixerCache):
        """One token per sequence: ``x`` [B,1,width] -> y [B,1,width]; ``cache`` moves on in place."""
        q, k, v, g, beta, turn = self._project(x)
        cum = quat_cumprod_fwd(turn, cache.turn)
        cache.turn.copy_(cum[:, -1])
        q, k = quat_norm_rotate_fwd(q, k, cum, self.w_q, self.w_k)
        o = quat_delta_step(q, k, v, g, beta, cache.state, scale=1.0)
        return self.out(o.flatten(2))
