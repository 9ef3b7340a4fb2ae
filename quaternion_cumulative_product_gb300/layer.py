"""A small sequence-mixer layer that runs the framework's operators together.

Per step: queries, keys, values, gates and one quaternion per four values of a head
are projected from the input; the quaternions' cumulative product
(:func:`.autograd.quat_cumprod`) is the position; the norm and rotation of queries
and keys (:func:`.autograd.quat_norm_rotate`) and the gated delta rule
(:func:`.autograd.quat_delta`) follow, and an output projection.  The same layer
trains on whole sequences, prefills a cache and continues it token by token
(:func:`.quat_delta_step` on the cache's states in place).

:class:`QuatDecayMixer` is the same layer with linear attention with a decay
(:func:`.autograd.quat_decay`, :func:`.quat_decay_step`) in place of the delta rule, and
:class:`QuatMixerBlock` the residual block around either: ``x + dropout(mixer(layer_norm(x)))``.
"""
from __future__ import annotations

import dataclasses

import torch

from . import quat_cumprod_fwd, quat_decay_step, quat_delta_step, quat_layer_norm_fwd, quat_norm_rotate_fwd
from .autograd import quat_cumprod, quat_decay, quat_delta, quat_dropout, quat_layer_norm, quat_norm_rotate

__all__ = ["QuatDeltaMixer", "QuatDecayMixer", "QuatMixerBlock", "MixerCache"]


@dataclasses.dataclass
class MixerCache:
    """What single tokens continue from: the last cumulative quaternion and the state."""
    turn: torch.Tensor    # [B, H, J, 4] float32
    state: torch.Tensor   # [B, Hv, D, D] float32


class QuatDeltaMixer(torch.nn.Module):
    """``width`` -> ``width``, with ``heads`` key heads of ``dim`` values shared by ``groups`` value heads each."""

    gates_per_head = 2

    def __init__(self, width, heads, dim, groups=1, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        if dim % 8:
            raise ValueError(f"dim must be a multiple of 8, got {dim}")
        self.heads, self.dim, self.groups, self.dtype = heads, dim, groups, dtype
        hv = heads * groups
        kw = {"bias": False, "dtype": dtype, "device": device}
        self.qkv = torch.nn.Linear(width, (2 * heads + hv) * dim, **kw)
        self.turn = torch.nn.Linear(width, heads * dim, **kw)
        self.gates = torch.nn.Linear(width, self.gates_per_head * hv, **kw)
        self.out = torch.nn.Linear(hv * dim, width, **kw)
        self.w_q = torch.nn.Parameter(torch.full((dim,), dim ** -0.5, device=device))   # unit vectors to start from
        self.w_k = torch.nn.Parameter(torch.full((dim,), dim ** -0.5, device=device))
        self.rate = torch.nn.Parameter(torch.linspace(-4.0, 0.0, hv, device=device))

    def _project(self, x):
        """q, k, v (views of one projection), the rule's gates, unit quaternions near the identity."""
        B, S, _ = x.shape
        H, hv = self.heads, self.heads * self.groups
        q, k, v = self.qkv(x).view(B, S, 2 * H + hv, self.dim).split([H, H, hv], dim=2)
        gates = self._gates(self.gates(x).float())
        turn = self.turn(x).float().view(B, S, H, self.dim // 4, 4)
        turn = torch.cat([1 + 0.1 * turn[..., :1], 0.1 * turn[..., 1:]], -1)
        turn = turn / turn.norm(dim=-1, keepdim=True)
        return q, k, v, gates, turn.contiguous()

    def _gates(self, t):
        """Log decays and beta."""
        a, b = t.chunk(2, dim=-1)
        return (-self.rate.exp() * torch.nn.functional.softplus(a)).contiguous(), torch.sigmoid(b).contiguous()

    def _attend(self, q, k, v, gates, state):
        return quat_delta(q, k, v, *gates, state, scale=1.0)

    def _attend_step(self, q, k, v, gates, state):
        return quat_delta_step(q, k, v, *gates, state, scale=1.0)

    def _identity(self, B, device):
        turn = torch.zeros(B, self.heads, self.dim // 4, 4, device=device)
        turn[..., 0] = 1
        return turn

    def forward(self, x, cache: MixerCache | None = None):
        """``x`` [B,S,width] -> (y [B,S,width], cache): training, or prefill after ``cache``."""
        B, S, _ = x.shape
        q, k, v, gates, turn = self._project(x)
        start = self._identity(B, x.device) if cache is None else cache.turn
        cum = quat_cumprod(turn, start, save_carries=True)
        q, k = quat_norm_rotate(q, k, cum, self.w_q.float(), self.w_k.float())
        o, state = self._attend(q, k, v, gates, None if cache is None else cache.state)
        # A copy: a view would keep all of cum, and step() would write into what autograd has saved.
        last = (cum[:, -1] if S else start).detach().clone(memory_format=torch.contiguous_format)
        return self.out(o.flatten(2)), MixerCache(last, state.detach())

    @torch.no_grad()
    def step(self, x, cache: MixerCache):
        """One token per sequence: ``x`` [B,1,width] -> y [B,1,width]; ``cache`` moves on in place."""
        q, k, v, gates, turn = self._project(x)
        cum = quat_cumprod_fwd(turn, cache.turn)
        cache.turn.copy_(cum[:, -1])
        q, k = quat_norm_rotate_fwd(q, k, cum, self.w_q.float(), self.w_k.float())
        o = self._attend_step(q, k, v, gates, cache.state)
        return self.out(o.flatten(2))


class QuatDecayMixer(QuatDeltaMixer):
    """The same with linear attention with a decay for each head: no beta, states that only add up."""

    gates_per_head = 1

    def _gates(self, t):
        """Log decays."""
        return ((-self.rate.exp() * torch.nn.functional.softplus(t)).contiguous(),)

    def _attend(self, q, k, v, gates, state):
        return quat_decay(q, k, v, *gates, state, scale=1.0)

    def _attend_step(self, q, k, v, gates, state):
        return quat_decay_step(q, k, v, *gates, state, scale=1.0)


class QuatMixerBlock(torch.nn.Module):
    """``x + dropout(mixer(layer_norm(x)))`` around a mixer of ``width``.

    ``key`` (a buffer: seed, offset) draws the dropout's mask; its offset is counted up by one
    each time the block trains, on the device, so that a captured step draws anew too.  Equal keys
    drop the same positions: without a ``seed`` a block takes one from torch's generator (``torch.manual_seed``),
    another for each block.  Replicas of a block want seeds of their own (a copy of a block, or a
    wrapper that broadcasts buffers, hands the first one's on).

    A forward that is run again for its gradients (activation checkpointing) has to draw the first
    one's mask: take ``key = block.next_key()`` outside of it and pass ``block(x, cache, key)``.  Without
    a key such a forward raises.
    """

    def __init__(self, mixer, width, p=0.0, eps=1e-5, seed=None, device="cuda"):
        super().__init__()
        self.mixer, self.p, self.eps = mixer, p, eps
        self.w = torch.nn.Parameter(torch.ones(width, device=device))
        self.b = torch.nn.Parameter(torch.zeros(width, device=device))
        if seed is None:
            seed = int(torch.randint(2 ** 63 - 1, (), device="cpu"))
        self.register_buffer("key", torch.tensor([seed, 0], dtype=torch.int64, device=device))

    def next_key(self):
        """The key that the next mask is drawn with, counted up: for a forward that is given its key."""
        key = self.key.clone()
        self.key[1] += 1
        return key

    def forward(self, x, cache: MixerCache | None = None, key=None):
        """``x`` [B,S,width] -> (y [B,S,width], cache), as the mixer's.  ``key``: the dropout's (None: the block's, counted up)."""
        drop = self.training and self.p > 0
        if drop and key is None and torch._C._current_graph_task_id() != -1:
            raise RuntimeError("a forward that runs again inside a backward needs the key of its first run: pass key=block.next_key()")
        y, cache = self.mixer(quat_layer_norm(x, self.w.float(), self.b.float(), eps=self.eps), cache)
        if not drop:
            return x + y, cache
        y = quat_dropout(y, self.key if key is None else key, self.p, x)
        if key is None:
            self.key[1] += 1
        return y, cache

    @torch.no_grad()
    def step(self, x, cache: MixerCache):
        """One token per sequence: ``x`` [B,1,width] -> y [B,1,width]; ``cache`` moves on in place."""
        return x + self.mixer.step(quat_layer_norm_fwd(x, self.w.float(), self.b.float(), eps=self.eps), cache)
