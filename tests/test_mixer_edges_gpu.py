"""The sequence-mixer operators on the GPU at their edges: degenerate arguments, shared scratch, cancellation.

Tolerances are those of ``test_mixer_gpu.py`` (normwise, 192 additions in fp32 and
the output's own rounding) where no other is derived.
"""
from __future__ import annotations

import numpy as np
import pytest

import mixer_reference as ref
import quaternion_cumulative_product_gb300 as qs
from test_mixer_gpu import FIVE, TOL, close, delta_inputs, rotate_inputs, torch, wide  # noqa: F401  (torch: the fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# Norm and rotation.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("size", [1.0, 1e-14])
@pytest.mark.parametrize("dims", [(1, 5, 2, 4, 2, 64, 16), (2, 777, 3, 3, 6, 72, 5), (1, 1, 1, 1, 1, 256, 40)])
@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_norm_rotate_gradients_without_eps(torch, norm, dims, size):  # noqa: F811
    """eps 0, with fewer items than lane groups (their rows count as nothing) and rows whose inverse norm cubed is past fp32."""
    x = rotate_inputs(torch, *dims, "f32", "f32", True, seed=41)
    x["q"], x["k"] = x["q"] * size, x["k"] * size
    d = qs.quat_norm_rotate_bwd(x["q"], x["k"], x["cum"], x["dq"], x["dk"], x["w_q"], x["w_k"], norm=norm, eps=0.0)
    n = {k: wide(v) for k, v in x.items()}
    gq = ref.norm_rotate_grad(n["q"], n["cum"], n["w_q"], norm, 0.0, n["dq"])
    gk = ref.norm_rotate_grad(n["k"], n["cum"], n["w_k"], norm, 0.0, n["dk"])
    for got, want, what in zip(d, (gq[0], gk[0], gq[1] + gk[1], gq[2], gk[2]), ("d_q", "d_k", "d_cum", "d_w_q", "d_w_k")):
        close(got, want, "f32", what)


# ---------------------------------------------------------------------------
# Scratch shared by the calls of a stream.
# ---------------------------------------------------------------------------
def backward_call(torch, S, seed):  # noqa: F811
    """A delta backward with shared heads and a rotation backward with weights: both hand values over in scratch."""
    x = delta_inputs(torch, 1, S, 2, 4, 64, 64, "f32", "f32", seed=seed)
    y = rotate_inputs(torch, 1, S, 2, 4, 2, 64, 16, "f32", "f32", True, seed=seed)
    five = [x[n] for n in FIVE]
    _, _, carries, errors = qs.quat_delta_fwd_carries(*five, x["init"])

    def call():
        return [*qs.quat_delta_bwd(*five, carries, errors, x["d_o"], x["d_final"]),
                *qs.quat_norm_rotate_bwd(y["q"], y["k"], y["cum"], y["dq"], y["dk"], y["w_q"], y["w_k"])]
    return call


def test_graph_replays_after_its_stream_needed_more(torch):  # noqa: F811
    """A captured graph keeps its scratch when a larger call on the same stream has grown the stream's."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        small, large = backward_call(torch, 130, 51), backward_call(torch, 9000, 52)
        want = [t.clone() for t in small()]
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = small()
    with torch.cuda.stream(s):
        large()   # more scratch than the first call's
        second = torch.cuda.CUDAGraph()
    s.synchronize()
    with torch.cuda.graph(second, stream=s):
        large_got = large()
    with torch.cuda.stream(s):
        large_want = [t.clone() for t in large()]
        for t in (*got, *large_got):
            t.fill_(float("nan"))
        for g in (graph, second, graph):
            g.replay()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all(torch.equal(a, b) for a, b in zip(large_got, large_want))
    with torch.cuda.stream(s):
        assert qs.quat_cumprod_status() == qs.QS_OK


def test_threads_share_a_stream(torch):  # noqa: F811
    """Host threads whose calls meet on one stream: each gets its own results, whatever the others need of the scratch."""
    import threading
    calls = [backward_call(torch, S, 60 + i) for i, S in enumerate((70, 1500, 333))]
    want = [[t.clone() for t in c()] for c in calls]
    stream, failed = torch.cuda.Stream(), []   # (a stream without scratch so far)
    stream.wait_stream(torch.cuda.current_stream())

    def work(i):
        with torch.cuda.stream(stream):
            for _ in range(40):
                got = calls[i]()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    failed.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed


# ---------------------------------------------------------------------------
# The gates' gradients where decays are strong.
# ---------------------------------------------------------------------------
DECAYED = [(1, 150, 1, 2, 64, 64), (2, 129, 2, 2, 128, 128), (1, 90, 2, 4, 24, 104), (1, 64, 1, 2, 96, 40)]


@pytest.mark.parametrize("dims", DECAYED)
@pytest.mark.parametrize("dt,gates", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
def test_delta_gate_gradients_of_decayed_heads(torch, dims, dt, gates):  # noqa: F811
    """d_g per head, one of them with strong decays only: its gradients are many orders below the chunk's largest products.

    d_g is a sum of products that each hold exp(g): the tolerance is the operators' own, per head.
    """
    B, S, Hk, Hv, Dk, Dv = dims
    x = delta_inputs(torch, *dims, dt, gates, seed=71)
    x["g"][..., -1] = (-8 - 12 * torch.rand(B, S, device="cuda")).to(x["g"].dtype)   # exp: 3e-4 .. 2e-9
    five = [x[n] for n in FIVE]
    _, _, carries, errors = qs.quat_delta_fwd_carries(*five, x["init"])
    d_g = qs.quat_delta_bwd(*five, carries, errors, x["d_o"], x["d_final"])[3]
    n = {k: wide(v) for k, v in x.items()}
    want = np.stack([ref.delta_grad(*[n[k][b] for k in FIVE], n["init"][b], Dk ** -0.5, n["d_o"][b], n["d_final"][b])[3] for b in range(B)])
    for h in range(Hv):
        close(d_g[..., h], want[..., h], gates, h)


@pytest.mark.parametrize("dt,gates", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("D", [64, 128])
def test_delta_gate_gradients_of_cleared_states(torch, D, dt, gates):  # noqa: F811
    """Where exp(g) is zero in fp32 nothing depends on g: d_g is exactly zero, and right everywhere else."""
    x = delta_inputs(torch, 2, 140, 1, 2, D, D, dt, gates, seed=72)
    cleared = torch.zeros(2, 140, 2, dtype=torch.bool, device="cuda")
    cleared[0, [0, 17, 63, 64, 139]] = True
    cleared[1, 30:50, 1] = True
    x["g"] = torch.where(cleared, torch.full_like(x["g"], -float("inf")), x["g"])
    x["g"][0, 64] = -300.0
    five = [x[n] for n in FIVE]
    _, _, carries, errors = qs.quat_delta_fwd_carries(*five, x["init"])
    d_g = qs.quat_delta_bwd(*five, carries, errors, x["d_o"], x["d_final"])[3]
    assert (d_g[cleared] == 0).all()
    n = {k: wide(v) for k, v in x.items()}
    want = np.stack([ref.delta_grad(*[n[k][b] for k in FIVE], n["init"][b], D ** -0.5, n["d_o"][b], n["d_final"][b])[3] for b in range(2)])
    for h in range(2):
        close(d_g[..., h], want[..., h], gates, h)


# ---------------------------------------------------------------------------
# Products of fp32 precision.
# ---------------------------------------------------------------------------
BITS = [0x3f80ffff, 0x3f8080ff, 0x3fffffff, 0x3fff7fff, 0x3f817fff, 0x3faa5555]


@pytest.mark.parametrize("low", BITS)
@pytest.mark.parametrize("D", [64, 128])
def test_delta_products_keep_fp32(torch, D, low):  # noqa: F811
    """One step from the zero state: the final state is k v^T, one product per value, like signs and low bits set.

    Tolerance: with these bits the pairs of terms left out are below 0.3 * 2^-24 of the product
    (terms that are cut off, not rounded: up to 7.9), the sum of the others is cut off by at most
    2^-23 when the first terms' product comes (and by 2^-8 of that before), and the state rounds
    once, 2^-24: under 4 * 2^-24 together.
    """
    value = float(np.array(low, np.uint32).view(np.float32))
    full = lambda *s: torch.full(s, value, device="cuda")  # noqa: E731
    k, v = full(1, 1, 1, D), full(1, 1, 1, D)
    v[..., ::2] *= -1
    g, beta = torch.zeros(1, 1, 1, device="cuda"), torch.ones(1, 1, 1, device="cuda")
    _, fin = qs.quat_delta_fwd(k, k, v, g, beta)
    want = wide(k)[0, 0, 0][:, None] * wide(v)[0, 0, 0][None]
    assert (np.abs(wide(fin)[0, 0] - want) <= 4 * 2.0 ** -24 * np.abs(want)).all(), np.abs(wide(fin)[0, 0] / want - 1).max() * 2 ** 24


# ---------------------------------------------------------------------------
# The layer.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("B,S", [(1, 70), (1, 1), (3, 1)])
def test_layer_cache_of_one_sequence(torch, B, S):  # noqa: F811
    """Tokens after a prefill neither write into its graph nor keep its rotations."""
    from quaternion_cumulative_product_gb300.layer import QuatDeltaMixer
    torch.manual_seed(81)
    layer = QuatDeltaMixer(96, 2, 64, groups=2, dtype=torch.float32)
    x = torch.randn(B, S + 2, 96, device="cuda")
    y, cache = layer(x[:, :S])
    assert cache.turn.untyped_storage().nbytes() == cache.turn.numel() * 4
    tokens = [layer.step(x[:, t : t + 1], cache) for t in (S, S + 1)]
    y.square().sum().backward()
    assert all(torch.isfinite(p.grad).all() for p in layer.parameters())
    with torch.no_grad():
        whole, end = layer(x)
    assert (torch.cat([y.detach(), *tokens], 1) - whole).abs().max() <= 1e-4 * whole.abs().max()   # the scan's tolerance
    assert (cache.state - end.state).abs().max() <= 1e-4 * end.state.abs().max()


# ---------------------------------------------------------------------------
# Inputs that are views, heads that are none, streams.
# ---------------------------------------------------------------------------
def test_delta_expanded_keys(torch):  # noqa: F811
    """Queries and keys that all heads or all sequences share, as expanded views in fp32."""
    x = delta_inputs(torch, 2, 130, 2, 4, 64, 64, "f32", "f32", seed=91)
    views = dict(x, q=x["q"][:1].expand(2, -1, -1, -1), k=x["k"][:, :, :1].expand(-1, -1, 2, -1), v=x["v"][:, :1].expand(-1, 130, -1, -1))
    whole = {n: t.contiguous() for n, t in views.items()}
    out = []
    for y in (views, whole):
        five = [y[n] for n in FIVE]
        o, fin, carries, errors = qs.quat_delta_fwd_carries(*five, y["init"])
        out.append([o, fin, *qs.quat_delta_bwd(*five, carries, errors, y["d_o"], y["d_final"])])
    assert all(torch.equal(a, b) for a, b in zip(*out))
    with pytest.raises(ValueError, match="k is an expanded view"):   # bfloat16 rows come by tensor maps
        qs.quat_delta_fwd(*[whole[n].bfloat16() if n != "k" else x["k"].bfloat16()[:, :, :1].expand(-1, -1, 2, -1) for n in FIVE])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_autograd_delta_takes_expanded_inputs(torch, dt):  # noqa: F811
    """A broadcast input's gradient is the sum over its copies."""
    from quaternion_cumulative_product_gb300 import autograd as ag
    x = delta_inputs(torch, 2, 100, 1, 2, 64, 64, dt, "f32", seed=92)
    k = x["k"][:1].clone().requires_grad_()
    full = x["k"][:1].repeat(2, 1, 1, 1).requires_grad_()
    grads = []
    for leaf, key in ((k, k.expand(2, -1, -1, -1)), (full, full)):
        o, _ = ag.quat_delta(x["q"], key, x["v"], x["g"], x["beta"])
        grads.append(torch.autograd.grad(o, leaf, x["d_o"])[0])
    want = grads[1].float().sum(0, keepdim=True)
    assert (grads[0].float() - want).abs().max() <= TOL[dt] * want.abs().max()


def test_delta_gradients_without_value_heads(torch):  # noqa: F811
    """No value head uses the keys: their gradients are zero, not whatever the memory held."""
    B, S, Hk, D = 1, 37, 2, 64
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    q = torch.randn(B, S, Hk, D, device="cuda")
    stale = [torch.full_like(q, float("nan")) for _ in range(4)]
    del stale   # (the allocator hands this memory out again)
    d = qs.quat_delta_bwd(q, q, e(B, S, 0, D), e(B, S, 0), e(B, S, 0), e(B, 1, 0, D, D), e(B, S, 0, D), e(B, S, 0, D))
    assert (d[0] == 0).all() and (d[1] == 0).all()
    assert d[2].shape == (B, S, 0, D) and d[5].shape == (B, 0, D, D)


def test_outputs_belong_to_the_call_s_stream(torch):  # noqa: F811
    """Outputs made for a call on another stream come from that stream's memory: dropped early, they are not handed
    out to work on the current stream while the call may still write them."""
    def owner(t):
        at, = [seg for seg in torch.cuda.memory_snapshot() if 0 <= t.data_ptr() - seg["address"] < seg["total_size"]]
        return at["stream"]

    x = delta_inputs(torch, 1, 200, 2, 2, 64, 64, "bf16", "f32", seed=93)
    y = rotate_inputs(torch, 1, 200, 2, 2, 2, 64, 16, "bf16", "f32", False, seed=93)
    five, s = [x[n] for n in FIVE], torch.cuda.Stream()
    states = [x["init"].clone(), x["init"].clone()]
    s.wait_stream(torch.cuda.current_stream())
    calls = [lambda st: qs.quat_delta_fwd(*five, x["init"], stream=st)[0], lambda st: qs.quat_norm_rotate_fwd(y["q"], y["k"], y["cum"], stream=st)[0],
             lambda st: qs.quat_delta_step(*five, states[st is not None], stream=st)]
    for call in calls:
        want = call(None)
        torch.cuda.synchronize()
        out = call(s)
        s.synchronize()
        assert torch.equal(out, want)
        assert owner(out) == s.cuda_stream and owner(want) == torch.cuda.current_stream().cuda_stream
