"""The sequence-mixer operators on the GPU against plain 64-bit forms.

Tolerances, normwise (max |difference| / max |reference|): a value of these
operators is built from at most 64 + 128 products added in fp32 between two
states (a chunk's 64 steps, a head's 128 values), each addition off by at most
half an ulp, 2^-24 of the running sum: 192 * 2^-24 = 1.15e-5.  bfloat16 outputs
add their one rounding, 2^-8 of the magnitude at most.  References run on the
very inputs the kernels get, widened to 64 bits.
"""
from __future__ import annotations

import numpy as np
import pytest

import mixer_reference as ref
import quaternion_cumulative_product_gb300 as qs

pytestmark = pytest.mark.gpu
TOL = {"f32": 192 * 2.0 ** -24, "bf16": 2.0 ** -8 + 192 * 2.0 ** -24}


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA GPU")
    return torch


def dtype_of(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def wide(t):
    return t.detach().double().cpu().numpy()


def off(got, want):
    got, want = wide(got), np.asarray(want, np.float64)
    assert got.shape == want.shape
    if want.size == 0:
        return 0.0
    scale = np.abs(want).max()
    assert np.isfinite(got).all()
    return np.abs(got - want).max() / (scale if scale > 0 else 1.0)


def close(got, want, dtype, what=""):
    assert off(got, want) <= TOL[dtype], (what, off(got, want))


# ---------------------------------------------------------------------------
# Norm and rotation.
# ---------------------------------------------------------------------------
def rotate_inputs(torch, B, S, H, Hq, Hk, D, J, dt, cum_dt, weights, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    dt, cum_dt = dtype_of(torch, dt), dtype_of(torch, cum_dt)
    return {"q": rnd(B, S, Hq, D).to(dt), "k": (2 * rnd(B, S, Hk, D)).to(dt), "cum": rnd(B, S, H, J, 4).to(cum_dt),
            "w_q": 1 + 0.3 * rnd(D) if weights else None, "w_k": 1 + 0.3 * rnd(D) if weights else None,
            "dq": rnd(B, S, Hq, D).to(dt), "dk": rnd(B, S, Hk, D).to(dt)}


ROTATE = [  # B, S, H, Hq, Hk, D, J
    (1, 1, 1, 1, 1, 8, 2), (2, 5, 2, 4, 2, 64, 16), (1, 67, 3, 3, 6, 128, 32), (2, 33, 1, 8, 1, 96, 16),
    (1, 9, 2, 2, 2, 12, 3), (3, 7, 2, 2, 2, 4, 1), (1, 11, 1, 2, 1, 256, 40), (1, 6, 2, 2, 2, 72, 5),
    (1, 5, 2, 2, 2, 100, 25), (1, 4, 1, 1, 1, 16, 0), (1, 3, 2, 0, 2, 32, 8),
]


@pytest.mark.parametrize("dims", ROTATE)
@pytest.mark.parametrize("dt,cum_dt", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("norm,weights", [("rms", True), ("l2", False)])
def test_norm_rotate(torch, dims, dt, cum_dt, norm, weights):
    x = rotate_inputs(torch, *dims, dt, cum_dt, weights)
    qo, ko = qs.quat_norm_rotate_fwd(x["q"], x["k"], x["cum"], x["w_q"], x["w_k"], norm=norm, eps=1e-5)
    d = qs.quat_norm_rotate_bwd(x["q"], x["k"], x["cum"], x["dq"], x["dk"], x["w_q"], x["w_k"], norm=norm, eps=1e-5)
    assert qs.quat_cumprod_status() == qs.QS_OK
    n = {k: None if v is None else wide(v) for k, v in x.items()}
    close(qo, ref.norm_rotate(n["q"], n["cum"], n["w_q"], norm, 1e-5), dt, "q")
    close(ko, ref.norm_rotate(n["k"], n["cum"], n["w_k"], norm, 1e-5), dt, "k")
    gq = ref.norm_rotate_grad(n["q"], n["cum"], n["w_q"], norm, 1e-5, n["dq"])
    gk = ref.norm_rotate_grad(n["k"], n["cum"], n["w_k"], norm, 1e-5, n["dk"])
    close(d[0], gq[0], dt, "d_q")
    close(d[1], gk[0], dt, "d_k")
    close(d[2], gq[1] + gk[1], cum_dt, "d_cum")
    if weights:
        close(d[3], gq[2], "f32", "d_w_q")
        close(d[4], gk[2], "f32", "d_w_k")
    else:
        assert d[3] is None and d[4] is None


def test_norm_rotate_many_rows_repeat_bitwise(torch):
    """More rows than the persistent backward runs at once; the weights' sums have a fixed order."""
    x = rotate_inputs(torch, 3, 2111, 4, 8, 4, 64, 16, "bf16", "f32", True)
    call = lambda: qs.quat_norm_rotate_bwd(x["q"], x["k"], x["cum"], x["dq"], x["dk"], x["w_q"], x["w_k"])  # noqa: E731
    a, b = call(), call()
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    n = {k: wide(v) for k, v in x.items()}
    gq = ref.norm_rotate_grad(n["q"], n["cum"], n["w_q"], "rms", 1e-6, n["dq"])
    gk = ref.norm_rotate_grad(n["k"], n["cum"], n["w_k"], "rms", 1e-6, n["dk"])
    close(a[0], gq[0], "bf16")
    close(a[2], gq[1] + gk[1], "f32")
    close(a[3], gq[2], "f32")
    close(a[4], gk[2], "f32")


def test_norm_rotate_views_and_stream(torch):
    """q and k as views of one projection, on a stream of its own."""
    B, S, H, D, J = 2, 37, 4, 64, 16
    joint = torch.randn(B, S, 3 * H, D, device="cuda").bfloat16()
    cum = torch.randn(B, S, H, J, 4, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q, k = joint[:, :, :H], joint[:, :, H : 2 * H]
        a = qs.quat_norm_rotate_fwd(q, k, cum)
        b = qs.quat_norm_rotate_fwd(q.contiguous(), k.contiguous(), cum)
    s.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_norm_rotate_relative(torch):
    """Inner products of rotated vectors depend on the rotation between their steps alone."""
    B, S, J = 1, 9, 4
    turn = torch.randn(B, S, 1, J, 4, device="cuda")
    turn = turn / turn.norm(dim=-1, keepdim=True)
    init = [torch.randn(B, 1, J, 4, device="cuda") for _ in range(2)]
    init = [i / i.norm(dim=-1, keepdim=True) for i in init]
    x = torch.randn(B, S, 1, 4 * J, device="cuda")
    dots = []
    for i in init:
        cum = qs.quat_cumprod_fwd(turn, i)
        q, k = qs.quat_norm_rotate_fwd(x, x, cum)
        dots.append(wide(q[0, :, 0] @ k[0, :, 0].T))
    assert np.abs(dots[0] - dots[1]).max() <= 1e-4 * np.abs(dots[0]).max()   # the scan's tolerance


# ---------------------------------------------------------------------------
# The gated delta rule.
# ---------------------------------------------------------------------------
def delta_inputs(torch, B, S, Hk, Hv, Dk, Dv, dt, gates, N=None, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    dt, gates = dtype_of(torch, dt), dtype_of(torch, gates)
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dt)  # noqa: E731
    N = B if N is None else N
    return {"q": unit(rnd(B, S, Hk, Dk)), "k": unit(rnd(B, S, Hk, Dk)), "v": rnd(B, S, Hv, Dv).to(dt),
            "g": (-torch.nn.functional.softplus(rnd(B, S, Hv)) * torch.logspace(-2, 0.3, Hv, device="cuda")).to(gates),
            "beta": torch.sigmoid(rnd(B, S, Hv)).to(gates), "init": 0.3 * rnd(N, Hv, Dk, Dv),
            "d_o": rnd(B, S, Hv, Dv).to(dt), "d_final": rnd(N, Hv, Dk, Dv)}


FIVE = ("q", "k", "v", "g", "beta")


def run_delta(x, init=True, final=True, offsets=None, scale=None):
    five = [x[n] for n in FIVE]
    o, fin, carries, errors = qs.quat_delta_fwd_carries(*five, x["init"] if init else None, offsets=offsets, scale=scale)
    plain = qs.quat_delta_fwd(*five, x["init"] if init else None, offsets=offsets, scale=scale)
    d = qs.quat_delta_bwd(*five, carries, errors, x["d_o"], x["d_final"] if final else None, offsets=offsets, scale=scale)
    assert qs.quat_cumprod_status() == qs.QS_OK
    assert off(plain[0], wide(o)) == 0 and off(plain[1], wide(fin)) == 0
    return o, fin, d


def check_delta(x, dt, gates, init=True, final=True, offsets=None, scale=None):
    o, fin, d = run_delta(x, init, final, offsets, scale)
    n = {k: wide(v) for k, v in x.items()}
    B, S, Hv, Dv = n["v"].shape
    Dk = n["q"].shape[-1]
    scale = Dk ** -0.5 if scale is None else scale
    if offsets is None:
        parts = [(b, 0, S) for b in range(B)]
    else:
        offs = offsets.tolist()
        parts = [(0, a, e) for a, e in zip(offs, offs[1:])]
    want_o, want = np.zeros(n["v"].shape), {k: np.zeros(n[k].shape) for k in FIVE}
    want_fin, want_init = np.zeros(n["init"].shape), np.zeros(n["init"].shape)
    for i, (b, a, e) in enumerate(parts):
        one = [n[k][b, a:e] for k in FIVE]
        m0 = n["init"][i] if init else np.zeros(n["init"][i].shape)
        dfin = n["d_final"][i] if final else np.zeros(m0.shape)
        want_o[b, a:e], want_fin[i] = ref.delta(*one, m0, scale)
        grads = ref.delta_grad(*one, m0, scale, n["d_o"][b, a:e], dfin)
        for k, gr in zip(FIVE, grads):
            want[k][b, a:e] = gr
        want_init[i] = grads[5]
    close(o, want_o, dt, "o")
    close(fin, want_fin, "f32", "final")
    for k, got in zip(FIVE, d):
        close(got, want[k], gates if k in ("g", "beta") else dt, "d_" + k)
    close(d[5], want_init, "f32", "d_init")


DELTA = [  # B, S, Hk, Hv, Dk, Dv
    (1, 1, 1, 1, 64, 64), (2, 63, 2, 2, 64, 64), (1, 64, 1, 2, 128, 128), (2, 65, 2, 4, 128, 64), (1, 130, 1, 1, 8, 8),
    (1, 200, 2, 2, 24, 40), (1, 129, 1, 3, 96, 128), (3, 17, 2, 2, 128, 128), (1, 321, 1, 1, 128, 128), (1, 100, 1, 2, 40, 104),
]


@pytest.mark.parametrize("dims", DELTA)
@pytest.mark.parametrize("dt,gates", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
def test_delta(torch, dims, dt, gates):
    check_delta(delta_inputs(torch, *dims, dt, gates), dt, gates)


@pytest.mark.parametrize("dims", [(1, 1500, 1, 2, 64, 64), (1, 2000, 1, 1, 128, 128), (2, 1290, 1, 1, 128, 40), (1, 1217, 1, 3, 24, 96)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_delta_long_sequences(torch, dims, dt):
    """Few long sequences: cut into segments that are joined (forward and backward)."""
    check_delta(delta_inputs(torch, *dims, dt, "f32", seed=11), dt, "f32")


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_delta_without_states(torch, dt):
    check_delta(delta_inputs(torch, 2, 140, 1, 2, 64, 64, dt, "f32"), dt, "f32", init=False, final=False, scale=0.7)


@pytest.mark.parametrize("lengths", [[0], [5], [0, 64, 0, 1, 63, 65, 0], [130, 128, 2], [1] * 9])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_delta_packed(torch, lengths, dt):
    total = sum(lengths)
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    x = delta_inputs(torch, 1, total, 2, 2, 64, 128, dt, "f32", N=len(lengths), seed=3)
    check_delta(x, dt, "f32", offsets=offsets)


@pytest.mark.parametrize("N", [80, 128, 129])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_delta_packed_many(torch, N, dt):
    """More walks than run at once: equal lengths, empty sequences and long ones in any place."""
    rng = np.random.default_rng(N)
    lengths = rng.choice([0, 1, 7, 64, 65, 200], N)
    lengths[[0, N // 2, N - 1]] = [64, 300, 131]
    lengths[N - 2] += max(0, 130 * N - lengths.sum())
    offsets = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    x = delta_inputs(torch, 1, int(lengths.sum()), 1, 2, 16, 24, dt, "f32", N=N, seed=N)
    check_delta(x, dt, "f32", offsets=offsets)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_delta_extreme_gates(torch, dt):
    """Cleared states (-inf), strong and no decay, beta of zero and one, a zero key."""
    x = delta_inputs(torch, 2, 150, 1, 2, 64, 64, dt, "f32", seed=5)
    x["g"][0, 10], x["g"][0, 64], x["g"][0, 127], x["g"][1, :70], x["g"][1, 80:90] = -float("inf"), -float("inf"), -300.0, 0.0, -40.0
    x["beta"][0, 20:30], x["beta"][1, 60:70] = 0.0, 1.0
    x["k"][0, 40] = 0
    check_delta(x, dt, "f32")


def test_delta_repeated_keys(torch):
    """The same key at every step with beta 1: the triangular system is as ill-behaved as it gets."""
    x = delta_inputs(torch, 1, 128, 1, 1, 64, 64, "f32", "f32", seed=6)
    x["k"] = x["k"][:, :1].expand(-1, 128, -1, -1).contiguous()
    x["beta"].fill_(1.0)
    x["g"].fill_(-1e-3)
    o, fin, _ = run_delta(x)
    n = {k: wide(v) for k, v in x.items()}
    want = ref.delta(*[n[k][0] for k in FIVE], n["init"][0], 64 ** -0.5)
    close(o[0], want[0], "f32")
    close(fin[0], want[1], "f32")


def test_delta_nan_stays_in_its_sequence(torch):
    """A NaN spoils its sequence from the start of its 64-step chunk on, and no other sequence."""
    x = delta_inputs(torch, 1, 192, 1, 2, 64, 64, "bf16", "f32", N=3, seed=7)
    offsets = torch.tensor([0, 50, 100, 192], dtype=torch.int32, device="cuda")
    five = [x[n] for n in FIVE]
    o, fin = qs.quat_delta_fwd(*five, x["init"], offsets=offsets)
    x["v"][0, 60] = float("nan")
    x["k"][0, 70, 0, 3] = float("inf")
    o2, fin2 = qs.quat_delta_fwd(*five, x["init"], offsets=offsets)
    assert torch.equal(o[0, :50], o2[0, :50]) and torch.equal(o[0, 100:], o2[0, 100:])
    assert torch.equal(fin[0], fin2[0]) and torch.equal(fin[2], fin2[2])
    assert torch.isnan(o2[0, 71:100].float()).all() and torch.isnan(fin2[1]).any()


def test_delta_views_repeat_bitwise(torch):
    """q, k and v as views of one projection give the same bits, call after call."""
    B, S, H, D = 2, 150, 2, 64
    joint = torch.randn(B, S, 3 * H, D, device="cuda")
    joint = (joint / joint.norm(dim=-1, keepdim=True)).bfloat16()
    x = delta_inputs(torch, B, S, H, H, D, D, "bf16", "f32")
    views = dict(x, q=joint[:, :, :H], k=joint[:, :, H : 2 * H], v=joint[:, :, 2 * H :])
    whole = {n: t.contiguous() for n, t in views.items()}
    a, b, c = run_delta(views), run_delta(whole), run_delta(whole)
    for s, t, u in zip((a[0], a[1], *a[2]), (b[0], b[1], *b[2]), (c[0], c[1], *c[2])):
        assert torch.equal(s, t) and torch.equal(s, u)


def test_delta_in_a_graph(torch):
    x = delta_inputs(torch, 1, 100, 1, 2, 64, 64, "bf16", "f32")
    five = [x[n] for n in FIVE]

    def step():
        o, fin, carries, errors = qs.quat_delta_fwd_carries(*five, x["init"])
        return [o, fin, *qs.quat_delta_bwd(*five, carries, errors, x["d_o"], x["d_final"])]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()   # sizes the stream's workspace
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    y = delta_inputs(torch, 1, 100, 1, 2, 64, 64, "bf16", "f32", seed=9)
    for n in x:
        x[n].copy_(y[n])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


# ---------------------------------------------------------------------------
# Single tokens.
# ---------------------------------------------------------------------------
STEP = [(1, 1, 1, 1, 64, 64), (5, 1, 2, 4, 128, 128), (3, 4, 1, 2, 96, 40), (2, 3, 2, 2, 8, 8), (4, 2, 1, 1, 24, 104), (2, 70, 1, 1, 128, 64)]


@pytest.mark.parametrize("dims", STEP)
@pytest.mark.parametrize("dt,gates", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
def test_step(torch, dims, dt, gates):
    N, T, Hk, Hv, Dk, Dv = dims
    x = delta_inputs(torch, N, T, Hk, Hv, Dk, Dv, dt, gates)
    pool = torch.full((N + 3, Hv, Dk, Dv), float("nan"), device="cuda")   # slots that no row names hold NaN
    slots = torch.randperm(N + 3, device="cuda")[:N].to(torch.int32)
    pool[slots.long()] = x["init"]
    o = qs.quat_delta_step(*[x[n] for n in FIVE], pool, slots=slots)
    n = {k: wide(v) for k, v in x.items()}
    for i in range(N):
        want_o, want_m = ref.delta(*[n[k][i] for k in FIVE], n["init"][i], Dk ** -0.5)
        close(o[i], want_o, dt, "o")
        close(pool[slots[i].long()], want_m, "f32", "state")
    free = sorted(set(range(N + 3)) - set(slots.tolist()))
    assert torch.isnan(pool[free]).all()


@pytest.mark.parametrize("dims", [(130, 1, 4, 8, 64, 64), (240, 3, 2, 4, 24, 40), (80, 2, 8, 16, 128, 128), (310, 1, 4, 4, 8, 16)])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_step_many_states(torch, dims, dt):
    """Enough states to be streamed through shared memory; some rows idle, the first and the last among them."""
    N, T, Hk, Hv, Dk, Dv = dims
    x = delta_inputs(torch, N, T, Hk, Hv, Dk, Dv, dt, "f32", seed=13)
    slots = torch.randperm(N + 2, device="cuda")[:N].to(torch.int32)
    slots[torch.tensor([0, 5, 6, N - 1], device="cuda")] = torch.tensor([-1, -7, N + 2, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    pool = 0.3 * torch.randn(N + 2, Hv, Dk, Dv, device="cuda")
    before = wide(pool)
    o = qs.quat_delta_step(*[x[n] for n in FIVE], pool, slots=slots)
    assert qs.quat_cumprod_status() == qs.QS_OK
    n, after = {k: wide(v) for k, v in x.items()}, wide(pool)
    want_o, want_pool = np.zeros(n["v"].shape), before.copy()
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < N + 2:
            want_o[i], want_pool[s] = ref.delta(*[n[k][i] for k in FIVE], before[s], Dk ** -0.5)
    close(o, want_o, dt, "o")
    assert np.abs(after - want_pool).max() <= TOL["f32"] * np.abs(want_pool).max()
    untouched = sorted(set(range(N + 2)) - set(slots.tolist()))
    assert (after[untouched] == before[untouched]).all()


def test_step_idle_rows(torch):
    x = delta_inputs(torch, 4, 2, 1, 2, 64, 64, "bf16", "f32")
    x["v"][1] = float("nan")
    pool = x["init"].clone()
    slots = torch.tensor([2, -1, 4, 0], dtype=torch.int32, device="cuda")
    o = qs.quat_delta_step(*[x[n] for n in FIVE], pool, slots=slots)
    assert (o[1] == 0).all() and (o[2] == 0).all()
    assert torch.equal(pool[1], x["init"][1]) and torch.equal(pool[3], x["init"][3])
    assert not torch.equal(pool[2], x["init"][2]) and not torch.equal(pool[0], x["init"][0])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_step_continues_the_sequence(torch, dt):
    """A prefill and then single tokens give what the whole sequence gives."""
    x = delta_inputs(torch, 2, 71, 2, 4, 128, 128, dt, "f32")
    five = [x[n] for n in FIVE]
    whole, last = qs.quat_delta_fwd(*five, x["init"])
    _, state = qs.quat_delta_fwd(*[t[:, :68].contiguous() for t in five], x["init"])
    for t in range(68, 71):
        o = qs.quat_delta_step(*[s[:, t : t + 1].contiguous() for s in five], state)
        close(o[:, 0], wide(whole[:, t]), dt)
    close(state, wide(last), "f32")


def test_zero_sizes(torch):
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    init = torch.randn(2, 1, 8, 8, device="cuda")
    o, fin = qs.quat_delta_fwd(e(2, 0, 1, 8), e(2, 0, 1, 8), e(2, 0, 1, 8), e(2, 0, 1), e(2, 0, 1), init)
    assert o.shape == (2, 0, 1, 8) and torch.equal(fin, init)
    d = qs.quat_delta_bwd(e(2, 0, 1, 8), e(2, 0, 1, 8), e(2, 0, 1, 8), e(2, 0, 1), e(2, 0, 1), e(2, 0, 1, 8, 8),
                          e(2, 0, 1, 8), e(2, 0, 1, 8), init)
    assert torch.equal(d[5], init)
    assert qs.quat_delta_step(e(0, 1, 1, 8), e(0, 1, 1, 8), e(0, 1, 1, 8), e(0, 1, 1), e(0, 1, 1), init).shape == (0, 1, 1, 8)
    q, k = qs.quat_norm_rotate_fwd(e(1, 0, 2, 8), e(1, 0, 2, 8), e(1, 0, 2, 2, 4))
    assert q.shape == (1, 0, 2, 8)
    w = torch.ones(8, device="cuda")
    d = qs.quat_norm_rotate_bwd(e(1, 0, 2, 8), e(1, 0, 2, 8), e(1, 0, 2, 2, 4), q, k, w, w)
    assert (d[3] == 0).all() and (d[4] == 0).all()


# ---------------------------------------------------------------------------
# Autograd, the layer, failures.
# ---------------------------------------------------------------------------
def test_autograd_chain(torch):
    """scan -> rotation -> delta rule through autograd equals the formulas chained by hand."""
    from quaternion_cumulative_product_gb300 import autograd as ag
    B, S, H, Hv, D = 1, 70, 2, 4, 64
    x = delta_inputs(torch, B, S, H, Hv, D, D, "f32", "f32", seed=21)
    turn = torch.randn(B, S, H, D // 4, 4, device="cuda")
    turn = turn / turn.norm(dim=-1, keepdim=True)
    start = turn[:, 0].clone()
    w = 1 + 0.1 * torch.randn(D, device="cuda")
    leaves = [t.clone().requires_grad_() for t in (x["q"], x["k"], x["v"], x["g"], x["beta"], x["init"], turn, start, w)]
    q, k, v, g, beta, init, tu, st, ww = leaves
    cum = ag.quat_cumprod(tu, st)
    qo, ko = ag.quat_norm_rotate(q, k, cum, ww, None, norm="l2")
    o, fin = ag.quat_delta(qo, ko, v, g, beta, init)
    got = torch.autograd.grad([o, fin], leaves, [x["d_o"], x["d_final"]])
    n = [wide(t) for t in (x["q"], x["k"], x["v"], x["g"], x["beta"], x["init"], turn, start, w)]
    c = wide(cum)
    zq, zk = ref.norm_rotate(n[0], c, n[8], "l2", 1e-6), ref.norm_rotate(n[1], c, None, "l2", 1e-6)
    d = ref.delta_grad(zq[0], zk[0], n[2][0], n[3][0], n[4][0], n[5][0], D ** -0.5, wide(x["d_o"])[0], wide(x["d_final"])[0])
    dq, dcq, dw = ref.norm_rotate_grad(n[0], c, n[8], "l2", 1e-6, d[0][None])
    dk, dck, _ = ref.norm_rotate_grad(n[1], c, None, "l2", 1e-6, d[1][None])
    import oracle
    d_turn, d_start = oracle.bwd(n[6], n[7], dcq + dck)
    # Three operators of the tolerance above and the scan's 1e-4 in a row.
    for a, b in zip(got, (dq, dk, d[2][None], d[3][None], d[4][None], d[5][None], d_turn, d_start, dw)):
        assert off(a, b) <= 1e-4 + 3 * TOL["f32"]
    with torch.no_grad():
        o2, fin2 = ag.quat_delta(qo, ko, v, g, beta, init)
    assert torch.equal(o, o2) and torch.equal(fin, fin2)


def test_layer_prefill_and_tokens(torch):
    """The layer's prefill in two parts, then single tokens, gives what one pass over the whole sequence gives."""
    from quaternion_cumulative_product_gb300.layer import QuatDeltaMixer
    torch.manual_seed(5)
    layer = QuatDeltaMixer(96, 2, 64, groups=2, dtype=torch.float32)
    x = torch.randn(3, 90, 96, device="cuda")
    with torch.no_grad():
        whole, end = layer(x)
        first, cache = layer(x[:, :70])
        second, cache = layer(x[:, 70:85], cache)
        tokens = [layer.step(x[:, t : t + 1], cache) for t in range(85, 90)]
    again = torch.cat([first, second, *tokens], 1)
    scale = whole.abs().max()
    assert (again - whole).abs().max() <= 1e-4 * scale   # the scan's tolerance
    assert (cache.state - end.state).abs().max() <= 1e-4 * end.state.abs().max()


def test_layer_learns(torch):
    from quaternion_cumulative_product_gb300.layer import QuatDeltaMixer
    torch.manual_seed(6)
    layer = QuatDeltaMixer(64, 2, 32, groups=1)
    x = torch.randn(4, 80, 64, device="cuda").bfloat16()
    want = torch.roll(x, 1, 1)
    opt = torch.optim.Adam(layer.parameters(), lr=3e-3)
    losses = []
    for _ in range(30):
        loss = (layer(x)[0].float() - want.float()).square().mean()
        opt.zero_grad()
        loss.backward()
        assert all(p.grad is not None and torch.isfinite(p.grad).all() for p in layer.parameters())
        opt.step()
        losses.append(loss.item())
    assert losses[-1] < 0.8 * losses[0]


@pytest.mark.parametrize("D", [64, 128])
def test_delta_stall_is_reported(torch, D):
    """Rows that never arrive: every wait runs out its limit, the call reports it, and the next one is clean."""
    lib = qs.load_library()
    x = delta_inputs(torch, 2, 200, 1, 2, D, D, "bf16", "f32", seed=31)
    five = [x[n] for n in FIVE]
    o, fin, carries, errors = qs.quat_delta_fwd_carries(*five, x["init"])
    try:
        lib.quat_cumprod_debug_set_timeout_ns(20_000_000)
        lib.quat_cumprod_debug_stall_tile(1)
        qs.quat_delta_fwd(*five, x["init"])
        assert qs.quat_cumprod_status() == qs.QS_ERR_TIMEOUT
        qs.quat_delta_bwd(*five, carries, errors, x["d_o"], x["d_final"])
        assert qs.quat_cumprod_status() == qs.QS_ERR_TIMEOUT
    finally:
        lib.quat_cumprod_debug_stall_tile(-1)
        lib.quat_cumprod_debug_set_timeout_ns(0)
    again = qs.quat_delta_fwd(*five, x["init"])
    assert qs.quat_cumprod_status() == qs.QS_OK
    assert torch.equal(again[0], o) and torch.equal(again[1], fin)
