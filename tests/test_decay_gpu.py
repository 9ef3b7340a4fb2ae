"""Linear attention with a decay for each head on the GPU against plain 64-bit forms.

Tolerances, normwise (max |difference| / max |reference|).  A value is built from at most
128 + 128 products added in fp32 between two states (a chunk's steps, a head's values), each
addition off by at most 2^-24 of the running sum: 256 * 2^-24.  d_g of bfloat16 inputs is made of
products that leave out at most 2^-15 on either side of a chunk's state: 2^-14.  A bfloat16 output
is rounded once, 2^-8 at most, and so is one factor of each of its products (P, and the state that a
chunk enters with): where a single product makes the value that is 2^-8 of it once more, 2^-7 in
all.  Where n products of either sign do, their n errors are independent, at most 2^-8 of their
terms and 2^-8 / sqrt(3) of them in the mean square, which is as much of the value's own mean
square: 4.5 deviations of that are 2.6 * 2^-8 of it, less than 2^-8 of the largest of many values
(four deviations).  In the 2-norm the two roundings together are sqrt(2/3) * 2^-8, at most 2^-8.
Two bfloat16 results are apart by twice as much as either from the reference.  References run
on the very inputs the kernels get, widened to 64 bits.
"""
from __future__ import annotations

import numpy as np
import pytest

import block_reference as ref
import quaternion_cumulative_product_gb300 as qs

pytestmark = pytest.mark.gpu
F32 = 256 * 2.0 ** -24
TOL = {"f32": F32, "bf16": 2.0 ** -7 + F32, "two of bf16": 2.0 ** -6 + F32, "gate of bf16": 2.0 ** -14 + F32,
       "gate in bf16": 2.0 ** -8 + 2.0 ** -14 + F32}


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA GPU")
    return torch


@pytest.fixture(autouse=True)
def status(torch):
    """No wait of a kernel has run out."""
    yield
    assert qs.quat_cumprod_status() == qs.QS_OK


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


def close(got, want, tol, what=""):
    assert off(got, want) <= TOL[tol], (what, off(got, want), TOL[tol])
    if tol == "bf16" and want.size >= 1000:
        assert np.linalg.norm(wide(got) - want) <= 2.0 ** -8 * np.linalg.norm(want), what


def inputs(torch, B, S, Hk, Hv, Dk, Dv, dt="bf16", gates="f32", N=None, init=True, seed=0, rate=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    types = {"f32": torch.float32, "bf16": torch.bfloat16}
    dt, ge, N = types[dt], types[gates], B if N is None else N
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    rate = torch.exp(torch.linspace(-4.0, 0.7, Hv, device="cuda")) if rate is None else rate
    return {"q": unit(rnd(B, S, Hk, Dk)).to(dt), "k": unit(rnd(B, S, Hk, Dk)).to(dt), "v": rnd(B, S, Hv, Dv).to(dt),
            "g": (-rate * torch.nn.functional.softplus(rnd(B, S, Hv))).to(ge),
            "init": 0.5 * rnd(N, Hv, Dk, Dv) if init else None,
            "d_o": rnd(B, S, Hv, Dv).to(dt), "d_final": 0.5 * rnd(N, Hv, Dk, Dv)}


def reference(x, scale, offsets=None, grads=True):
    """(o, final, d_q, d_k, d_v, d_g, d_init), sequence by sequence."""
    B, S = x["g"].shape[:2]
    seqs = [(b, 0, S) for b in range(B)] if offsets is None else [(0, a, b) for a, b in zip(offsets, offsets[1:])]
    w = {n: None if t is None else wide(t) for n, t in x.items()}
    out = [np.zeros(w["v"].shape), np.zeros(w["d_final"].shape), *(np.zeros(w[n].shape) for n in ("q", "k", "v", "g")), np.zeros(w["d_final"].shape)]
    for n, (b, lo, hi) in enumerate(seqs):
        part = [w[m][b, lo:hi] for m in ("q", "k", "v", "g")]
        init = np.zeros(w["d_final"].shape[1:]) if w["init"] is None else w["init"][n]
        out[0][b, lo:hi], out[1][n] = ref.decay(*part, init, scale)
        if grads:
            d = ref.decay_grad(*part, init, scale, w["d_o"][b, lo:hi], w["d_final"][n])
            for i in range(4):
                out[2 + i][b, lo:hi] = d[i]
            out[6][n] = d[4]
    return out


def check(torch, x, scale=None, offsets=None, grads=True):
    off_t = None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device="cuda")
    dt = "f32" if x["q"].dtype == torch.float32 else "bf16"
    gates = "gate in bf16" if x["g"].dtype == torch.bfloat16 else "gate of bf16" if dt == "bf16" else "f32"
    want = reference(x, x["q"].shape[-1] ** -0.5 if scale is None else scale, offsets, grads)
    o, final = qs.quat_decay_fwd(x["q"], x["k"], x["v"], x["g"], x["init"], scale=scale, offsets=off_t)
    close(o, want[0], dt, "o")
    close(final, want[1], "f32", "final")
    if not grads:
        return
    d = qs.quat_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], x["d_final"], x["init"], scale=scale, offsets=off_t)
    for got, w, tol, name in zip(d, want[2:], (dt, dt, dt, gates, "f32"), ("d_q", "d_k", "d_v", "d_g", "d_init")):
        close(got, w, tol, name)


SHAPES = [  # B, S, Hk, Hv, Dk, Dv
    (1, 1, 1, 1, 8, 8), (2, 63, 1, 1, 64, 64), (1, 64, 2, 2, 128, 128), (1, 65, 1, 2, 32, 64), (2, 127, 2, 2, 128, 64),
    (1, 128, 1, 1, 128, 128), (1, 129, 2, 4, 128, 128), (3, 40, 2, 2, 16, 120), (1, 300, 1, 2, 96, 80), (2, 257, 2, 2, 64, 64),
    (1, 31, 1, 3, 72, 8), (1, 1300, 1, 1, 128, 128), (1, 1150, 2, 2, 40, 64),
]


@pytest.mark.parametrize("dt,gates", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_decay(torch, shape, dt, gates):
    check(torch, inputs(torch, *shape, dt, gates, init=shape[1] % 2 == 1))


@pytest.mark.parametrize("dt,gates", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("shape", [(1, 2100, 1, 2, 96, 128), (2, 1100, 2, 4, 128, 72), (1, 1700, 1, 1, 64, 24), (3, 1030, 4, 16, 64, 64)], ids=str)
def test_many_chunks(torch, shape, dt, gates):
    """Sequences in many segments, heads of two lengths, and more chunks than CTAs run at once."""
    check(torch, inputs(torch, *shape, dt, gates))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_scale_and_no_decay(torch, dt):
    """g = 0: a plain running sum."""
    x = inputs(torch, 1, 200, 1, 1, 64, 64, dt)
    x["g"].zero_()
    check(torch, x, scale=1.7)


OFFSETS = [[0, 70], [0, 0, 5, 5, 133, 400, 400], [0, 128, 256, 300], [0, 1, 2, 3, 67], list(range(0, 300, 7)) + [300]]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("offsets", OFFSETS, ids=lambda o: str(len(o)) + " to " + str(o[-1]))
def test_packed(torch, offsets, dt):
    check(torch, inputs(torch, 1, offsets[-1], 2, 4, 64, 96, dt, N=len(offsets) - 1), offsets=offsets)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_cleared_states(torch, dt):
    """g = -inf clears the state; far below zero is as good as that; their gradients are exactly zero."""
    x = inputs(torch, 2, 200, 1, 2, 64, 64, dt)
    for t, v in ((0, -np.inf), (60, -np.inf), (64, -1e30), (130, -300.0), (131, -np.inf), (199, -1000.0)):
        x["g"][:, t] = v
    x["g"][1, 3, 1] = -20.0   # a strong decay, whose small gradient is not lost in its neighbours' rounding
    check(torch, x)
    d_g = qs.quat_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], x["d_final"], x["init"])[3]
    assert (d_g[:, [0, 60, 64, 130, 131, 199]] == 0).all()
    want = reference(x, 64 ** -0.5)[5][1, 3, 1]
    assert abs(float(d_g[1, 3, 1]) - want) <= 2.0 ** -8 * np.exp(-20.0) * 64


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_views(torch, dt):
    """q, k and v as slices of one projection, and a batch that is every second row."""
    B, S, H, D = 2, 150, 2, 64
    x = inputs(torch, B, S, H, H, D, D, dt)
    joint = torch.zeros(2 * B, S, 3 * H + 1, D, dtype=x["q"].dtype, device="cuda")
    for i, n in enumerate("qkv"):
        view = joint[::2, :, i * H:(i + 1) * H]
        view.copy_(x[n])
        x[n] = view
    check(torch, x)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_expanded(torch, dt):
    x = inputs(torch, 2, 40, 1, 1, 64, 64, dt)
    x["q"] = x["q"][:1].expand(2, -1, -1, -1)
    if dt == "f32":
        check(torch, x)
    else:
        with pytest.raises(ValueError, match="expanded"):
            qs.quat_decay_fwd(x["q"], x["k"], x["v"], x["g"])


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_bad_values_stay_in_their_sequence(torch, dt, bad):
    offsets = [0, 50, 117, 300]
    x = inputs(torch, 1, 300, 1, 2, 64, 64, dt, N=3)
    clean = {n: t.clone() for n, t in x.items()}
    off_t = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    for n in ("q", "k", "v", "d_o"):
        x[n][0, 60] = bad
    x["g"][0, 61] = float("nan")

    def run(x):
        o, f = qs.quat_decay_fwd(x["q"], x["k"], x["v"], x["g"], x["init"], offsets=off_t)
        d = qs.quat_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], x["d_final"], x["init"], offsets=off_t)
        return o, *d[:4], f, d[4]

    for a, b in zip(run(x)[:5], run(clean)[:5]):
        assert torch.equal(a[0, :50], b[0, :50]) and torch.equal(a[0, 117:], b[0, 117:])
    for a, b in zip(run(x)[5:], run(clean)[5:]):
        assert torch.equal(a[[0, 2]], b[[0, 2]])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_empty(torch, dt):
    x = inputs(torch, 2, 0, 1, 2, 64, 64, dt)
    o, final = qs.quat_decay_fwd(x["q"], x["k"], x["v"], x["g"], x["init"])
    assert o.shape == (2, 0, 2, 64) and torch.equal(final, x["init"])
    assert (qs.quat_decay_fwd(x["q"], x["k"], x["v"], x["g"])[1] == 0).all()
    d = qs.quat_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], x["d_final"], x["init"])
    assert torch.equal(d[4], x["d_final"]) and all(t.numel() == 0 for t in d[:4])
    x = inputs(torch, 0, 10, 1, 2, 64, 64, dt)
    assert qs.quat_decay_fwd(x["q"], x["k"], x["v"], x["g"])[0].shape == (0, 10, 2, 64)
    x = inputs(torch, 1, 10, 2, 2, 64, 64, dt)
    none = {n: t[:, :, :0] for n, t in x.items() if n in ("v", "g", "d_o")}
    d = qs.quat_decay_bwd(x["q"], x["k"], none["v"], none["g"].contiguous(), none["d_o"].contiguous())
    assert (d[0] == 0).all() and (d[1] == 0).all()


def test_no_final_cotangent_and_same_results_twice(torch):
    for dt in ("f32", "bf16"):
        x = inputs(torch, 2, 333, 1, 2, 128, 128, dt)
        run = lambda df: [*qs.quat_decay_fwd(x["q"], x["k"], x["v"], x["g"], x["init"]),  # noqa: E731
                          *qs.quat_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], df, x["init"])]
        first = run(None)
        for a, b in zip(first, run(None)):
            assert torch.equal(a, b)
        for a, b in zip(first, run(torch.zeros_like(x["d_final"]))):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_whole_is_its_parts(torch, dt):
    """A sequence in two calls, the state handed on, and its last steps token by token."""
    x = inputs(torch, 2, 200, 2, 4, 64, 128, dt)
    cut = lambda a, b: [x[n][:, a:b].contiguous() for n in ("q", "k", "v", "g")]  # noqa: E731
    o, final = qs.quat_decay_fwd(*cut(0, 200), x["init"])
    o1, mid = qs.quat_decay_fwd(*cut(0, 131), x["init"])
    o2, end = qs.quat_decay_fwd(*cut(131, 190), mid)
    rest = []
    for t in range(190, 194):
        rest.append(qs.quat_decay_step(*cut(t, t + 1), end))
    rest.append(qs.quat_decay_step(*cut(194, 200), end))
    close(torch.cat([o1, o2, *rest], 1), wide(o), "two of bf16" if dt == "bf16" else dt)
    close(end, wide(final), "f32")


# ---------------------------------------------------------------------------
# Single tokens.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dt,gates", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 8, 8), (5, 1, 2, 4, 128, 128), (3, 4, 1, 1, 64, 40), (9, 3, 2, 2, 72, 128)], ids=str)
def test_step(torch, shape, dt, gates):
    N, T, Hk, Hv, Dk, Dv = shape
    x = inputs(torch, *shape, dt, gates)
    P = N + 3
    pool = torch.randn(P, Hv, Dk, Dv, device="cuda")
    slots = torch.randperm(P, device="cuda")[:N].to(torch.int32)
    if N > 2:
        slots[1], slots[2] = -1, P
    before = pool.clone()
    o = qs.quat_decay_step(x["q"], x["k"], x["v"], x["g"], pool, slots=slots)
    want = wide(before)
    for n, s in enumerate(slots.tolist()):
        if not 0 <= s < P:
            assert (o[n] == 0).all()
            continue
        part, want[s] = ref.decay(*(wide(x[m][n]) for m in ("q", "k", "v", "g")), want[s], Dk ** -0.5)
        close(o[n], part, dt)
    close(pool, want, "f32")
    idle = torch.ones(P, dtype=torch.bool, device="cuda")
    idle[[s for s in slots.tolist() if 0 <= s < P]] = False
    assert torch.equal(pool[idle], before[idle])


def test_captured(torch):
    """Forward, backward and a token in one graph, replayed on new values."""
    x = inputs(torch, 2, 260, 2, 2, 64, 64, "bf16")
    state = torch.zeros(2, 2, 64, 64, device="cuda")
    token = [x[n][:, :1].contiguous() for n in ("q", "k", "v", "g")]

    def run():
        return (*qs.quat_decay_fwd(x["q"], x["k"], x["v"], x["g"], x["init"]),
                *qs.quat_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], x["d_final"], x["init"]),
                qs.quat_decay_step(*token, state))

    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        run()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = run()
        y = inputs(torch, 2, 260, 2, 2, 64, 64, "bf16", seed=5)
        for n in x:
            x[n].copy_(y[n])
        for a, b in zip(token, (x["q"], x["k"], x["v"], x["g"])):
            a.copy_(b[:, :1])
        state.zero_()
        want = run()
        state.zero_()
        graph.replay()
        stream.synchronize()
    for a, b in zip(out, want):
        assert torch.equal(a, b)


def test_another_stream(torch):
    x = inputs(torch, 1, 500, 2, 2, 128, 128, "bf16")
    want = qs.quat_decay_fwd(x["q"], x["k"], x["v"], x["g"], x["init"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = qs.quat_decay_fwd(x["q"], x["k"], x["v"], x["g"], x["init"], stream=s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D", [64, 128])
def test_stall_is_reported(torch, D):
    """Rows that never arrive: every wait runs out its limit, the call reports it, and the next one is clean."""
    lib = qs.load_library()
    x = inputs(torch, 2, 300, 1, 2, D, D, "bf16", seed=31)
    args = (x["q"], x["k"], x["v"], x["g"])
    want = qs.quat_decay_fwd(*args, x["init"])
    back = qs.quat_decay_bwd(*args, x["d_o"], x["d_final"], x["init"])
    try:
        lib.quat_cumprod_debug_set_timeout_ns(20_000_000)
        lib.quat_cumprod_debug_stall_tile(1)
        qs.quat_decay_fwd(*args, x["init"])
        assert qs.quat_cumprod_status() == qs.QS_ERR_TIMEOUT
        qs.quat_decay_bwd(*args, x["d_o"], x["d_final"], x["init"])
        assert qs.quat_cumprod_status() == qs.QS_ERR_TIMEOUT
    finally:
        lib.quat_cumprod_debug_stall_tile(-1)
        lib.quat_cumprod_debug_set_timeout_ns(0)
    for a, b in zip(qs.quat_decay_fwd(*args, x["init"]), want):
        assert torch.equal(a, b)
    for a, b in zip(qs.quat_decay_bwd(*args, x["d_o"], x["d_final"], x["init"]), back):
        assert torch.equal(a, b)


def test_many_packed_sequences(torch):
    """More sequences than are put in order, and more walks than run at once."""
    for N, most in ((150, 9), (60, 40)):
        gen = np.random.default_rng(N)
        offsets = [0, *np.cumsum(gen.integers(0, most, N)).tolist()]
        check(torch, inputs(torch, 1, offsets[-1], 2, 4, 64, 64, "bf16", N=N), offsets=offsets)
    offsets = [0, 700, 710, 1400, 1500, 2700]
    check(torch, inputs(torch, 1, 2700, 1, 32, 16, 16, "bf16", N=5), offsets=offsets)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_rows_behind_the_last_sequence(torch, dt):
    """Packed sequences that end before S: what stands behind them in the outputs stays."""
    import ctypes

    from quaternion_cumulative_product_gb300 import mixer

    S, end, Hk, Hv, D = 420, 333, 2, 4, 64
    x = inputs(torch, 1, S, Hk, Hv, D, D, dt, N=2, seed=17)
    for n in ("q", "k", "v", "d_o"):
        x[n][:, end:] = float("nan")
    offsets = torch.tensor([0, 130, end], dtype=torch.int32, device="cuda")
    sizes = [2, 1, S, Hk, Hv, D, D]
    code = 0 if dt == "f32" else 1
    gate = 0 if x["g"].dtype == torch.float32 else 1
    lib, stream = mixer._lib(), torch.cuda.current_stream().cuda_stream
    o = torch.full_like(x["v"], 7.0)
    final = torch.zeros(2, Hv, D, D, device="cuda")
    p = [ctypes.c_void_p(t.data_ptr()) for t in (x["q"], x["k"], x["v"], x["g"], x["init"])]
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    assert lib.quat_decay_fwd(code, gate, 0.125, *p, ptr(o), ptr(final), None, ptr(offsets), *sizes, stream) == 0
    out = [torch.full_like(x[n], 7.0) for n in ("q", "k", "v", "g")] + [torch.zeros_like(x["init"])]
    assert lib.quat_decay_bwd(code, gate, 0.125, *p, ptr(x["d_o"]), None, *map(ptr, out), None, ptr(offsets), *sizes, stream) == 0
    whole = {n: x[n][:, :end].contiguous() if n in ("q", "k", "v", "g", "d_o") else x[n] for n in x}
    want_o, want_final = qs.quat_decay_fwd(whole["q"], whole["k"], whole["v"], whole["g"], whole["init"], scale=0.125, offsets=offsets)
    want = qs.quat_decay_bwd(whole["q"], whole["k"], whole["v"], whole["g"], whole["d_o"], None, whole["init"], scale=0.125, offsets=offsets)
    assert torch.equal(final, want_final) and torch.equal(out[4], want[4])
    for got, w in zip([o] + out[:4], (want_o, *want[:4])):
        assert torch.equal(got[:, :end], w)
        assert (got[:, end:] == 7.0).all()
