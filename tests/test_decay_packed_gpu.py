"""Packed sequences of linear attention that are cut into segments, against plain 64-bit forms.

Tolerances as in the other tests of linear attention: 256 * 2^-24 normwise in fp32 (at most 256 additions between
two states).
"""
from __future__ import annotations

import numpy as np
import pytest

import block_reference as ref
import quaternion_cumulative_product_gb300 as qs

pytestmark = pytest.mark.gpu
F32 = 256 * 2.0 ** -24


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


def inputs(torch, offsets, Hk, Hv, Dk, Dv, seed=0, behind=0, dtype=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)  # noqa: E731
    S, N, dtype = offsets[-1] + behind, len(offsets) - 1, dtype or torch.float32
    rate = torch.exp(torch.linspace(-5.0, 0.0, Hv, device="cuda"))
    return {"q": unit(rnd(1, S, Hk, Dk)).to(dtype), "k": unit(rnd(1, S, Hk, Dk)).to(dtype), "v": rnd(1, S, Hv, Dv).to(dtype),
            "g": -rate * torch.nn.functional.softplus(rnd(1, S, Hv)), "init": 0.5 * rnd(N, Hv, Dk, Dv),
            "d_o": rnd(1, S, Hv, Dv).to(dtype), "d_final": 0.5 * rnd(N, Hv, Dk, Dv),
            "offsets": torch.tensor(offsets, dtype=torch.int32, device="cuda")}


def run(x):
    o, final = qs.quat_decay_fwd(x["q"], x["k"], x["v"], x["g"], x["init"], offsets=x["offsets"])
    d = qs.quat_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], x["d_final"], x["init"], offsets=x["offsets"])
    return {"o": o, "final": final, **dict(zip(("d_q", "d_k", "d_v", "d_g", "d_init"), d))}


def reference(x, scale):
    w = {n: wide(t) for n, t in x.items() if n != "offsets"}
    offsets = x["offsets"].tolist()
    out = {"o": np.zeros(w["v"].shape), "final": np.zeros(w["init"].shape), **{"d_" + n: np.zeros(w[n].shape) for n in ("q", "k", "v", "g", "init")}}
    for n, (a, b) in enumerate(zip(offsets, offsets[1:])):
        part = [w[m][0, a:b] for m in ("q", "k", "v", "g")]
        out["o"][0, a:b], out["final"][n] = ref.decay(*part, w["init"][n], scale)
        d = ref.decay_grad(*part, w["init"][n], scale, w["d_o"][0, a:b], w["d_final"][n])
        for m, t in zip("qkvg", d):
            out["d_" + m][0, a:b] = t
        out["d_init"][n] = d[4]
    return out


CUTS = [
    [0, 2500],                                              # one, in many segments
    [0, 1030, 1030, 1031, 3000, 3100],                      # long ones, an empty one, short ones
    [0, 0, 1100, 1100],                                     # empty ones first and last
    [0, 512, 1024, 1792, 2561, 3300],                       # exactly a segment, the longest that is whole, one step more
    [*range(0, 149), 1500, 1510, 2800],                     # more than are put in order of length
]


@pytest.mark.parametrize("heads", [(1, 2, 64, 64), (1, 1, 128, 96), (2, 2, 32, 128)], ids=str)
@pytest.mark.parametrize("offsets", CUTS, ids=lambda o: f"{len(o) - 1} of {o[-1]}")
def test_long_sequences(torch, offsets, heads):
    x = inputs(torch, offsets, *heads)
    want = reference(x, heads[2] ** -0.5)
    for name, got in run(x).items():
        assert np.abs(wide(got) - want[name]).max() <= F32 * np.abs(want[name]).max(), name


def test_more_segments_than_run_at_once(torch):
    """Sixteen heads: a segment is longer than the shortest; some sequences are cut, some are not."""
    offsets = [0, 700, 4000, 4100, 4800, 9000]
    x = inputs(torch, offsets, 8, 16, 16, 16, seed=3)
    want = reference(x, 0.25)
    first = run(x)
    for name, got in first.items():
        assert np.abs(wide(got) - want[name]).max() <= F32 * np.abs(want[name]).max(), name
    for name, again in run(x).items():
        assert torch.equal(again, first[name]), name


def test_rows_behind_the_last_sequence(torch):
    """What stands behind the last sequence is not used: the same results, bit for bit, whatever it is."""
    offsets = [0, 1500, 1600]
    x = inputs(torch, offsets, 1, 2, 64, 64, seed=5, behind=130)
    first = run(x)
    for n in ("q", "k", "v", "g", "d_o"):
        x[n][:, offsets[-1]:] = float("nan")
    for name, got in run(x).items():
        rows = slice(None) if name in ("final", "d_init") else slice(0, offsets[-1])
        a, b = (got, first[name]) if name in ("final", "d_init") else (got[:, rows], first[name][:, rows])
        assert torch.equal(a, b), name


def test_bad_values_stay_in_their_sequence(torch):
    offsets = [0, 1100, 2300, 2400]
    x = inputs(torch, offsets, 1, 1, 64, 64, seed=6)
    first = run(x)
    x["v"][0, 1500], x["g"][0, 1700], x["d_o"][0, 1900] = float("nan"), float("inf"), float("-inf")
    for name, got in run(x).items():
        if name in ("final", "d_init"):
            assert torch.equal(got[[0, 2]], first[name][[0, 2]]), name
        else:
            assert torch.equal(got[:, :1100], first[name][:, :1100]) and torch.equal(got[:, 2300:], first[name][:, 2300:]), name


def test_captured_with_other_lengths(torch):
    """The lengths are the device's: a graph replayed with other offsets (and what is then cut) gives their results."""
    x = inputs(torch, [0, 100, 200, 2000], 1, 2, 64, 64, seed=7)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        run(x)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = run(x)
        for offsets in ([0, 1700, 1700, 2000], [0, 600, 1300, 2000]):
            x["offsets"].copy_(torch.tensor(offsets, dtype=torch.int32))
            graph.replay()
            stream.synchronize()
            want = run(x)
            stream.synchronize()
            for name in out:
                assert torch.equal(out[name], want[name]), name


def test_one_sequence_packed_or_not(torch):
    """A single packed sequence against the same as a batch of one: two ways to cut it."""
    x = inputs(torch, [0, 5000], 1, 1, 64, 64, seed=8)
    packed = run(x)
    whole = run({**x, "offsets": None})
    for name in packed:
        a, b = wide(packed[name]), wide(whole[name])
        assert np.abs(a - b).max() <= 2 * F32 * np.abs(b).max(), name


def test_walks_in_order_of_length_repeat(torch):
    """More bfloat16 walks than run at once, the longest first: their order is worked out where the tiles then come,
    and the results are the same every time, and those of the sequences by themselves."""
    offsets = [0, 130, 1430, 1500, 2100, 2101, 3000]
    x = inputs(torch, offsets, 32, 32, 64, 64, seed=9, dtype=torch.bfloat16)
    first = run(x)
    for _ in range(20):
        for name, again in run(x).items():
            assert torch.equal(again, first[name]), name
    a, b = offsets[1:3]
    alone = {n: x[n][:, a:b].contiguous() for n in ("q", "k", "v", "g", "d_o")}
    alone |= {"init": x["init"][1:2].clone(), "d_final": x["d_final"][1:2].clone(), "offsets": torch.tensor([0, b - a], dtype=torch.int32, device="cuda")}
    for name, got in run(alone).items():
        want = first[name][1:2] if name in ("final", "d_init") else first[name][:, a:b]
        assert torch.equal(got, want), name


def test_without_room_for_the_states(torch):
    """In a capture scratch does not grow: without room for the states of a cut, sequences are walked whole, as a call with
    little memory left does, and the results are as near."""
    x = inputs(torch, [0, 1500, 2000], 1, 2, 64, 64, seed=10)
    small = inputs(torch, [0, 20], 1, 1, 64, 64, seed=11)
    forward = lambda x: qs.quat_decay_fwd(x["q"], x["k"], x["v"], x["g"], x["init"], offsets=x["offsets"])  # noqa: E731
    want = reference(x, 64 ** -0.5)
    # Scratch goes with the stream, which torch may hand out again: one of many that has none of this size yet.
    for _ in range(40):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            forward(small)
            stream.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                out = forward(x)
            graph.replay()
            stream.synchronize()
            assert qs.quat_cumprod_status(stream=stream) == qs.QS_OK
        for name, got in zip(("o", "final"), out):
            assert np.abs(wide(got) - want[name]).max() <= F32 * np.abs(want[name]).max(), name
