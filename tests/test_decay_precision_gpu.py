"""How exact linear attention with a decay is: element by element, and where a shorter term would show.

bfloat16 outputs (o, d_q, d_k, d_v) are one sum, out_t = scale sum_s D_ts <x_t, y_s> z_s, in chunks of
C = 128 steps with the state M between them: out = f x M + P z.  P and M are carried in two
bfloat16 terms, which leave out at most 2^-17 of them; the sums are fp32, at most 256
additions of at most 2^-24 of the terms' absolute sum between two states; and the output is
rounded once, by 2^-8 of itself.  So each element is within

    2^-8 |out| + 2^-16 (sum |P| |z| + |f x| |M|) + 2^-16 sum D |x|.|y| |z|

of its value (2^-16: twice 2^-17, for the two factors f and D, that are exp2 of rounded sums).  One term of P
or M leaves out up to 2^-8, many times that where the output's terms cancel.

d_g with fp32 gates has three terms of M.  With states of one value c = 1 + 2^-8 - 2^-17 - 2^-22, of which two terms leave
out 2^-17 - 2^-22, with rows that pick one element of the state, and without decays, d_g_t is a sum of
equal terms scale c, each exact up to one rounding, added up in at most 16 roundings: 2^-20 of it.
"""
from __future__ import annotations

import numpy as np
import pytest

import block_reference as ref
import quaternion_cumulative_product_gb300 as qs

pytestmark = pytest.mark.gpu
C = 128


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA GPU")
    return torch


def one_sum(x, y, z, g, first, scale):
    """(out, sum |P||z| + |f x||M|, sum D |x|.|y| |z|) of x, y [S,K], z [S,V], g [S], first [K,V]."""
    out, kept, whole = np.zeros(z.shape), np.zeros(z.shape), np.zeros(z.shape)
    state, total = first, np.abs(first)
    for a in range(0, len(x), C):
        X, Y, Z, G = x[a:a + C], y[a:a + C], z[a:a + C], np.cumsum(g[a:a + C])
        D = np.tril(np.exp(np.minimum(G[:, None] - G[None], 0.0)))
        P, f, h = scale * D * (X @ Y.T), scale * np.exp(G)[:, None], np.exp(G[-1] - G)[:, None]
        out[a:a + C] = P @ Z + (f * X) @ state
        kept[a:a + C] = np.abs(P) @ np.abs(Z) + np.abs(f * X) @ np.abs(state)
        whole[a:a + C] = scale * D * (np.abs(X) @ np.abs(Y).T) @ np.abs(Z) + np.abs(f * X) @ total
        state, total = np.exp(G[-1]) * state + (h * Y).T @ Z, np.exp(G[-1]) * total + np.abs(h * Y).T @ np.abs(Z)
    return out, kept, whole


def four_sums(q, k, v, g, init, d_o, d_final, scale):
    """o, d_q, d_k, d_v of one head, each with its two sums (backward in time: the same, turned round)."""
    turn, back = np.concatenate([[0.0], g[:0:-1]]), lambda r: tuple(t[::-1] for t in r)
    forward = one_sum(q, k, v, g, init, scale), one_sum(d_o, v, k, g, init.T, scale)
    # (out's factor of the last state is exp(G_C - G_t) alone)
    d_k = back(one_sum(v[::-1], d_o[::-1], q[::-1], turn, d_final.T / scale, scale))
    d_v = back(one_sum(k[::-1], q[::-1], d_o[::-1], turn, d_final / scale, scale))
    return *forward, d_k, d_v


def bound(s):
    return 2.0 ** -8 * np.abs(s[0]) + 2.0 ** -16 * (s[1] + s[2])


def wide(t):
    return t.detach().double().cpu().numpy()


def inputs(torch, B, S, H, Dk, Dv, seed, gates=None):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).bfloat16()  # noqa: E731
    rate = torch.exp(torch.linspace(-5.0, 0.0, H, device="cuda"))
    g = (-rate * torch.nn.functional.softplus(rnd(B, S, H))).to(gates or torch.float32)
    return {"q": unit(rnd(B, S, H, Dk)), "k": unit(rnd(B, S, H, Dk)), "v": rnd(B, S, H, Dv).bfloat16(), "g": g,
            "init": 0.5 * rnd(B, H, Dk, Dv), "d_o": rnd(B, S, H, Dv).bfloat16(), "d_final": 0.5 * rnd(B, H, Dk, Dv)}


@pytest.mark.parametrize("shape", [(1, 128, 2, 128, 128), (2, 384, 2, 64, 64), (1, 384, 3, 128, 128), (1, 256, 2, 32, 96), (1, 1536, 1, 64, 64)], ids=str)
@pytest.mark.parametrize("gates", ["f32", "bf16"])
def test_each_element(torch, shape, gates):
    """The last shape is cut into segments.  (S is whole chunks: they are the same from either end.)"""
    x = inputs(torch, *shape, seed=shape[1], gates=torch.bfloat16 if gates == "bf16" else None)
    scale = shape[3] ** -0.5
    o = qs.quat_decay_fwd(x["q"], x["k"], x["v"], x["g"], x["init"])[0]
    d = qs.quat_decay_bwd(x["q"], x["k"], x["v"], x["g"], x["d_o"], x["d_final"], x["init"])
    assert qs.quat_cumprod_status() == qs.QS_OK
    w = {n: wide(t) for n, t in x.items()}
    for b in range(shape[0]):
        for h in range(shape[2]):
            part = [w[n][b, :, h] for n in ("q", "k", "v", "g")]
            sums = four_sums(*part, w["init"][b, h], w["d_o"][b, :, h], w["d_final"][b, h], scale)
            for name, got, s in zip(("o", "d_q", "d_k", "d_v"), (o, *d[:3]), sums):
                over = np.abs(wide(got)[b, :, h] - s[0]) / bound(s)
                assert over.max() <= 1, (name, over.max())


def test_the_sums_are_those_of_the_steps(torch):
    """The formulas above against the recurrence, step by step."""
    w = {n: wide(t) for n, t in inputs(torch, 1, 200, 1, 8, 16, seed=1).items()}
    part = [w[n][0] for n in ("q", "k", "v", "g")]
    o, _ = ref.decay(*part, w["init"][0], 0.3)
    d = ref.decay_grad(*part, w["init"][0], 0.3, w["d_o"][0], w["d_final"][0])
    sums = four_sums(*[p[:, 0] for p in part], w["init"][0, 0], w["d_o"][0, :, 0], w["d_final"][0, 0], 0.3)
    for s, want in zip(sums, (o, *d[:3])):
        assert np.abs(s[0] - want[:, 0]).max() <= 1e-10


@pytest.mark.parametrize("D", [64, 128])
def test_gates_gradient_has_three_terms_of_the_state(torch, D):
    c, S = 1 + 2.0 ** -8 - 2.0 ** -17 - 2.0 ** -22, 300
    ones = torch.full((1, 1, D, D), c, device="cuda")
    assert float(ones[0, 0, 0, 0]) == c
    pick = torch.zeros(1, S, 1, D, device="cuda", dtype=torch.bfloat16)
    pick[0, torch.arange(S), 0, torch.arange(S) * 7 % D] = 1
    none, g = torch.zeros_like(pick), torch.zeros(1, S, 1, device="cuda")
    scale = 0.125
    # d_g_t = sum over r >= t of <q_r, M do_r> = scale c, M = init throughout
    d_g = wide(qs.quat_decay_bwd(pick, none, none, g, pick, None, ones, scale=scale)[3])[0, :, 0]
    want = scale * c * (S - np.arange(S))
    assert (np.abs(d_g - want) <= 2.0 ** -20 * want).all(), np.abs(d_g / want - 1).max()
    # d_g_t = sum over s < t of <k_s, dM v_s> = c, dM = d_final throughout
    d_g = wide(qs.quat_decay_bwd(none, pick, pick, g, none, ones, None, scale=scale)[3])[0, :, 0]
    want = c * np.arange(S)
    assert (np.abs(d_g - want) <= 2.0 ** -20 * want).all(), np.abs(d_g[1:] / want[1:] - 1).max()


def test_decay_of_long_segments(torch):
    """An initial state alone, decayed over 1024 chunks in many segments: exp(sum of g) of it.  A segment's decay comes from
    the sum of its log decays, kept in two floats: the total's rounding in base-2 units (2^-24 of 24 at most), and in each of at most
    64 segments and, in the last, 1024 / 2 chunks an exp2 (2^-22) and a product (2^-24)."""
    S = 131072
    g = torch.full((1, S, 1), -1.3e-4, device="cuda")
    zero = torch.zeros(1, S, 1, 64, device="cuda", dtype=torch.bfloat16)
    init = torch.ones(1, 1, 64, 64, device="cuda")
    _, final = qs.quat_decay_fwd(zero, zero, zero, g, init)
    want = np.exp(g.double().sum().item())
    assert np.abs(wide(final) / want - 1).max() <= 24 * 2.0 ** -24 + (64 + 512) * (2.0 ** -22 + 2.0 ** -24)
