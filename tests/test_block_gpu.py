"""Layer norm and dropout on the GPU against plain 64-bit forms.

Tolerances.  Layer norm, relative to the largest value of a row's result (weights' gradients:
of all): the mean is a sum of D values in fp32, off by at most log2(D) + 16 half ulps of the
largest partial sum (at most 16 values a thread one after the other, then a tree), and so are
the other sums; half an ulp more for each of the ten operations behind them.  With |mean| up
to 4 standard deviations that is (4 * (14 + 16) + (14 + 16) + 10) * 2^-24 < 160 * 2^-24.  The
weights' gradients add up rows (an error of at most R * 2^-24 of the sum of magnitudes for R
rows, far less as it is: sqrt(R) + 16 half ulps of the root of the sum of squares are granted);
a term dy n of d_w brings the error of n = (x - m) r, which is the one above: absolute, 160 * 2^-24
of the row's largest n + 1 however small n itself is, so the terms' errors add up to at most
160 * 2^-24 * sum |dy| (max |n| + 1).  bfloat16 adds its rounding, 2^-8 at most.
Dropout rounds 1 / (1 - p), the product and the sum: three half ulps.
"""
from __future__ import annotations

import numpy as np
import pytest

import block_reference as ref
import quaternion_cumulative_product_gb300 as qs

pytestmark = pytest.mark.gpu
NORM = 160 * 2.0 ** -24
STEP = {"f32": 0.0, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA GPU")
    return torch


def wide(t):
    return t.detach().double().cpu().numpy()


def types(torch, dt):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[dt]


def norm_inputs(torch, shape, dt, weights, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    D = shape[-1]
    x = (rnd(*shape) + 2 * rnd(*shape[:-1], 1).clamp(-2, 2)).to(types(torch, dt))
    return x, 1 + 0.3 * rnd(D) if weights else None, rnd(D) if weights else None, rnd(*shape).to(types(torch, dt))


def check_norm(torch, x, w, b, dy, dt, eps=1e-5):
    X, W, B, DY = (None if t is None else wide(t) for t in (x, w, b, dy))
    y = qs.quat_layer_norm_fwd(x, w, b, eps=eps)
    want = ref.layer_norm(X, W, B, eps)
    assert y.is_contiguous() and y.shape == x.shape and y.dtype == x.dtype
    row = np.abs(want).max(-1, keepdims=True) + 1
    assert (np.abs(wide(y) - want) <= (NORM + STEP[dt]) * row).all()
    d_x, d_w, d_b = qs.quat_layer_norm_bwd(x, dy, w, b, eps=eps)
    w_x, w_w, w_b = ref.layer_norm_grad(X, W, eps, DY)
    # d_x is r times a difference of terms as large as dy w and n: their size, not the difference's, is rounded.
    r = 1 / np.sqrt(X.var(-1, keepdims=True) + eps)
    big = r * (np.abs(DY * (1 if W is None else W)).max(-1, keepdims=True) + 1) * (np.abs(ref.layer_norm(X, None, None, eps)).max(-1, keepdims=True) + 1)
    assert (np.abs(wide(d_x) - w_x) <= NORM * big + STEP[dt] * np.abs(w_x)).all()
    if w is None:
        assert d_w is None and d_b is None
        return
    rows, d = X.reshape(-1, X.shape[-1]), DY.reshape(-1, X.shape[-1])
    n = ref.layer_norm(rows, None, None, eps)
    far = (np.sqrt(len(rows)) + 16) * 2.0 ** -24
    each = NORM * (np.abs(d) * (np.abs(n).max(-1, keepdims=True) + 1)).sum(0)
    assert (np.abs(wide(d_w) - w_w) <= far * np.sqrt((d * n * d * n).sum(0)) + each).all()
    assert (np.abs(wide(d_b) - w_b) <= far * np.sqrt((d * d).sum(0)) + 1e-30).all()


SHAPES = [(1, 1), (3, 2), (5, 7), (2, 3, 32), (1, 2048), (8, 1, 2048), (300, 2048), (17, 1001), (33, 4096), (700, 96), (2, 2, 2, 40),
          (5000, 64), (4, 8192), (3, 8191), (2, 16384), (3, 16383), (9000, 33), (64,), (40, 520), (1300, 1544),
          (5003, 520), (4900, 1024), (2600, 1100), (2451, 2048), (1301, 4096), (650, 8192)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_layer_norm(torch, shape, dt):
    check_norm(torch, *norm_inputs(torch, shape, dt, len(shape) != 2 or shape[0] % 2 == 1 or shape[0] > 100), dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("D,left,right", [(64, 0, 64), (64, 8, 8), (64, 1, 0), (100, 0, 3), (128, 64, 0)])
def test_layer_norm_of_a_slice(torch, dt, D, left, right):
    x, w, b, dy = norm_inputs(torch, (3, 21, left + D + right), dt, True)
    check_norm(torch, x[..., left: left + D], w[left: left + D].clone(), b[left: left + D].clone(), dy[..., :D].contiguous(), dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("R,D,right", [(5001, 520, 80), (2500, 2048, 8)])
def test_layer_norm_of_many_rows_of_a_slice(torch, dt, R, D, right):
    x, w, b, dy = norm_inputs(torch, (R, D + right), dt, True)
    check_norm(torch, x[:, :D], w[:D].clone(), b[:D].clone(), dy[:, :D].contiguous(), dt)


def test_layer_norm_bwd_without_bias_or_weight(torch):
    """Each gradient is made where its parameter is given, whatever else is."""
    for R in (40, 5000):
        x, w, b, dy = norm_inputs(torch, (R, 512), "bf16", True)
        both = qs.quat_layer_norm_bwd(x, dy, w, b)
        one = qs.quat_layer_norm_bwd(x, dy, w)
        assert one[2] is None and torch.equal(one[0], both[0]) and torch.equal(one[1], both[1])
        ones = torch.ones_like(w)
        flat, plain = qs.quat_layer_norm_bwd(x, dy, None, b), qs.quat_layer_norm_bwd(x, dy, ones, b)
        assert flat[1] is None and torch.equal(flat[0], plain[0]) and torch.equal(flat[2], plain[2])
        assert torch.equal(qs.quat_layer_norm_bwd(x, dy)[0], plain[0])


def test_layer_norm_rows_elsewhere(torch):
    x, w, b, dy = norm_inputs(torch, (4, 6, 64), "f32", True)
    check_norm(torch, x[:, ::2], w, b, dy[:, ::2].contiguous(), "f32")          # one distance all the same
    check_norm(torch, x[:1, :1].expand(1, 9, 64), w, b, dy.view(24, 64)[:9].view(1, 9, 64), "f32")
    with pytest.raises(ValueError, match="one distance"):
        qs.quat_layer_norm_fwd(x[:, :4])
    with pytest.raises(ValueError, match="contiguous"):
        qs.quat_layer_norm_fwd(x.transpose(1, 2))
    with pytest.raises(ValueError, match="at most"):
        qs.quat_layer_norm_fwd(torch.zeros(2, qs.QS_NORM_MAX_D + 1, device="cuda"))
    with pytest.raises(TypeError):
        qs.quat_layer_norm_fwd(x.half())
    with pytest.raises(ValueError, match="shape"):
        qs.quat_layer_norm_fwd(x, w[:32])


def test_layer_norm_of_nothing_and_of_nan(torch):
    x, w, b, dy = norm_inputs(torch, (6, 64), "f32", True)
    assert qs.quat_layer_norm_fwd(x[:0], w, b).shape == (0, 64)
    d_x, d_w, d_b = qs.quat_layer_norm_bwd(x[:0], dy[:0], w, b)
    assert d_x.shape == (0, 64) and (d_w == 0).all() and (d_b == 0).all()
    assert qs.quat_layer_norm_fwd(x[:, :0]).shape == (6, 0)
    clean = qs.quat_layer_norm_fwd(x, w, b)
    x[2, 5] = float("nan")
    x[4, 5] = float("inf")
    y = qs.quat_layer_norm_fwd(x, w, b)
    assert torch.equal(y[[0, 1, 3, 5]], clean[[0, 1, 3, 5]]) and y[[2, 4]].isnan().all()
    same = torch.full((2, 64), 3.0, device="cuda")   # no spread: eps alone decides
    assert (qs.quat_layer_norm_fwd(same) == 0).all()


def test_layer_norm_far_from_zero(torch):
    """The squares are summed about the mean: a mean of 1000 deviations costs ten bits, not twenty."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = 1000 + torch.randn(50, 768, generator=gen, device="cuda")
    want = ref.layer_norm(wide(x), None, None, 1e-5)
    assert np.abs(wide(qs.quat_layer_norm_fwd(x)) - want).max() <= 1000 * 30 * 2.0 ** -24 + NORM * 5


def test_layer_norm_bwd_twice_the_same(torch):
    x, w, b, dy = norm_inputs(torch, (5000, 640), "bf16", True)
    for a, c in zip(qs.quat_layer_norm_bwd(x, dy, w, b), qs.quat_layer_norm_bwd(x, dy, w, b)):
        assert torch.equal(a, c)


# ---------------------------------------------------------------------------
# Dropout.
# ---------------------------------------------------------------------------
KEYS = [(0, 0), (12345, 7), (2 ** 62 + 3, 2 ** 40 + 1), (-1, -2)]


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("shape,p", [((1,), 0.5), ((3,), 0.1), ((4, 5), 0.9), ((2, 3, 101), 0.25), ((1, 4096), 0.1), ((5000,), 0.0), ((33,), 1.0), ((4099, 3), 0.5)], ids=str)
def test_dropout(torch, shape, p, dt):
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda: torch.randn(*shape, generator=gen, device="cuda").to(types(torch, dt))  # noqa: E731
    x, res = rnd(), rnd()
    for seed, offset in KEYS:
        key = torch.tensor([seed, offset], device="cuda")
        for r in (None, res):
            got = wide(qs.quat_dropout_fwd(x, key, p, r))
            want = ref.dropout(wide(x), seed % 2 ** 64, offset % 2 ** 64, p, None if r is None else wide(r))
            big = np.abs(wide(x)) / (1 - p if p < 1 else 1) + (0 if r is None else np.abs(wide(r)))
            assert (np.abs(got - want) <= 3 * 2.0 ** -24 * big + STEP[dt] * np.abs(want)).all()
            if r is None:
                assert ((got == 0) == (want == 0)).all()
        assert torch.equal(qs.quat_dropout_bwd(x, key, p), qs.quat_dropout_fwd(x, key, p))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_dropout_alignment_and_dropped_nan(torch, dt):
    key = torch.tensor([5, 6], device="cuda")
    x = torch.randn(1001, device="cuda").to(types(torch, dt))
    res = torch.randn(1001, device="cuda").to(types(torch, dt))
    want = qs.quat_dropout_fwd(x, key, 0.5, res)
    skew = lambda t: torch.cat([t[:1], t])[1:]  # noqa: E731
    assert skew(x).data_ptr() % 16 != 0
    for a, b in ((skew(x), res), (x, skew(res)), (skew(x), skew(res))):
        assert torch.equal(qs.quat_dropout_fwd(a, key, 0.5, b), want)
    y = torch.empty(1002, dtype=x.dtype, device="cuda")[1:]
    assert torch.equal(qs.quat_dropout_fwd(x, key, 0.5, res, y=y), want)
    kept = qs.quat_dropout_fwd(torch.ones_like(x), key, 0.5) != 0
    got = qs.quat_dropout_fwd(torch.full_like(x, float("nan")), key, 0.5, res)
    assert got[kept].isnan().all() and torch.equal(got[~kept], res[~kept])
    assert qs.quat_dropout_fwd(x[:0], key, 0.5).numel() == 0


def test_dropout_share_and_large_offsets(torch):
    """The share that is kept, and other words for other offsets, beyond 2^32 values too."""
    key = torch.tensor([11, 0], device="cuda")
    ones = torch.ones(2 ** 22, dtype=torch.bfloat16, device="cuda")
    for p in (0.1, 0.5):
        share = (qs.quat_dropout_fwd(ones, key, p) == 0).double().mean().item()
        assert abs(share - p) < 6 * np.sqrt(p * (1 - p) / 2 ** 22)   # six deviations of a binomial
    a = qs.quat_dropout_fwd(ones, key, 0.5)
    key[1] += 1
    b = qs.quat_dropout_fwd(ones, key, 0.5)
    assert abs((a == b).double().mean().item() - 0.5) < 6 * 0.5 / 2 ** 11
    long = torch.ones(2 ** 32 + 2 ** 12, dtype=torch.bfloat16, device="cuda")   # counters are element / 4: above 2^30 here
    tail = wide(qs.quat_dropout_fwd(long, key, 0.5)[-8:])
    n = long.numel()
    del long
    c = [(n - 8) // 4, (n - 8) // 4 + 1]
    assert ((tail != 0) == np.concatenate([ref_words(11, 1, i) >= 2 ** 31 for i in c])).all()


def ref_words(seed, offset, block):
    low, c, k = 0xFFFFFFFF, [block & 0xFFFFFFFF, block >> 32, offset, 0], [seed, 0]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & low, (a >> 32) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    return np.array(c, dtype=np.uint64)


def test_dropout_refusals(torch):
    key = torch.tensor([1, 2], device="cuda")
    x = torch.ones(8, 8, device="cuda")
    for p in (-0.1, 1.5, float("nan")):
        with pytest.raises(ValueError):
            qs.quat_dropout_fwd(x, key, p)
    with pytest.raises(TypeError):
        qs.quat_dropout_fwd(x, key.int(), 0.5)
    with pytest.raises(ValueError):
        qs.quat_dropout_fwd(x, key.cpu(), 0.5)
    with pytest.raises(ValueError):
        qs.quat_dropout_fwd(x.t()[:, :4], key, 0.5)
    with pytest.raises(ValueError):
        qs.quat_dropout_fwd(x, key, 0.5, x[:4])
    with pytest.raises(qs.QuatScanError):
        qs.quat_dropout_fwd(x, key, 0.5, y=x)


def test_dropout_captured(torch):
    """A replayed graph draws anew once the offset has been counted up, which the graph may do itself."""
    x, key = torch.ones(4096, device="cuda"), torch.tensor([9, 0], device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        qs.quat_dropout_fwd(x, key, 0.5)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            y = qs.quat_dropout_fwd(x, key, 0.5)
            key[1] += 1
        key[1] = 0
        seen = []
        for _ in range(3):
            graph.replay()
            seen.append(y.clone())
        s.synchronize()
    for i, got in enumerate(seen):
        assert torch.equal(got, qs.quat_dropout_fwd(x, torch.tensor([9, i], device="cuda"), 0.5))


@pytest.mark.parametrize("R", [40, 6000])
def test_layer_norm_bwd_on_threads(torch, R):
    """Rows of different lengths on several host threads at once (the limits of a kernel's shared memory are the process's)."""
    import threading

    widths = (256, 1024, 2000)
    sets = []
    for D in widths:
        gen = torch.Generator(device="cuda").manual_seed(D)
        x, d = (torch.randn(R, D, generator=gen, device="cuda") for _ in range(2))
        w = torch.randn(D, generator=gen, device="cuda")
        sets.append((x, d, w, qs.quat_layer_norm_bwd(x, d, w, w)))
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        x, d, w, want = sets[i]
        with torch.cuda.stream(torch.cuda.Stream()):
            try:
                for _ in range(100):
                    got = qs.quat_layer_norm_bwd(x, d, w, w)
                if not all(torch.equal(a, b) for a, b in zip(got, want)):
                    wrong.append(widths[i])
            except Exception as e:  # noqa: BLE001
                wrong.append((widths[i], repr(e)))

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(widths))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
