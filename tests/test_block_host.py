"""The residual block's operators and linear attention with a decay on the host: formulas, refusals, layers (no GPU)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

import block_reference as ref
import quaternion_cumulative_product_gb300 as qs
from quaternion_cumulative_product_gb300 import build as qbuild
from test_mixer_host import at, differences, strides


def test_decay_gradient_by_differences():
    rng = np.random.default_rng(1)
    S, Hk, Hv, Dk, Dv = 5, 1, 2, 3, 2
    q, k, v = (rng.standard_normal(s) for s in ((S, Hk, Dk), (S, Hk, Dk), (S, Hv, Dv)))
    g, init = -rng.random((S, Hv)), rng.standard_normal((Hv, Dk, Dv))
    do, df = rng.standard_normal(v.shape), rng.standard_normal(init.shape)

    def loss():
        o, f = ref.decay(q, k, v, g, init, 0.7)
        return float((o * do).sum() + (f * df).sum())

    for got, leaf in zip(ref.decay_grad(q, k, v, g, init, 0.7, do, df), (q, k, v, g, init)):
        assert np.abs(got - differences(loss, leaf)).max() < 1e-7


def test_layer_norm_gradient_by_differences():
    rng = np.random.default_rng(2)
    x, w, b, dy = rng.standard_normal((3, 7)) + 2, rng.standard_normal(7), rng.standard_normal(7), rng.standard_normal((3, 7))
    loss = lambda: float((ref.layer_norm(x, w, b, 0.1) * dy).sum())  # noqa: E731
    for got, leaf in zip(ref.layer_norm_grad(x, w, 0.1, dy), (x, w, b)):
        assert np.abs(got - differences(loss, leaf)).max() < 1e-7


def test_philox_known_answers():
    """The published test vectors of Philox4x32-10 that a counter (block, offset) can take."""
    words = lambda seed, offset, n: [hex(w) for w in ref.philox_words(seed, offset, n).tolist()]  # noqa: E731
    assert words(0, 0, 4) == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    block = lambda counter, key: _philox(counter, key)  # noqa: E731
    assert block([0xFFFFFFFF] * 4, [0xFFFFFFFF] * 2) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    assert block([0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344], [0xA4093822, 0x299F31D0]) == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]
    assert ref.philox_words(5, 9, 11).tolist() == sum((_philox([i, 0, 9, 0], [5, 0]) for i in range(3)), [])[:11]


def _philox(c, k):
    c, k, low = list(c), list(k), 0xFFFFFFFF
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & low, (a >> 32) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + 0x9E3779B9) & low, (k[1] + 0xBB67AE85) & low]
    return c


# ---------------------------------------------------------------------------
# Refusals of the C entry points: before any CUDA call, with pointers that nobody follows.
# ---------------------------------------------------------------------------
@pytest.fixture(scope="module")
def lib():
    pytest.importorskip("torch")
    qbuild.build()
    from quaternion_cumulative_product_gb300 import block, mixer
    mixer._lib()
    return block._lib()


DECAY = dict(dtype=1, gate=0, scale=1.0, N=2, B=2, S=5, Hk=1, Hv=2, Dk=16, Dv=8)


def decay(lib, call, ptrs=None, st=None, offsets=None, **kw):
    a = dict(DECAY, **kw)
    tail = [a["N"], a["B"], a["S"], a["Hk"], a["Hv"], a["Dk"], a["Dv"], None]
    n = {"fwd": 7, "bwd": 12, "step": 7}[call]
    p = [at(i) for i in range(n)] if ptrs is None else ptrs
    head = [a["dtype"], a["gate"], a["scale"], *p, st]
    if call == "step":
        return lib.quat_decay_step(*head, a["N"] + 1, *[a[x] for x in ("N", "S", "Hk", "Hv", "Dk", "Dv")], None)
    return getattr(lib, "quat_decay_" + call)(*head, offsets, *tail)


@pytest.mark.parametrize("call", ["fwd", "bwd", "step"])
def test_decay_refusals(lib, call):
    for bad in (dict(dtype=2), dict(gate=5), dict(S=-1), dict(S=1 << 31), dict(Hk=0), dict(Hv=3, Hk=2), dict(Dk=12), dict(Dv=136), dict(Dk=-8),
                dict(N=1 << 30, B=1 << 30, Hv=4)):
        assert decay(lib, call, **bad) == qs.QS_ERR_DIMS, bad
    if call != "step":
        assert decay(lib, call, N=3) == qs.QS_ERR_DIMS                      # without offsets as many sequences as the batch
        assert decay(lib, call, offsets=at(30)) == qs.QS_ERR_DIMS           # packed: a batch of one
        assert decay(lib, call, Dk=0) == qs.QS_ERR_DIMS
    n = {"fwd": 7, "bwd": 12, "step": 7}[call]
    may = {"fwd": (4, 6), "bwd": (4, 6, 11), "step": (5,)}[call]            # optional pointers
    for i in range(n):
        p = [at(j) for j in range(n)]
        p[i] = ctypes.c_void_p(p[i].value + 4)
        assert decay(lib, call, p) == qs.QS_ERR_MISALIGNED, i
        p[i] = None
        if i not in may:
            assert decay(lib, call, p) == qs.QS_ERR_NULL, i
    out = {"fwd": 5, "bwd": 7, "step": 6}[call]
    for i in range(3):
        p = [at(j) for j in range(n)]
        p[out] = p[i]
        assert decay(lib, call, p) == qs.QS_ERR_ALIAS
    good = [5 * 16, 16, 16, 5 * 16, 16, 16, 5 * 16, 16, 8]
    for i, bad in ((1, 17), (4, -16), (7, 9)):
        s = list(good)
        s[i] = bad
        assert decay(lib, call, st=strides(*s)) == qs.QS_ERR_MISALIGNED, (i, bad)
    if call != "step":   # bfloat16 rows come by tensor maps: no expanded dimension
        assert decay(lib, call, st=strides(0, *good[1:])) == qs.QS_ERR_MISALIGNED


def test_decay_without_work(lib):
    none = [None] * 7
    assert decay(lib, "fwd", none, N=0, B=0) == qs.QS_OK
    assert decay(lib, "step", none, N=0, B=0) == qs.QS_OK
    assert decay(lib, "bwd", [None] * 12, N=0, B=0) == qs.QS_OK


def norm(lib, bwd, ptrs=None, dtype=1, eps=1e-5, R=4, D=64, ld=64):
    p = [at(i) for i in range(6 if bwd else 4)] if ptrs is None else ptrs
    return (lib.quat_layer_norm_bwd if bwd else lib.quat_layer_norm_fwd)(dtype, eps, *p, R, D, ld, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_layer_norm_refusals(lib, bwd):
    for bad in (dict(dtype=2), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(R=-1), dict(R=1 << 31), dict(D=-1),
                dict(D=qs.QS_NORM_MAX_D + 1), dict(ld=-64), dict(ld=1 << 40)):
        assert norm(lib, bwd, **bad) == qs.QS_ERR_DIMS, bad
    n, need = (6, (0, 2, 3)) if bwd else (4, (0, 3))
    for i in range(n):
        p = [at(j) for j in range(n)]
        p[i] = ctypes.c_void_p(p[i].value + 1)
        assert norm(lib, bwd, p) == qs.QS_ERR_MISALIGNED, i
        p[i] = None
        if i in need:
            assert norm(lib, bwd, p) == qs.QS_ERR_NULL, i
    p = [at(j) for j in range(n)]
    p[3] = p[0]
    assert norm(lib, bwd, p) == qs.QS_ERR_ALIAS
    assert norm(lib, False, [None] * 4, R=0) == qs.QS_OK and norm(lib, True, [None] * 6, D=0) == qs.QS_OK


def test_dropout_refusals(lib):
    fwd = lambda p=0.5, dtype=1, n=8, ptrs=None: lib.quat_dropout_fwd(dtype, p, *(ptrs or [at(i) for i in range(4)]), n, None)  # noqa: E731
    bwd = lambda ptrs: lib.quat_dropout_bwd(1, 0.5, *ptrs, 8, None)  # noqa: E731
    for bad in (dict(p=-0.1), dict(p=1.1), dict(p=float("nan")), dict(dtype=2), dict(n=-1), dict(n=1 << 40)):
        assert fwd(**bad) == qs.QS_ERR_DIMS, bad
    for i in (0, 1, 3):
        p = [at(j) for j in range(4)]
        p[i] = None
        assert fwd(ptrs=p) == qs.QS_ERR_NULL
    for i, m in ((0, 4), (1, 1), (2, 1), (3, 1)):
        p = [at(j) for j in range(4)]
        p[i] = ctypes.c_void_p(p[i].value + m)
        assert fwd(ptrs=p) == qs.QS_ERR_MISALIGNED
    p = [at(0), at(1), at(2), at(2)]
    assert fwd(ptrs=p) == qs.QS_ERR_ALIAS and bwd([at(0), at(1), at(1)]) == qs.QS_ERR_ALIAS
    assert fwd(n=0, ptrs=[None] * 4) == qs.QS_OK


# ---------------------------------------------------------------------------
# Python: checks of tensors, and the layers around plain forms.
# ---------------------------------------------------------------------------
def test_calls_refuse_cpu_tensors(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros(1, 2, 1, 8)
    g = torch.zeros(1, 2, 1)
    for call in (lambda: qs.quat_decay_fwd(x, x, x, g), lambda: qs.quat_decay_bwd(x, x, x, g, x), lambda: qs.quat_decay_step(x, x, x, g, x),
                 lambda: qs.quat_layer_norm_fwd(x), lambda: qs.quat_layer_norm_bwd(x, x), lambda: qs.quat_dropout_fwd(x, g, 0.5), lambda: qs.quat_dropout_bwd(x, g, 0.5)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(TypeError):
        qs.quat_layer_norm_fwd([1.0])


def test_rows_at_one_distance(lib):
    torch = pytest.importorskip("torch")
    from quaternion_cumulative_product_gb300.block import _rows
    x = torch.zeros(3, 4, 10)
    assert _rows(x) == (12, 10, 10) and _rows(x[..., 2:8]) == (12, 6, 10) and _rows(x[1]) == (4, 10, 10)
    assert _rows(x[:, 1:2, 3:]) == (3, 7, 40) and _rows(x[:1].expand(1, 4, 10)) == (4, 10, 10) and _rows(x[0, 0]) == (1, 10, 10)
    assert _rows(x[:1, :1].expand(1, 5, 10)) == (5, 10, 0) and _rows(x[:, :, :0])[1] == 0 and _rows(x[:0])[0] == 0
    for bad in (x[:, 1:3], x.transpose(0, 1), x[..., ::2], x.transpose(1, 2)):
        with pytest.raises(ValueError):
            _rows(bad)


@pytest.fixture
def block(monkeypatch):
    torch = pytest.importorskip("torch")
    import block_plain
    from quaternion_cumulative_product_gb300 import layer
    block_plain.install(monkeypatch, layer)
    torch.manual_seed(0)
    mixer = layer.QuatDecayMixer(32, 2, 8, groups=2, dtype=torch.float32, device="cpu")
    return layer.QuatMixerBlock(mixer, 32, p=0.25, seed=7, device="cpu")


def test_block_tokens_continue_a_prompt(block):
    import torch
    block.eval()
    x = torch.randn(2, 9, 32)
    whole, _ = block(x)
    y, cache = block(x[:, :5])
    rest = [block.step(x[:, t:t + 1], cache) for t in range(5, 9)]
    assert torch.allclose(torch.cat([y, *rest], 1), whole, atol=1e-5)


def test_block_draws_anew_and_stores_its_key(block):
    import torch
    x = torch.randn(1, 4, 32)
    a, b = block(x)[0], block(x)[0]
    assert not torch.equal(a, b) and block.key.tolist() == [7, 2]
    block.key[1] = 0
    assert torch.equal(block(x)[0], a)
    assert "key" in block.state_dict()
    block.eval()
    assert torch.equal(block(x)[0], block(x)[0]) and block.key.tolist() == [7, 1]
