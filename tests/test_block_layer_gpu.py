"""The operators of a residual block together, as a program uses them: autograd forms, the block, captured training."""
from __future__ import annotations

import numpy as np
import pytest

import quaternion_cumulative_product_gb300 as qs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA GPU")
    return torch


def make(torch, dtype, p=0.0, width=64, heads=2, dim=32, groups=2, seed=0):
    from quaternion_cumulative_product_gb300.layer import QuatDecayMixer, QuatMixerBlock
    torch.manual_seed(seed)
    return QuatMixerBlock(QuatDecayMixer(width, heads, dim, groups, dtype=dtype), width, p=p, seed=3)


def wide_copy(torch, monkeypatch, block, p):
    """The same block on the CPU in 64 bits, around plain forms."""
    import block_plain
    from quaternion_cumulative_product_gb300 import layer
    block_plain.install(monkeypatch, layer)
    mixer = layer.QuatDecayMixer(64, 2, 32, 2, dtype=torch.float64, device="cpu")
    other = layer.QuatMixerBlock(mixer, 64, p=p, seed=3, device="cpu").double()
    other.load_state_dict({n: t.cpu() if n == "key" else t.double().cpu() for n, t in block.state_dict().items()})
    # The layer computes its gates and turns in 32 bits, where it says float().
    monkeypatch.setattr(torch.Tensor, "float", lambda t: t.double())
    return other


@pytest.mark.parametrize("p", [0.0, 0.3])
def test_block_and_its_gradients(torch, monkeypatch, p):
    """fp32 throughout: each value is at most a few hundred fp32 operations from the 64-bit one, of which the longest
    sums have 128 terms: 2^-24 * 1024 of the largest value, and of the largest gradient of a tensor, is granted."""
    block = make(torch, torch.float32, p)
    x = torch.randn(2, 37, 64, device="cuda", requires_grad=True)
    dy = torch.randn(2, 37, 64, device="cuda")
    y, cache = block(x)
    (y * dy).sum().backward()
    got = {"x": x.grad, **{n: t.grad for n, t in block.named_parameters()}}
    got = {n: t.double().cpu().numpy() for n, t in got.items()}
    y, state = y.detach().double().cpu(), cache.state.double().cpu()
    block.key[1] = 0
    wide = wide_copy(torch, monkeypatch, block, p)
    xw = x.detach().double().cpu().requires_grad_()
    yw, cw = wide(xw)
    (yw * dy.double().cpu()).sum().backward()
    tol = 1024 * 2.0 ** -24
    assert (y - yw).abs().max() <= tol * yw.abs().max() and (state - cw.state).abs().max() <= tol * cw.state.abs().max()
    want = {"x": xw.grad, **{n: t.grad for n, t in wide.named_parameters()}}
    for n, w in want.items():
        w = w.numpy()
        assert np.abs(got[n] - w).max() <= tol * np.abs(w).max(), n


def test_block_prefill_and_tokens(torch):
    """bfloat16: a value passes about eight roundings of 2^-8, of either way."""
    block = make(torch, torch.bfloat16, width=256, heads=2, dim=128).eval()
    x = torch.randn(3, 150, 256, device="cuda").bfloat16()
    with torch.no_grad():
        whole, _ = block(x)
        y, cache = block(x[:, :147])
        rest = [block.step(x[:, t:t + 1], cache) for t in range(147, 150)]
    got = torch.cat([y, *rest], 1).float()
    assert (got - whole.float()).abs().max() <= 8 * 2.0 ** -8 * whole.float().abs().max()


def test_autograd_forms(torch):
    """Gradients go where they are needed only, cotangents of one output alone are taken, second derivatives refused."""
    from quaternion_cumulative_product_gb300 import autograd as ag
    q, k, v = (torch.randn(2, 70, h, 64, device="cuda").requires_grad_(h == 2) for h in (1, 1, 2))
    g = (-torch.rand(2, 70, 2, device="cuda")).requires_grad_()
    init = torch.randn(2, 2, 64, 64, device="cuda", requires_grad=True)
    o, final = ag.quat_decay(q, k, v, g, init)
    final.sum().backward(retain_graph=True)
    want = qs.quat_decay_bwd(q, k, v, g, torch.zeros_like(o), torch.ones_like(final), init)
    assert q.grad is None and torch.equal(v.grad, want[2]) and torch.equal(g.grad, want[3]) and torch.equal(init.grad, want[4])
    d, = torch.autograd.grad(o.sum(), v, create_graph=True)
    with pytest.raises(RuntimeError):
        d.sum().backward()
    x = torch.randn(6, 8, 96, device="cuda", requires_grad=True)
    w = torch.ones(64, device="cuda", requires_grad=True)
    y = ag.quat_layer_norm(x[:, 2:5, :64], w)          # rows at no single distance: copied
    y.square().sum().backward()
    assert (x.grad[:, 2:5, :64] != 0).any() and (x.grad[:, :, 64:] == 0).all() and w.grad.shape == (64,)
    key = torch.tensor([1, 5], device="cuda")
    x, r = torch.randn(50, 30, device="cuda", requires_grad=True), torch.randn(50, 30, device="cuda", requires_grad=True)
    y = ag.quat_dropout(x, key, 0.4, r)
    key[1] += 1                                         # the backward keeps the key that it had
    y.sum().backward()
    assert torch.equal(x.grad != 0, (y - r).detach() != 0) and (r.grad == 1).all()
    with torch.no_grad():
        assert not ag.quat_dropout(x, key, 0.4).requires_grad


def test_captured_training_step(torch):
    """A whole training step of the block in a graph: the replays draw new masks and match eager steps."""
    from quaternion_cumulative_product_gb300.layer import QuatDecayMixer, QuatMixerBlock

    def fresh():
        torch.manual_seed(1)
        block = QuatMixerBlock(QuatDecayMixer(128, 2, 64, dtype=torch.bfloat16), 128, p=0.2, seed=9)
        return block, torch.randn(2, 140, 128, device="cuda").bfloat16()

    def step(block, x):
        for t in block.parameters():
            t.grad = None
        y, _ = block(x)
        y.float().square().mean().backward()
        return [t.grad for t in block.parameters()]

    block, x = fresh()
    eager = []
    for _ in range(4):
        eager.append([t.clone() for t in step(block, x)])
    del block
    block, x = fresh()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(block, x)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            grads = step(block, x)
        got = []
        for _ in range(3):
            graph.replay()
            got.append([t.clone() for t in grads])
        s.synchronize()
    for a, b in zip(got, eager[1:]):
        for u, w in zip(a, b):
            assert torch.equal(u, w)
    assert not torch.equal(got[0][0], got[1][0])


def test_two_streams_at_once(torch):
    """Calls on two streams, each with its own scratch, do not disturb each other."""
    def call(seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
        q, k, v, d = (rnd(2, 700, 2, 64).bfloat16() for _ in range(4))
        g, x = -torch.rand(2, 700, 2, generator=gen, device="cuda"), rnd(3000, 1024).bfloat16()
        w = rnd(1024)
        return lambda: [*qs.quat_decay_fwd(q, k, v, g), *qs.quat_decay_bwd(q, k, v, g, d), *qs.quat_layer_norm_bwd(x, x, w, w)]

    one, two = call(1), call(2)
    want = [one(), two()]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [None, None]
    for _ in range(3):
        for i, f in enumerate((one, two)):
            with torch.cuda.stream(streams[i]):
                got[i] = f()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for u, w in zip(a, b):
            assert torch.equal(u, w)
