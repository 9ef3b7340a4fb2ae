"""The residual block's keys on the CPU, around plain forms: which masks blocks draw, and when they are the same."""
from __future__ import annotations

import pytest


@pytest.fixture
def layer(monkeypatch):
    pytest.importorskip("torch")
    import block_plain
    from quaternion_cumulative_product_gb300 import layer
    block_plain.install(monkeypatch, layer)
    return layer


def stack(layer, n=2, **kw):
    """Blocks of one shape, whose mixers give ones: what a block drops is seen in its output."""
    import torch

    class Ones(torch.nn.Module):
        def forward(self, x, cache):
            return torch.ones_like(x), cache

    return [layer.QuatMixerBlock(Ones(), 16, p=0.5, device="cpu", **kw) for _ in range(n)]


def dropped(block):
    import torch
    return block(torch.zeros(2, 32, 16))[0] == 0


def test_blocks_of_a_stack_drop_different_positions(layer):
    import torch
    a, b = (dropped(block) for block in stack(layer))
    # 1024 positions, half of them dropped in each: half of them alike, 512 of deviation 16.
    assert 512 - 160 < int((a == b).sum()) < 512 + 160
    torch.manual_seed(3)
    first = [dropped(block) for block in stack(layer)]
    torch.manual_seed(3)
    assert all(torch.equal(x, dropped(block)) for x, block in zip(first, stack(layer)))


def test_a_seed_is_taken_as_it_is(layer):
    import torch
    state = torch.get_rng_state()
    a, b = stack(layer, seed=5)
    assert a.key.tolist() == b.key.tolist() == [5, 0] and torch.equal(torch.get_rng_state(), state)
    assert torch.equal(dropped(a), dropped(b))


@pytest.mark.parametrize("reentrant", [False, True])
def test_checkpointing(layer, reentrant):
    """With its key handed in, a forward that runs again gives the gradients of the first; without one it is refused."""
    import torch
    from torch.utils.checkpoint import checkpoint
    torch.manual_seed(0)
    block = layer.QuatMixerBlock(layer.QuatDecayMixer(16, 1, 8, dtype=torch.float32, device="cpu"), 16, p=0.5, seed=7, device="cpu")
    x, d_y = torch.randn(1, 6, 16, requires_grad=True), torch.randn(1, 6, 16)
    leaves = [x, *block.parameters()]

    def grads(y):
        for t in leaves:
            t.grad = None
        (y * d_y).sum().backward()
        return [t.grad for t in leaves]

    want = grads(block(x)[0])
    assert block.key.tolist() == [7, 1]
    block.key[1] = 0
    key = block.next_key()
    assert key.tolist() == [7, 0] and block.key.tolist() == [7, 1]
    got = grads(checkpoint(lambda t, k: block(t, None, k)[0], x, key, use_reentrant=reentrant))
    assert block.key.tolist() == [7, 1] and all(torch.equal(a, b) for a, b in zip(got, want))
    y = checkpoint(lambda t: block(t)[0], x, use_reentrant=reentrant)
    with pytest.raises(RuntimeError, match="next_key"):
        y.sum().backward()
    block.eval()
    y = checkpoint(lambda t: block(t)[0], x, use_reentrant=reentrant)   # nothing is drawn
    y.sum().backward()
