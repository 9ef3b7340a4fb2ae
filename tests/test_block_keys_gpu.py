"""The residual block's keys on the GPU, with the framework's own operators."""
from __future__ import annotations

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA GPU")
    return torch


def make(torch, **kw):
    from quaternion_cumulative_product_gb300.layer import QuatDecayMixer, QuatMixerBlock
    torch.manual_seed(0)
    return QuatMixerBlock(QuatDecayMixer(128, 2, 64, dtype=torch.bfloat16), 128, p=0.3, **kw)


@pytest.mark.parametrize("reentrant", [False, True])
def test_checkpointing(torch, reentrant):
    from torch.utils.checkpoint import checkpoint
    block = make(torch)
    x, d_y = (torch.randn(2, 150, 128, device="cuda").bfloat16() for _ in range(2))
    x.requires_grad_()
    leaves = [x, *block.parameters()]

    def grads(y):
        for t in leaves:
            t.grad = None
        (y * d_y).sum().backward()
        return [t.grad for t in leaves]

    want = grads(block(x)[0])
    block.key[1] = 0
    got = grads(checkpoint(lambda t, k: block(t, None, k)[0], x, block.next_key(), use_reentrant=reentrant))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    y = checkpoint(lambda t: block(t)[0], x, use_reentrant=reentrant)
    with pytest.raises(RuntimeError, match="next_key"):
        y.sum().backward()
    assert all(torch.equal(a, b) for a, b in zip(grads(checkpoint(lambda t, k: block(t, None, k)[0], x, torch.stack([block.key[0], block.key[1] * 0]),
                                                                  use_reentrant=reentrant)), want))
