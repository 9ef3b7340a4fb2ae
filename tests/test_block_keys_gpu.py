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


@pytest.mark.parametrize("rule", ["QuatDecayMixer", "QuatDeltaMixer"])
def test_block_in_bfloat16(torch, rule):
    """Every parameter in bfloat16: the norms' weights are widened for the operators, whose results are those of the same
    weights in fp32, bit for bit."""
    from quaternion_cumulative_product_gb300 import layer
    torch.manual_seed(0)
    block = layer.QuatMixerBlock(getattr(layer, rule)(128, 2, 64, dtype=torch.bfloat16), 128, p=0.1, seed=1)
    with torch.no_grad():
        for t in block.parameters():
            t.copy_((t + 0.1 * torch.randn_like(t)).bfloat16())   # values that both types hold
    x, d_y = (torch.randn(2, 70, 128, device="cuda").bfloat16() for _ in range(2))
    rate = block.mixer.rate

    def run():
        for t in block.parameters():
            t.grad = None
        block.key[1] = 0
        block.train()
        y, cache = block(x)
        (y * d_y).sum().backward()
        block.eval()
        return [y.detach(), block.step(x[:, :1], cache)], {n: t.grad.float() for n, t in block.named_parameters()}

    with torch.no_grad():
        rate.zero_()   # exp(0): exact in both types
    want, grads = run()
    block.to(torch.bfloat16)
    assert block.w.dtype is torch.bfloat16 and block.key.dtype is torch.int64
    got, small = run()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for n, t in small.items():
        assert torch.equal(t, grads[n].bfloat16().float()) or n == "mixer.rate", n
