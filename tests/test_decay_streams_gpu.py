"""Linear attention behind other work on its stream: what a call reads has been written, and only its own waits count."""
from __future__ import annotations

import pytest

import quaternion_cumulative_product_gb300 as qs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA GPU")
    return torch


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_without_steps_behind_a_writer(torch, dt):
    """No steps: d_init is d_final and the final state the initial one, as the kernel before has just written them."""
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    q, v = (torch.empty(1, 0, h, 128, device="cuda", dtype=dtype) for h in (1, 4))
    g = torch.empty(1, 0, 4, device="cuda")
    state, more = torch.zeros(1, 4, 128, 128, device="cuda"), torch.randn(4096, 4096, device="cuda")
    got = []
    for i in range(1, 31):
        busy = more @ more                          # keeps the writer waiting, and the call behind it
        state.copy_(busy[0, 0] * 0 + float(i))
        d_init = qs.quat_decay_bwd(q, q, v, g, v, state, state)[4]
        final = qs.quat_decay_fwd(q, q, v, g, state)[1]
        got.append((d_init, final))
    for i, pair in enumerate(got, 1):
        for t in pair:
            assert (t == i).all(), i
