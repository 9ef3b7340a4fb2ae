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


def test_limit_of_waits_is_a_kernels_own(torch):
    """A walk of one long packed sequence takes many times the limit of a wait, and the next walk, started early, waits
    for it: none of the waits inside either is long, and none is reported.  (2^19 steps: 4096 chunks of at least 2 us a walk,
    8 ms; a limit of 2 ms.)"""
    S = 1 << 19
    gen = torch.Generator(device="cuda").manual_seed(0)
    q, k, v, d_o = (torch.randn(1, S, 1, 64, generator=gen, device="cuda").bfloat16() for _ in range(4))
    g = -torch.rand(1, S, 1, generator=gen, device="cuda")
    offsets = torch.tensor([0, S], dtype=torch.int32, device="cuda")
    args = (q, k, v, g, d_o)
    want = qs.quat_decay_bwd(*args, offsets=offsets)
    assert qs.quat_cumprod_status() == qs.QS_OK
    lib = qs.load_library()
    try:
        lib.quat_cumprod_debug_set_timeout_ns(2_000_000)
        got = qs.quat_decay_bwd(*args, offsets=offsets)
        torch.cuda.synchronize()
    finally:
        lib.quat_cumprod_debug_set_timeout_ns(0)
    assert qs.quat_cumprod_status() == qs.QS_OK
    for a, b in zip(got, want):
        assert torch.equal(a, b)
