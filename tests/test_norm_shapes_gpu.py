"""Layer norm backward of many aligned fp32 rows of up to 512 values: a warp to a row, sixteen rows to a tile.

(The tolerances are those of the other tests of layer norm.)
"""
from __future__ import annotations

import pytest

import quaternion_cumulative_product_gb300 as qs
from test_block_gpu import check_norm, norm_inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA GPU")
    return torch


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("shape", [(5003, 256), (5003, 392), (4900, 512), (4864, 264), (20011, 256)], ids=str)
def test_rows_of_a_warp(torch, shape, weights, dt):
    check_norm(torch, *norm_inputs(torch, shape, dt, weights, seed=shape[0]), dt)


@pytest.mark.parametrize("R,D,right", [(5001, 388, 12), (4999, 512, 4), (5003, 260, 60)])
def test_rows_of_a_warp_apart(torch, R, D, right):
    """Rows that a copy each brings; the last tile is not full."""
    x, w, b, dy = norm_inputs(torch, (R, D + right), "f32", True, seed=R)
    x[:, D:] = float("nan")
    check_norm(torch, x[:, :D], w[:D].clone(), b[:D].clone(), dy[:, :D].contiguous(), "f32")


def test_weights_of_many_tiles_repeat(torch):
    x, w, b, dy = norm_inputs(torch, (30001, 388), "f32", True)
    first = qs.quat_layer_norm_bwd(x, dy, w, b)
    for _ in range(5):
        for a, c in zip(qs.quat_layer_norm_bwd(x, dy, w, b), first):
            assert torch.equal(a, c)
    assert qs.quat_cumprod_status() == qs.QS_OK
