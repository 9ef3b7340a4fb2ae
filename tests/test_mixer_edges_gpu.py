"""The sequence-mixer operators on the GPU at their edges: degenerate arguments, shared scratch, cancellation.

Tolerances are those of ``test_mixer_gpu.py`` (normwise, 192 additions in fp32 and
the output's own rounding) where no other is derived.
"""
from __future__ import annotations

import numpy as np
import pytest

import mixer_reference as ref
import quaternion_cumulative_product_gb300 as qs
from test_mixer_gpu import close, rotate_inputs, torch, wide  # noqa: F401  (torch: the fixture)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# Norm and rotation.
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("size", [1.0, 1e-14])
@pytest.mark.parametrize("dims", [(1, 5, 2, 4, 2, 64, 16), (2, 777, 3, 3, 6, 72, 5), (1, 1, 1, 1, 1, 256, 40)])
@pytest.mark.parametrize("norm", ["rms", "l2"])
def test_norm_rotate_gradients_without_eps(torch, norm, dims, size):  # noqa: F811
    """eps 0, with fewer items than lane groups (their rows count as nothing) and rows whose inverse norm cubed is past fp32."""
    x = rotate_inputs(torch, *dims, "f32", "f32", True, seed=41)
    x["q"], x["k"] = x["q"] * size, x["k"] * size
    d = qs.quat_norm_rotate_bwd(x["q"], x["k"], x["cum"], x["dq"], x["dk"], x["w_q"], x["w_k"], norm=norm, eps=0.0)
    n = {k: wide(v) for k, v in x.items()}
    gq = ref.norm_rotate_grad(n["q"], n["cum"], n["w_q"], norm, 0.0, n["dq"])
    gk = ref.norm_rotate_grad(n["k"], n["cum"], n["w_k"], norm, 0.0, n["dk"])
    for got, want, what in zip(d, (gq[0], gk[0], gq[1] + gk[1], gq[2], gk[2]), ("d_q", "d_k", "d_cum", "d_w_q", "d_w_k")):
        close(got, want, "f32", what)
