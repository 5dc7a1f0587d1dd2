"""Gated experts (moe_glu_*) where a rounding, a tail or a NaN counts (GPU)."""
from __future__ import annotations

import pytest
import torch

from .test_gpu_glu import experts, make

pytestmark = pytest.mark.gpu

PATHS = pytest.mark.parametrize("C", [5, 70], ids=["few rows", "tiles"])


@PATHS
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("fn", ["silu", "gelu", "relu"])
def test_nan_in_one_gate_weight_is_not_lost(fn, dtype, C):
    """A NaN in a column of Wg: g of that column is NaN, u is not."""
    x, dy, W13, W2, n = make(2, C, 128, 192, dtype, [C, C - 1], seed=3)
    j = 37
    W13[0, 11, j] = float("nan")
    ex = experts(C, W13, W2, fn)
    y = ex(x, n, out=torch.zeros_like(x))
    g = ex.backward(x, n, dy, out={"dx": torch.zeros_like(x)})
    assert y[0].isnan().all() and g["dx"][0].isnan().all()
    hit13 = torch.zeros(2 * 192, dtype=torch.bool, device="cuda")
    hit13[[j, 192 + j]] = True
    assert bool((g["dW13"][0].isnan() == hit13[None, :]).all())
    assert bool((g["dW2"][0].isnan() == hit13[:192, None]).all())
    assert not y[1].isnan().any() and not any(t[1].isnan().any() for t in g.values())


def test_nan_in_a_gate_weight_of_experts_in_8_bits():
    """The layer's f(g) u pass: a NaN makes its block of Wg all NaN, u stays finite."""
    from gshard_top_gating_b200.fp8 import quantize_weights
    from gshard_top_gating_b200.inputs import Workload, make_inputs
    from gshard_top_gating_b200.layer import MoeLayer
    w = Workload("case", 60, 128, 256, 1, 1, 1.0, "bf16")
    x, Wg, b, W1, W2 = make_inputs(w, device="cuda")
    W13 = torch.cat([W1, W1], 2).contiguous()
    for fn in ("silu", "gelu", "relu"):
        y = MoeLayer(60, 128, 256, 1, 1, 1.0, Wg, b, quantize_weights(W13), quantize_weights(W2), activation=fn)(x)
        assert y.isfinite().all()
    W13[0, 3, 5] = float("nan")
    for fn in ("silu", "gelu", "relu"):
        y = MoeLayer(60, 128, 256, 1, 1, 1.0, Wg, b, quantize_weights(W13), quantize_weights(W2), activation=fn)(x)
        assert y.isnan().all(), fn
