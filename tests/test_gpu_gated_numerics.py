"""Gated experts (moe_glu_*) where a rounding, a tail or a NaN counts (GPU).

Tolerances, from the arithmetic:

g and u between the passes: 32 columns of a row as fp16 where they fit it.  The first of the 32
is the nearest of the odd codes, so within a step: 2^-24 below 2^-14.  A code of at most 8
bits is exact in bf16, so du = dh f(g) of such a g shows it as it was kept.
"""
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


def unit_experts(E, H, gate, up=1.0):
    """x with ones in columns 0 and 1; Wg's first two rows `gate` [E, 2, H] and Wu's first `up`; W2 and dy so
    that y = h and dh = 1."""
    M = 64
    x = torch.zeros(E, 1, M, dtype=torch.bfloat16, device="cuda")
    x[:, :, :2] = 1.0
    W13 = torch.zeros(E, M, 2 * H, dtype=torch.bfloat16, device="cuda")
    W13[:, :2, :H] = gate.bfloat16()
    W13[:, 0, H:] = up
    W2 = torch.eye(H, M, dtype=torch.bfloat16, device="cuda").expand(E, H, M).contiguous()
    n = torch.ones(E, dtype=torch.int32, device="cuda")
    return x, W13, W2, n


def in_capacity(t, C):
    out = torch.full((t.shape[0], C, t.shape[2]), float("nan"), dtype=t.dtype, device="cuda")
    out[:, :1] = t
    return out


@PATHS
@pytest.mark.parametrize("rest", [0.45, 1.55])
def test_first_of_32_small_gates_is_kept_within_a_step(C, rest):
    """fp16's subnormal range: g = (2k + rest) 2^-24 in column 0, 1 in the other 31."""
    E, step = 32, 2.0**-24
    codes = 128 + 4 * torch.arange(E, device="cuda")
    gate = torch.zeros(E, 2, 64, device="cuda")
    gate[:, 0] = 1.0
    whole = int(rest)
    gate[:, 0, 0], gate[:, 1, 0] = (codes + whole) * step, (rest - whole) * step
    x, W13, W2, n = unit_experts(E, 64, gate)
    x = in_capacity(x, C)
    ex = experts(C, W13, W2, "relu")
    ex(x, n)
    du = ex.backward(x, n, torch.ones_like(x))["dW13"][:, 0, 64].double()
    want = W13[:, 0, 0].double() + W13[:, 1, 0].double()
    assert bool(((du - want).abs() <= step * (1 + 2.0**-10)).all()), float(((du - want) / step).abs().max())
