"""Gated experts (moe_glu_*) where a rounding, a tail or a NaN counts (GPU).

Tolerances, from the arithmetic:

gelu far below 0: f(g) = g F(g), F the normal distribution.  Its approximation is off by
2^-17.9 of itself; the exponential's argument -g^2 / 2 carries two roundings, 2 * 2^-24 * 40.5
of the result at g = -9, and the hardware exponential 2 + 1.173 * 40.5 units of 2^-23: in all
below 2^-15.  What is stored of it is rounded to bf16 once, 2^-8.

g and u between the passes: 32 columns of a row as fp16 where they fit it.  The first of the 32
is the nearest of the odd codes, so within a step: 2^-24 below 2^-14.  A code of at most 8
bits is exact in bf16, so du = dh f(g) of such a g shows it as it was kept.

Norms in bf16, inputs normal: one rounding of such values is off by 1.65e-3 of their norm.  Two
independent ones (y: h and y; dW2: h and dW2) by 2.34e-3; dx and dW13 (dg and du, the result)
likewise, as g and u in fp16 add 0.2e-3 each; with g and u in bf16 it would be three, 2.9e-3.
The same steps in 64 bits with these roundings give 2.16e-3 to 2.41e-3 (3.0e-3 with g and u in
bf16) over shapes of 5 to 300 rows: bars of 2.6e-3 and 2.7e-3.
"""
from __future__ import annotations

import math

import pytest
import torch

from .test_gpu_glu import act, experts, make

pytestmark = pytest.mark.gpu

PATHS = pytest.mark.parametrize("C", [5, 70], ids=["few rows", "tiles"])
U = torch.finfo(torch.bfloat16).eps / 2


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
def test_gelu_far_below_zero(C):
    """All gates between -5 and -9: h and the gradients through it, relative to their value."""
    gate = torch.zeros(3, 2, 64, device="cuda")
    gate[:, 0] = -torch.linspace(5, 9, 192, device="cuda").view(3, 64)
    x, W13, W2, n = unit_experts(3, 64, gate)
    x = in_capacity(x, C)
    ex = experts(C, W13, W2, "gelu")
    y = ex(x, n)[:, 0].double()
    g = ex.backward(x, n, torch.ones_like(x))
    z = W13[:, 0, :64].double()
    phi = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    cdf = 0.5 * torch.erfc(-z * 0.5**0.5)               # (1 + erf would lose its digits here)
    f, df = z * cdf, cdf + z * phi
    bar = U + 2.0**-15
    assert bool(((y - f).abs() <= bar * f.abs()).all()), float(((y - f) / f).abs().max())
    dW2 = g["dW2"].double()[:, :, 0]                    # h^T dy, dy = 1
    assert bool(((dW2 - f).abs() <= bar * f.abs()).all())
    # g as kept between the passes is exact but for the first of 32
    keep = torch.arange(64, device="cuda") % 32 != 0
    for got, want in ((g["dW13"][:, 0, 64:], f), (g["dW13"][:, 0, :64], df)):
        d = ((got.double() - want).abs() / want.abs())[:, keep]
        assert bool((d <= U + 2.0**-14).all()), float(d.max())


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


@pytest.mark.parametrize("fn", ["silu", "gelu"])
@pytest.mark.parametrize("case", [(16, 8, 256, 512, "few rows"), (3, 70, 256, 512, "tiles"), (2, 300, 128, 320, "tiles of 300")],
                         ids=lambda c: c[4])
def test_norm_of_the_error_is_that_of_its_roundings(case, fn):
    E, C, M, H, _ = case
    x, dy, W13, W2, n = make(E, C, M, H, torch.bfloat16, [C] * E, seed=11)
    ex = experts(C, W13, W2, fn)
    y = ex(x, n)
    g = ex.backward(x, n, dy)
    X, D, Wg, Wu, W = (t.double() for t in (x, dy, W13[:, :, :H], W13[:, :, H:], W2))
    gate, up = X @ Wg, X @ Wu
    f, df = act(fn, gate)
    h, dh = f * up, D @ W.transpose(1, 2)
    dg, du = dh * up * df, dh * f
    want = {"y": h @ W, "dW2": h.transpose(1, 2) @ D, "dx": dg @ Wg.transpose(1, 2) + du @ Wu.transpose(1, 2),
            "dW13": X.transpose(1, 2) @ torch.cat([dg, du], 2)}
    for name, bar in (("y", 2.6e-3), ("dW2", 2.6e-3), ("dx", 2.7e-3), ("dW13", 2.7e-3)):
        got = (y if name == "y" else g[name]).double()
        off = float((got - want[name]).norm() / want[name].norm())
        assert off <= bar, (name, off)
