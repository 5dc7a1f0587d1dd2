"""What the Python binding takes for a pointer, and what the layer refuses before any device work (CPU)."""
from __future__ import annotations

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from gshard_top_gating_b200 import _lib as L
from gshard_top_gating_b200.layer import MoeLayer


def test_a_pointer_is_a_tensor_an_integer_or_anything_with_data_ptr():
    class Buffer:
        def data_ptr(self):
            return 4096

    t = torch.zeros(3)
    assert L._ptr(t) == t.data_ptr() and L._ptr(None) is None and L._ptr(64) == 64 and L._ptr(Buffer()) == 4096


@pytest.fixture
def gated_layer(monkeypatch):
    """A layer of 4 gated experts without a device: tensors have shapes only, calls are recorded."""
    calls = []
    for name in ("moe_create_gated", "moe_enable_backward", "moe_destroy", "moe_set_backward_flags", "moe_forward", "moe_forward_host",
                 "moe_backward"):
        monkeypatch.setattr(L, name, lambda *a, name=name: calls.append(name) or 1)
    with FakeTensorMode():
        new = lambda *shape, dtype=torch.bfloat16, device="cuda": torch.empty(shape, dtype=dtype, device=device)  # noqa: E731
        layer = MoeLayer(64, 64, 128, 4, 2, 1.25, new(64, 4, dtype=torch.float32), None, new(4, 64, 256), new(4, 128, 64),
                         activation="silu")
        yield layer, new, calls
    layer.h = None


def test_buffers_that_do_not_hold_what_the_kernels_write_are_refused(gated_layer):
    layer, new, calls = gated_layer
    x, dy = new(60, 64), new(60, 64)
    layer(x)
    layer(x, out=new(64, 64))                              # a longer one than x is fine
    layer.backward(x, dy, out={"dW1": new(4, 64, 256), "dW2": new(4 * 128 * 64)})
    assert calls.count("moe_forward") == 2 and calls.count("moe_backward") == 1
    for out in (new(59, 64), new(60, 64, dtype=torch.float32), new(64, 60).t(), new(60, 64, device="cpu")):
        with pytest.raises(ValueError):
            layer(x, out=out)
    for grads in ({"dW1": new(4, 64, 128)},                # a ReLU layer's, half of [Wg | Wu]
                  {"dW1": new(4, 64, 256, dtype=torch.float32)}, {"dW2": new(4, 64, 64)}, {"dx": new(59, 64)},
                  {"dWg": new(64, 4)}, {"dWg": new(4, dtype=torch.float32)}, {"dW2": new(4, 128, 64, device="cpu")}):
        with pytest.raises(ValueError):
            layer.backward(x, dy, out=grads)
    with pytest.raises(ValueError):
        layer.backward(x, new(59, 64))
    with pytest.raises(ValueError):
        layer(new(60, 64, device="cpu"))
    assert calls.count("moe_forward") == 2 and calls.count("moe_backward") == 1
    host = new(60, 64, device="cpu")
    layer.forward_host(host, new(60, 64, device="cpu"))
    for y in (new(59, 64, device="cpu"), new(60, 64, device="cpu", dtype=torch.float32)):
        with pytest.raises(ValueError):
            layer.forward_host(host, y)
    assert calls.count("moe_forward_host") == 1
