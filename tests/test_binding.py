"""What the Python binding takes for a pointer, and what the layer refuses before any device work (CPU)."""
from __future__ import annotations

import torch

from gshard_top_gating_b200 import _lib as L


def test_a_pointer_is_a_tensor_an_integer_or_anything_with_data_ptr():
    class Buffer:
        def data_ptr(self):
            return 4096

    t = torch.zeros(3)
    assert L._ptr(t) == t.data_ptr() and L._ptr(None) is None and L._ptr(64) == 64 and L._ptr(Buffer()) == 4096
