"""GatedExperts: an owning wrapper around one moe_glu_* handle (marshalling only).

    ex = GatedExperts(C_max, W13, W2, activation="silu")   # W13 [E, M, 2H], W2 [E, H, M]
    y = ex(x, counts)                                       # x [E, C, M], counts int32 [E]
    ex.enable_backward()                                    # training: forwards keep g and u
    g = ex.backward(x, counts, dy)                          # dx, dW13, dW2

Expert e holds the first counts[e] of its C rows; the rows past them are neither read as
data nor written.  Which kernels run goes by C, as the host does not see the counts: keep C
close to the most rows that an expert holds.  The weights are borrowed by the C library; this
object keeps references to them so they outlive the handle.  Its buffers serve all its calls,
graphs captured from it included: one at a time, in the order of one stream.
"""
from __future__ import annotations

import torch

from . import _lib as L

ACTIVATIONS = {"silu": L.MOE_GLU_SILU, "gelu": L.MOE_GLU_GELU, "relu": L.MOE_GLU_RELU}


def check_tensor(name, t, shape, dtype, device) -> None:
    if t.shape != shape or t.dtype != dtype or t.get_device() != device.index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor of {dtype} on {device}, "
                         f"not {tuple(t.shape)} of {t.dtype} on {t.device}")


_current_device, _current_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def launch_on(device, stream, tensors, call):
    """call(raw stream) with the operator's device current and `stream` (default: that device's
    current stream) the one that new tensors are allocated on; tensors of other streams that
    the call uses are recorded on it."""
    if stream is None and _current_device() == device.index:     # the usual call, without contexts
        return call(_current_stream(device.index))
    with torch.cuda.device(device):
        current = torch.cuda.current_stream(device)
        if stream is None:
            stream = current
        elif isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        if stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the operator on {device}")
        with torch.cuda.stream(stream):
            if stream != current:
                for t in tensors:
                    if t is not None:
                        t.record_stream(stream)
            return call(stream.cuda_stream)


class GatedExperts:
    def __init__(self, C_max: int, W13: torch.Tensor, W2: torch.Tensor, activation: str = "silu"):
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
        if W13.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("expert weights must be float32 or bfloat16")
        if not W13.is_cuda or W13.dim() != 3 or W13.shape[2] % 2 or not W13.is_contiguous():
            raise ValueError("W13 must be a contiguous [E, M, 2H] CUDA tensor")
        self.E, self.M, self.H = W13.shape[0], W13.shape[1], W13.shape[2] // 2
        self.C_max, self.act, self.device = C_max, W13.dtype, W13.device
        check_tensor("W2", W2, (self.E, self.H, self.M), self.act, self.device)
        self._keep = (W13, W2)
        with torch.cuda.device(self.device):
            self.h = L.moe_glu_create(self.E, C_max, self.M, self.H, self.act, ACTIVATIONS[activation], W13, W2)

    def _rows(self, name, t, C=None):
        if t.dim() != 3:
            raise ValueError(f"{name} must be [E, C, M]")
        if C is None:
            C = t.shape[1]
        check_tensor(name, t, (self.E, C, self.M), self.act, self.device)
        return C

    def __call__(self, x: torch.Tensor, counts: torch.Tensor, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
        """y [E, C, M]: the experts' outputs for the rows they hold.  The other rows of `out`
        stay as they are; of a new tensor they are unset."""
        C = self._rows("x", x)
        check_tensor("counts", counts, (self.E,), torch.int32, self.device)
        if out is not None:
            self._rows("out", out, C)

        def call(st):
            y = torch.empty_like(x) if out is None else out
            L.moe_glu_forward(self.h, C, x, counts, y, st)
            return y
        return launch_on(self.device, stream, (x, counts, out), call)

    def enable_backward(self) -> None:
        """Allocate the backward's workspace; the forwards that follow keep g and u."""
        with torch.cuda.device(self.device):
            L.moe_glu_enable_backward(self.h)

    def backward(self, x: torch.Tensor, counts: torch.Tensor, dy: torch.Tensor, out: dict | None = None,
                 skip_empty_experts: bool = False, stream=None) -> dict:
        """Gradients dx, dW13, dW2 for the last call (which took x and counts): new tensors, or
        those of `out` (same keys) written in place.  dx has the rows the experts hold; with
        skip_empty_experts the weight gradients of an expert without rows are left as they are."""
        C = self._rows("x", x)
        self._rows("dy", dy, C)
        check_tensor("counts", counts, (self.E,), torch.int32, self.device)
        out = out or {}
        dx, dW13, dW2 = out.get("dx"), out.get("dW13"), out.get("dW2")
        W13, W2 = self._keep
        for name, t, like in (("dx", dx, x), ("dW13", dW13, W13), ("dW2", dW2, W2)):
            if t is not None:
                check_tensor(name, t, like.shape, self.act, self.device)

        def call(st):
            g = {"dx": torch.empty_like(x) if dx is None else dx,
                 "dW13": torch.empty_like(W13) if dW13 is None else dW13,
                 "dW2": torch.empty_like(W2) if dW2 is None else dW2}
            L.moe_glu_backward(self.h, C, x, counts, dy, g["dx"], g["dW13"], g["dW2"],
                               L.MOE_BWD_SKIP_EMPTY_EXPERTS if skip_empty_experts else 0, st)
            return g
        return launch_on(self.device, stream, (x, counts, dy, dx, dW13, dW2), call)

    def check(self, stream=None) -> None:
        """Synchronise and raise a pending device error of this handle."""
        launch_on(self.device, stream, (), lambda st: L.moe_glu_check(self.h, st))

    def close(self) -> None:
        if getattr(self, "h", None):
            with torch.cuda.device(self.device):
                L.moe_glu_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
