"""8-bit products with a scale for each block of 128 (marshalling only).

    wq, ws = quantize_weights(W)            # W [E, K, N] -> [E, N, K] e4m3, [E, N/128, K/128]
    mm = Fp8Matmul(C_max, wq, ws)           # weights borrowed, as in GatedExperts
    xq, xs = quantize_rows(x)               # [..., K] -> e4m3, [..., K/128]
    y = mm(xq, xs, counts)                  # [E, C, N] bf16; counts int32 [E]

A value stands for q * s of its block: 1 x 128 of a row, 128 x 128 of a weight matrix; a
last block may be cut short.  As with GatedExperts, C chooses the kernels and an Fp8Matmul
runs one call at a time.
"""
from __future__ import annotations

import torch

from . import _lib as L
from .experts import check_tensor, launch_on

BLOCK = 128
E4M3 = torch.float8_e4m3fn
_SOURCES = (torch.bfloat16, torch.float32)


def blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def _source(t, name):
    if t.dtype not in _SOURCES:
        raise TypeError(f"{name} must be float32 or bfloat16")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")


def quantize_rows(x: torch.Tensor, out=None, stream=None):
    """(q, s) of the rows of x [..., K]: q e4m3 like x, s float32 [..., ceil(K/128)]; new
    tensors, or the pair `out`."""
    _source(x, "x")
    shape, device = x.shape, x.device
    if not shape:
        raise ValueError("x must have rows")
    K = shape[-1]
    sshape = (shape[0], (K + 127) // 128) if len(shape) == 2 else (*shape[:-1], blocks(K))
    if out is not None:
        check_tensor("q", out[0], shape, E4M3, device)
        check_tensor("s", out[1], sshape, torch.float32, device)

    def call(st):
        q, s = out if out is not None else (torch.empty(shape, dtype=E4M3, device=device),
                                            torch.empty(sshape, dtype=torch.float32, device=device))
        L.moe_fp8_quantize_rows(x.numel() // K if K else 0, K, x, q, s, st)
        return q, s
    return launch_on(device, stream, (x, *(out or ())), call)


def quantize_weights(W: torch.Tensor, stream=None):
    """(q, s) of expert weights W [E, K, N]: q e4m3 [E, N, K], s float32 [E, ceil(N/128),
    ceil(K/128)]."""
    _source(W, "W")
    if W.dim() != 3:
        raise ValueError("W must be [E, K, N]")
    E, K, N = W.shape

    def call(st):
        q = torch.empty(E, N, K, dtype=E4M3, device=W.device)
        s = torch.empty(E, blocks(N), blocks(K), dtype=torch.float32, device=W.device)
        L.moe_fp8_quantize_weights(E, K, N, W, q, s, st)
        return q, s
    return launch_on(W.device, stream, (W,), call)


class Fp8Matmul:
    """y[e] = (xq * xs)[e] (wq * ws)[e]^T for the rows each expert holds (one moe_fp8_* handle)."""

    def __init__(self, C_max: int, wq: torch.Tensor, ws: torch.Tensor):
        if not wq.is_cuda or wq.dtype != E4M3 or wq.dim() != 3 or not wq.is_contiguous():
            raise ValueError("wq must be a contiguous [E, N, K] CUDA tensor of float8_e4m3fn")
        self.E, self.N, self.K = wq.shape
        self.C_max, self.device = C_max, wq.device
        check_tensor("ws", ws, (self.E, blocks(self.N), blocks(self.K)), torch.float32, self.device)
        self._keep = (wq, ws)
        with torch.cuda.device(self.device):
            self.h = L.moe_fp8_create(self.E, C_max, self.K, self.N, wq, ws)

    def __call__(self, xq: torch.Tensor, xs: torch.Tensor, counts: torch.Tensor, out: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
        """y [E, C, N] bf16 of xq [E, C, K] and xs [E, C, ceil(K/128)].  Rows past counts[e] of
        `out` stay as they are; of a new tensor they are unset."""
        if xq.dim() != 3:
            raise ValueError("xq must be [E, C, K]")
        C = xq.size(1)
        check_tensor("xq", xq, (self.E, C, self.K), E4M3, self.device)
        check_tensor("xs", xs, (self.E, C, blocks(self.K)), torch.float32, self.device)
        check_tensor("counts", counts, (self.E,), torch.int32, self.device)
        if out is not None:
            check_tensor("out", out, (self.E, C, self.N), torch.bfloat16, self.device)

        def call(st):
            y = torch.empty(self.E, C, self.N, dtype=torch.bfloat16, device=self.device) if out is None else out
            L.moe_fp8_matmul(self.h, C, xq, xs, counts, y, st)
            return y
        return launch_on(self.device, stream, (xq, xs, counts, out), call)

    def check(self, stream=None) -> None:
        """Synchronise and raise a pending device error of this handle."""
        launch_on(self.device, stream, (), lambda st: L.moe_fp8_check(self.h, st))

    def close(self) -> None:
        if getattr(self, "h", None):
            with torch.cuda.device(self.device):
                L.moe_fp8_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
