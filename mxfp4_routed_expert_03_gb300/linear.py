"""Buffer bookkeeping around the norm and the dense product in 8 bits of the C ABI.

Holds the tensors whose pointers the library keeps and calls the C entry points;
it computes nothing itself. What the C side cannot see of a tensor (its type, its
length, its device) is checked here and refused with a ValueError; everything else
is left to the C side and its codes.
"""
from __future__ import annotations

import ctypes

import torch

from . import (MOE_LINEAR_BF16, MOE_LINEAR_F32, _stream, lib, moe_fp8_rows, moe_linear_create, moe_linear_desc,
               moe_linear_destroy, moe_linear_status, moe_norm_create, moe_norm_desc, moe_norm_destroy)
from .checks import BITS16, bf16_rows, matrix, on_device

_BITS8 = (torch.float8_e4m3fn, torch.uint8, torch.int8)


class Fp8Rows:
    """Rows of E4M3 codes with a scale per 128 columns; keeps the tensors. q: [T][d]
    (float8_e4m3fn or bytes), s: fp32 [T][ceil(d / 128)]; rows of either may be strided."""

    def __init__(self, q, s):
        if q.dim() != 2 or q.dtype not in _BITS8 or (q.shape[1] > 1 and q.stride(1) != 1):
            raise ValueError("codes: a 2D tensor of E4M3 elements with contiguous rows")
        if (s.dim() != 2 or s.dtype is not torch.float32 or (s.shape[1] > 1 and s.stride(1) != 1)
                or s.shape[0] < q.shape[0] or s.shape[1] * 128 < q.shape[1]):
            raise ValueError("scales: fp32, a row per row of codes, one per 128 columns")
        self.device = q.get_device()
        on_device(self.device, s)
        self.q, self.s = q, s
        self.n, self.width = q.shape
        self.desc = moe_fp8_rows(q.data_ptr(), q.stride(0), s.data_ptr(), s.stride(0))
        self.ref = ctypes.byref(self.desc)

    @classmethod
    def empty(cls, T: int, d: int, device="cuda") -> "Fp8Rows":
        """Uninitialised rows, as Norm.forward fills them."""
        return cls(torch.empty(T, d, dtype=torch.float8_e4m3fn, device=device),
                   torch.empty(T, -(-d // 128), dtype=torch.float32, device=device))

    def check(self, T: int, width: int, device: int) -> None:
        if self.n < T or self.width < width or self.device != device:
            raise ValueError(f"8-bit rows: {T} rows of {width} codes on the handle's device")


class Norm:
    """Residual addition, RMS norm and conversion to 8 bits of rows of d elements. weight: bf16
    [d], or None for no norm. Belongs to the device that is current when it is made."""

    def __init__(self, d: int, eps: float = 1e-6, weight=None):
        self.h = None
        self.d, self.weight = d, weight
        self.device = torch.cuda.current_device()
        if weight is not None:
            if weight.dtype not in BITS16 or weight.numel() < d or not weight.is_contiguous():
                raise ValueError(f"weight: {d} contiguous bf16 elements")
            on_device(self.device, weight)
        self.h = moe_norm_create(moe_norm_desc(d, eps, None if weight is None else weight.data_ptr()))

    def close(self):
        if self.h:
            moe_norm_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, T, x, residual=None, total=None, y=None, y8: Fp8Rows | None = None, stream=None) -> int:
        """total: x + residual; y: the norm of that in bf16; y8: in 8 bits (each may be left out)."""
        dev, d = self.device, self.d
        x, xs = bf16_rows(x, T, d, dev)
        residual, rs = bf16_rows(residual, T, d, dev)
        total, ts = bf16_rows(total, T, d, dev)
        y, ys = bf16_rows(y, T, d, dev)
        if y8 is not None:
            y8.check(T, d, dev)
            y8 = y8.ref
        return lib().moe_add_norm(self.h, T, x, xs, residual, rs, total, ts, y, ys, y8, _stream(stream))


class Linear:
    """A projection with E4M3 weights: w_q [d_out][d_in] codes, w_s fp32 [ceil(d_out / 128)]
    [ceil(d_in / 128)]. The tensors are kept; their contents may change between calls. Belongs
    to the device that is current when it is made, where the weights are."""

    def __init__(self, d_in: int, d_out: int, w_q, w_s):
        self.h = None
        self.d_in, self.d_out = d_in, d_out
        self.device = torch.cuda.current_device()
        matrix(w_q, d_out, d_in, _BITS8, "w_q")
        matrix(w_s, -(-d_out // 128), -(-d_in // 128), (torch.float32,), "w_s")
        on_device(self.device, w_q, w_s)
        self.w_q, self.w_s = w_q, w_s
        self.h = moe_linear_create(moe_linear_desc(d_in, d_out), w_q, w_s)

    def close(self):
        if self.h:
            moe_linear_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def forward(self, T, x: Fp8Rows, out, stream=None) -> int:
        """out: [T][d_out] in bf16 or fp32 (rows may be strided)."""
        dev = self.device
        if x is not None:
            x.check(T, self.d_in, dev)
            x = x.ref
        if out is not None and out.dtype is torch.float32:
            if out.dim() != 2 or out.stride(1) != 1 or out.shape[0] < T or out.shape[1] < self.d_out:
                raise ValueError(f"out: {T} contiguous rows of {self.d_out} elements")
            on_device(dev, out)
            kind, ptr, stride = MOE_LINEAR_F32, out.data_ptr(), out.stride(0)
        else:
            kind, (ptr, stride) = MOE_LINEAR_BF16, bf16_rows(out, T, self.d_out, dev)
        return lib().moe_linear_forward(self.h, T, x, ptr, stride, kind, _stream(stream))

    def status(self, stream=None) -> int:
        return moe_linear_status(self.h, stream)
