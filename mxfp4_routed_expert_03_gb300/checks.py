"""Checks of tensors whose pointers go to the C entry points, which see neither type nor length."""
from __future__ import annotations

import torch


def rows(t, n: int, width: int):
    """Pointer and row stride of n token rows of `width` 16-bit elements ((None, 0) for None)."""
    if t is None:
        return None, 0
    try:
        (stride, one), (have, cols) = t.stride(), t.shape
    except ValueError:
        one = 0  # not 2D
    if one != 1:
        raise ValueError("token rows: a 2D tensor with contiguous rows")
    if have < n or cols < width or t.element_size() != 2:
        raise ValueError(f"token rows: {n} rows of {width} bf16 elements")
    return t.data_ptr(), stride


def flat(t, n: int, dtype, what: str):
    """Pointer of t (a tensor, a pointer or None) once it is known to hold n contiguous elements."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype is not dtype or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{what}: {n} contiguous elements of {dtype}")
    return t.data_ptr()
