"""Checks of tensors whose pointers go to the C entry points, which see neither type nor length."""
from __future__ import annotations

import torch

BITS16 = (torch.bfloat16, torch.int16, torch.uint16)  # bf16, or its bit patterns


def rows(t, n: int, width: int):
    """Pointer and row stride of n token rows of `width` bf16 elements, or their bit patterns ((None, 0) for None)."""
    if t is None:
        return None, 0
    try:
        (stride, one), (have, cols) = t.stride(), t.shape
    except ValueError:
        one = 0  # not 2D
    if one != 1:
        raise ValueError("token rows: a 2D tensor with contiguous rows")
    if have < n or cols < width or t.dtype not in BITS16:
        raise ValueError(f"token rows: {n} rows of {width} bf16 elements")
    return t.data_ptr(), stride


def bf16_rows(t, n: int, width: int, device: int):
    """As rows, on CUDA device `device`."""
    if t is not None and t.get_device() != device:
        raise ValueError(f"token rows: on the handle's device cuda:{device}")
    return rows(t, n, width)


def flat(t, n: int, dtype, what: str):
    """Pointer of t (a tensor, a pointer or None) once it is known to hold n contiguous elements."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype is not dtype or t.numel() < n or not t.is_contiguous():
        raise ValueError(f"{what}: {n} contiguous elements of {dtype}")
    return t.data_ptr()


def matrix(t, n: int, width: int, dtypes, what: str) -> None:
    """Refuses what is not a contiguous matrix of n rows of `width` elements by its shape (more rows, rows in
    several dimensions, dimensions of 1 and all of it in one dimension are fine)."""
    shape = [s for s in t.shape if s != 1]
    if (t.dtype not in dtypes or not t.is_contiguous() or t.numel() < n * width
            or (len(shape) > 1 and shape[-1] != width and width > 1)):
        raise ValueError(f"{what}: [{n}][{width}] contiguous elements of {dtypes[0]}")


def on_device(index: int, *tensors) -> None:
    """Refuses tensors that are not on CUDA device `index` (pointers and None are left alone)."""
    for t in tensors:
        if t is not None and t.__class__ is not int and t.get_device() != index:
            raise ValueError(f"a tensor on {t.device}: not on the handle's device cuda:{index}")
