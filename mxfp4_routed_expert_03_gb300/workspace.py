"""Scratch buffers of an object's calls."""
from __future__ import annotations

import ctypes

import torch


def handle(stream) -> int:
    """The stream's handle, 0 for the default stream (None)."""
    return 0 if stream is None else stream if isinstance(stream, int) else stream.cuda_stream


def _on(stream: int, device):
    """Context in which `stream` is the current stream."""
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device) if stream
                             else torch.cuda.default_stream(device))


def _capturing(stream: int) -> bool:
    """Whether a graph is being captured on the stream (which need not be the current one)."""
    if stream == 1:  # (the default stream by its other name)
        return False
    from . import lib
    status = ctypes.c_int(0)
    query = lib().cudaStreamIsCapturing  # (the CUDA runtime, which the library is linked with)
    return query(ctypes.c_void_p(stream), ctypes.byref(status)) != 0 or status.value != 0


def empty_on(n: int, stream, device) -> torch.Tensor:
    """n bytes that belong to `stream` in torch's allocator."""
    with _on(handle(stream), device):
        return torch.empty(n, dtype=torch.uint8, device=device)


class Workspace:
    """A buffer per stream, so that calls on two streams share none, grown as calls need. A
    buffer belongs to its stream in torch's allocator, which hands freed memory on only in that
    stream's order; one that a captured graph may hold is kept as long as this object."""

    def __init__(self, device="cuda"):
        self.device = device
        self.bufs = {}         # by stream handle
        self._captured = set()  # streams whose buffer a graph may hold
        self._kept = []

    def get(self, n: int, stream=None) -> torch.Tensor:
        """At least n bytes for a call on `stream`."""
        key = handle(stream)
        buf = self.bufs.get(key)
        if buf is None or buf.numel() < n:
            if key in self._captured:
                self._captured.discard(key)
                self._kept.append(buf)
            buf = self.bufs[key] = empty_on(max(n, 256), key, self.device)
        if key and _capturing(key):  # (the default stream cannot be captured)
            self._captured.add(key)
        return buf
