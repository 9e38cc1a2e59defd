"""Buffer bookkeeping around the attention half of the C ABI.

Holds torch-owned device buffers (the MXFP4 key/value cache, workspace) and
calls the C entry points; it computes nothing itself. Tensors of token rows
may be slices of wider ones (their row stride is passed on).
"""
from __future__ import annotations

import torch

from . import (moe_attn_batch, moe_attn_create, moe_attn_desc, moe_attn_destroy, moe_attn_forward,
               moe_attn_status, moe_attn_workspace_bytes, moe_kv_append, moe_kv_cache, moe_kv_read,
               moe_qk_norm_rope, moe_rope_desc)
from .workspace import Workspace

CACHE_NAMES = ("k_q", "k_s", "v_q", "v_s")


def alloc_kv_cache(n_kv_heads: int, head_dim: int, page_size: int, n_pages: int,
                   device="cuda") -> dict:
    """Zeroed cache arrays (uint8) in the library's layout: all tokens read as 0."""
    z = lambda *shape: torch.zeros(shape, dtype=torch.uint8, device=device)
    nb = head_dim // 32
    return {"k_q": z(n_pages, n_kv_heads, page_size // 8, nb, 8, 16),
            "k_s": z(n_pages, n_kv_heads, page_size, nb),
            "v_q": z(n_pages, n_kv_heads, page_size // 8, nb, 8, 16),
            "v_s": z(n_pages, n_kv_heads, page_size // 2, nb, 2)}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rows(t):
    """Pointer and row stride of a tensor of token rows ((None, 0) for None)."""
    if t is None:
        return None, 0
    s = t.stride()
    if len(s) != 2 or s[1] != 1:
        raise ValueError("token rows: a 2D tensor with contiguous rows")
    return t.data_ptr(), s[0]


class Rope:
    """Norm and rotation parameters; keeps the tensors they point at. cos_sin:
    fp32 [n_pos][rope_dim] (cosines, then sines), or None for no rotation;
    q_weight / k_weight: bf16 [head_dim], or None for no norm."""

    def __init__(self, cos_sin, rope_dim: int, interleaved: bool = False, eps: float = 1e-6,
                 q_weight=None, k_weight=None):
        self.tensors = (cos_sin, q_weight, k_weight)
        n_pos = 0 if cos_sin is None else cos_sin.shape[0]
        self.desc = moe_rope_desc(rope_dim, int(interleaved), n_pos, eps, _ptr(cos_sin),
                                  _ptr(q_weight), _ptr(k_weight))


class Batch:
    """A batch of sequences for Attention.forward; keeps the tensors it points
    at. cu_q: int32 [n_seqs + 1] or None (one query row per sequence); kv_len:
    int32 [n_seqs]; page_table: int32 [n_seqs][pages]; max_q / max_kv bound a
    sequence's query rows and cached tokens."""

    def __init__(self, n_seqs: int, n_tokens: int, max_q: int, max_kv: int, cu_q, kv_len,
                 page_table, scale: float, window: int = 0):
        if page_table is not None and (page_table.dim() != 2 or page_table.stride(1) != 1):
            raise ValueError("page_table: a 2D tensor with contiguous rows")
        self.tensors = (cu_q, kv_len, page_table)
        self.key = (n_seqs, n_tokens, max_q, max_kv)
        stride = 0 if page_table is None else page_table.stride(0)
        self.desc = moe_attn_batch(n_seqs, n_tokens, max_q, max_kv, stride, window, scale,
                                   _ptr(cu_q), _ptr(kv_len), _ptr(page_table))


class Attention:
    """One layer's attention: head shape, the paged MXFP4 cache and the library handle."""

    def __init__(self, n_heads: int, n_kv_heads: int, head_dim: int, page_size: int, n_pages: int,
                 cache: dict):
        self.cache = cache
        self.h = None
        self.desc = moe_attn_desc(n_heads, n_kv_heads, head_dim, page_size, n_pages)
        self.h = moe_attn_create(self.desc, moe_kv_cache(*[cache[n].data_ptr() for n in CACHE_NAMES]))
        self._space = Workspace(cache["k_q"].device)
        self._need = (None, 0)  # the last batch bounds and their workspace bytes

    def close(self):
        if self.h:
            moe_attn_destroy(self.h)
            self.h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def norm_rope(self, T, q, k, positions, rope: Rope, q_out, k_out, stream=None) -> int:
        return moe_qk_norm_rope(self.h, T, rope.desc, positions, *_rows(q), *_rows(k), *_rows(q_out),
                                *_rows(k_out), stream)

    def append(self, T, k, v, slots, stream=None) -> int:
        return moe_kv_append(self.h, T, *_rows(k), *_rows(v), slots, stream)

    def read(self, n, slots, k, v, stream=None) -> int:
        return moe_kv_read(self.h, n, slots, *_rows(k), *_rows(v), stream)

    @property
    def _ws(self):
        """The default stream's buffer."""
        return self._space.bufs.get(0)

    @_ws.setter
    def _ws(self, buf):
        self._space.bufs[0] = buf

    def workspace_bytes(self, batch: Batch) -> int:
        if self._need[0] != batch.key:
            self._need = (batch.key, moe_attn_workspace_bytes(self.h, *batch.key))
        return self._need[1]

    def workspace(self, batch: Batch, stream=None) -> tuple:
        """Scratch of a call on `stream` (each stream has its own; see Workspace) and the bytes it needs."""
        n = self.workspace_bytes(batch)
        return self._space.get(n, stream), n

    def forward(self, batch: Batch, q, out, lse=None, stream=None, ws=None) -> int:
        """ws: the call's own scratch (a tensor of workspace_bytes(batch) or more), for calls that may
        overlap others of the same stream: graphs that were captured on one and run at a time."""
        if ws is None:
            ws, n = self.workspace(batch, stream)
        else:
            n = ws.numel() * ws.element_size()
        return moe_attn_forward(self.h, batch.desc, *_rows(q), *_rows(out), lse, ws, n, stream)

    def status(self, stream=None) -> int:
        return moe_attn_status(self.h, stream)
