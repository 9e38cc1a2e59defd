"""Buffer bookkeeping around the attention half of the C ABI.

Holds torch-owned device buffers (the MXFP4 key/value cache, workspace) and
calls the C entry points; it computes nothing itself. Tensors of token rows
may be slices of wider ones (their row stride is passed on). What the C side
cannot see of a tensor (its type, its length) is checked here and refused with
a ValueError; everything else is left to the C side and its codes.
"""
from __future__ import annotations

import ctypes

import torch

from . import (_stream, lib, moe_attn_batch, moe_attn_create, moe_attn_desc, moe_attn_destroy,
               moe_attn_status, moe_attn_workspace_bytes, moe_kv_cache, moe_kv_code_bytes,
               moe_kv_scale_bytes, moe_rope_desc)
from .checks import BITS16, bf16_rows, flat, on_device, rows
from .workspace import Workspace

_i32, _f32 = torch.int32, torch.float32

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


class Rope:
    """Norm and rotation parameters; keeps the tensors they point at. cos_sin:
    fp32 [n_pos][rope_dim] (cosines, then sines), or None for no rotation;
    q_weight / k_weight: bf16 [head_dim], or None for no norm."""

    def __init__(self, cos_sin, rope_dim: int, interleaved: bool = False, eps: float = 1e-6,
                 q_weight=None, k_weight=None):
        self.tensors = (cos_sin, q_weight, k_weight)
        n_pos = 0 if cos_sin is None else cos_sin.shape[0]
        if rope_dim > 0 and rope_dim % 16 == 0:  # (others are refused by the call)
            flat(cos_sin, n_pos * rope_dim, _f32, "cos_sin")
            if cos_sin is not None and cos_sin.numel() != n_pos * rope_dim:
                raise ValueError("cos_sin: rows of rope_dim elements")
        weights = [w for w in (q_weight, k_weight) if w is not None]
        if any(w.element_size() != 2 or not w.is_contiguous() for w in weights):
            raise ValueError("norm weights: contiguous bf16 elements")
        self.width = min([w.numel() for w in weights], default=1 << 30)  # that the weights have
        self.bf16 = all(w.dtype in BITS16 for w in weights)
        self.desc = moe_rope_desc(rope_dim, int(interleaved), n_pos, eps, _ptr(cos_sin),
                                  _ptr(q_weight), _ptr(k_weight))
        self.ref = ctypes.byref(self.desc)


class Batch:
    """A batch of sequences for Attention.forward; keeps the tensors it points
    at. cu_q: int32 [n_seqs + 1] or None (one query row per sequence); kv_len:
    int32 [n_seqs]; page_table: int32 [n_seqs][pages]; max_q / max_kv bound a
    sequence's query rows and cached tokens."""

    def __init__(self, n_seqs: int, n_tokens: int, max_q: int, max_kv: int, cu_q, kv_len,
                 page_table, scale: float, window: int = 0):
        if page_table is not None and (page_table.dim() != 2 or page_table.stride(1) != 1):
            raise ValueError("page_table: a 2D tensor with contiguous rows")
        flat(cu_q, n_seqs + 1, _i32, "cu_q")
        flat(kv_len, n_seqs, _i32, "kv_len")
        stride, self.cols = 0, None  # cols: entries of a row, where rows have gaps between them
        if page_table is not None:
            if page_table.dtype != torch.int32 or page_table.shape[0] < n_seqs:
                raise ValueError("page_table: int32, a row per sequence")
            stride = page_table.stride(0)
            if stride > page_table.shape[1]:
                self.cols = page_table.shape[1]
        self.tensors = (cu_q, kv_len, page_table)
        self.n_tokens, self.key = n_tokens, (n_seqs, n_tokens, max_q, max_kv)
        self.desc = moe_attn_batch(n_seqs, n_tokens, max_q, max_kv, stride, window, scale,
                                   _ptr(cu_q), _ptr(kv_len), _ptr(page_table))
        self.ref = ctypes.byref(self.desc)


class Attention:
    """One layer's attention: head shape, the paged MXFP4 cache and the library handle."""

    def __init__(self, n_heads: int, n_kv_heads: int, head_dim: int, page_size: int, n_pages: int,
                 cache: dict):
        self.cache = cache
        self.h = None
        self.desc = moe_attn_desc(n_heads, n_kv_heads, head_dim, page_size, n_pages)
        self.head_dim, self.n_heads, self.q_width, self.kv_width = head_dim, n_heads, n_heads * head_dim, n_kv_heads * head_dim
        for name in CACHE_NAMES:
            need = (moe_kv_code_bytes if name.endswith("_q") else moe_kv_scale_bytes)(self.desc)
            if need >= 0 and (cache[name].nbytes < need or not cache[name].is_contiguous()):
                raise ValueError(f"cache {name}: {need} contiguous bytes")
        self.h = moe_attn_create(self.desc, moe_kv_cache(*[cache[n].data_ptr() for n in CACHE_NAMES]))
        self._space = Workspace(cache["k_q"].device)
        self.device = cache["k_q"].get_device()
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

    # (the calls go to the library without the package's wrappers: a step's host time counts)
    def norm_rope(self, T, q, k, positions, rope: Rope, q_out, k_out, stream=None) -> int:
        if rope.width < self.head_dim or not rope.bf16:
            raise ValueError("norm weights: head_dim bf16 elements")
        positions = flat(positions, T, _i32, "positions")
        q, qs = rows(q, T, self.q_width)
        k, ks = rows(k, T, self.kv_width)
        q_out, qos = rows(q_out, T, self.q_width)
        k_out, kos = rows(k_out, T, self.kv_width)
        return lib().moe_qk_norm_rope(self.h, T, rope.ref, positions, q, qs, k, ks, q_out, qos, k_out, kos,
                                      _stream(stream))

    def append(self, T, k, v, slots, stream=None) -> int:
        slots = flat(slots, T, _i32, "slots")
        k, ks = rows(k, T, self.kv_width)
        v, vs = rows(v, T, self.kv_width)
        return lib().moe_kv_append(self.h, T, k, ks, v, vs, slots, _stream(stream))

    def rope_append(self, T, q, k, v, positions, rope: Rope, q_out, slots, stream=None) -> int:
        """norm_rope of q into q_out and of k, which goes with v into the cache (q may be None with q_out)."""
        dev = self.device
        if rope.width < self.head_dim or not rope.bf16:
            raise ValueError("norm weights: head_dim bf16 elements")
        on_device(dev, positions, slots, *rope.tensors)
        positions = flat(positions, T, _i32, "positions")
        slots = flat(slots, T, _i32, "slots")
        q, qs = bf16_rows(q, T, self.q_width, dev)
        k, ks = bf16_rows(k, T, self.kv_width, dev)
        v, vs = bf16_rows(v, T, self.kv_width, dev)
        q_out, qos = bf16_rows(q_out, T, self.q_width, dev)
        return lib().moe_rope_append(self.h, T, rope.ref, positions, q, qs, k, ks, v, vs, slots, q_out, qos,
                                     _stream(stream))

    def read(self, n, slots, k, v, stream=None) -> int:
        slots = flat(slots, n, _i32, "slots")
        k, ks = rows(k, n, self.kv_width)
        v, vs = rows(v, n, self.kv_width)
        return lib().moe_kv_read(self.h, n, slots, k, ks, v, vs, _stream(stream))

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
        T = batch.n_tokens
        if batch.cols is not None and batch.cols * self.desc.page_size < batch.key[3]:
            raise ValueError("page_table: entries for max_kv tokens in a row")
        lse = flat(lse, T * self.n_heads, _f32, "lse")
        q, qs = rows(q, T, self.q_width)
        out, os = rows(out, T, self.q_width)
        if ws is None:
            ws, n = self.workspace(batch, stream)
        else:
            n = ws.numel() * ws.element_size()
        return lib().moe_attn_forward(self.h, batch.ref, q, qs, out, os, lse, ws.data_ptr(), n, _stream(stream))

    def status(self, stream=None) -> int:
        return moe_attn_status(self.h, stream)
