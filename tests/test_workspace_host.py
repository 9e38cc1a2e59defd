"""Workspace bookkeeping: which buffer a call gets and which buffers stay (no GPU)."""
import contextlib
import weakref

import pytest


@pytest.fixture()
def W(monkeypatch):
    """The module on CPU memory: `capturing` holds the streams that are being captured,
    `used` the streams that memory was asked for on."""
    from mxfp4_routed_expert_03_gb300 import workspace as w
    w.capturing, w.used = set(), []
    monkeypatch.setattr(w, "_capturing", lambda key: key in w.capturing)

    def on(key, device):
        w.used.append(key)
        return contextlib.nullcontext()
    monkeypatch.setattr(w, "_on", on)
    return w


def test_buffers_grow_and_are_reused(W):
    ws = W.Workspace("cpu")
    a = ws.get(0)
    assert a.numel() == 256 and ws.get(256) is a
    b = ws.get(1000)
    assert b.numel() == 1000 and ws.get(10) is b and ws.get(1000) is b


def test_streams_share_no_buffer_and_own_their_memory(W):
    class Stream:
        cuda_stream = 77
    ws = W.Workspace("cpu")
    a, b, c = ws.get(10), ws.get(10, 5), ws.get(10, Stream())
    assert len({t.data_ptr() for t in (a, b, c)}) == 3
    assert ws.get(10, 5) is b and ws.get(10, 77) is c and ws.get(10, None) is a and ws.get(10, 0) is a
    ws.get(5000, 5)
    assert W.used == [0, 5, 77, 5]


def test_a_captured_buffer_outlives_larger_calls(W):
    ws = W.Workspace("cpu")
    plain = weakref.ref(ws.get(10, 5))
    ws.get(1000, 5)
    assert plain() is None              # nothing holds a replaced buffer
    W.capturing.add(5)
    held = weakref.ref(ws.get(1000, 5))
    W.capturing.clear()
    assert ws.get(500, 5) is held()
    grown = ws.get(2000, 5)
    assert held() is not None and grown is not held()
    again = weakref.ref(grown)
    del grown
    ws.get(3000, 5)                     # a buffer that no capture saw goes
    assert again() is None and held() is not None
    W.capturing.add(5)
    inside = weakref.ref(ws.get(4000, 5))  # grown inside the capture
    W.capturing.clear()
    ws.get(5000, 5)
    assert inside() is not None
    del ws
    assert held() is None and inside() is None


@pytest.mark.parametrize("T", [1, 70])
def test_layer_and_attention_ask_for_the_calls_stream(W, monkeypatch, T):
    from mxfp4_routed_expert_03_gb300 import attention, layer
    asked = []

    class Space:
        def get(self, n, stream=None):
            asked.append((n, stream))
            import torch
            return torch.empty(max(n, 1), dtype=torch.uint8)
    monkeypatch.setattr(layer, "moe_workspace_bytes", lambda h, T, op: 10 * T + op)
    for n in ("moe_plan", "moe_plan_scored", "moe_decode", "moe_forward"):
        monkeypatch.setattr(layer, n, lambda *a: 0)
    L = layer.Layer.__new__(layer.Layer)
    L.h, L.router_mode, L.atoms, L._space = None, 0, object(), Space()

    L.E = 8

    class P:
        buf = None
    P.T = T
    L.plan(T, None, None, P, 3)
    L.plan_scored(T, None, None, P, None, None, 4)
    L.decode(T, None, P, None, 5)
    L.forward(T, None, P, None, 6)
    assert [s for _, s in asked] == [3, 4, 5, 6]
    asked.clear()
    monkeypatch.setattr(attention, "moe_attn_workspace_bytes", lambda h, *key: sum(key))
    given = []

    class Lib:
        def moe_attn_forward(self, *a):
            given.append(a[-3:])
            return 0
    monkeypatch.setattr(attention, "lib", Lib)
    A = attention.Attention.__new__(attention.Attention)
    A.h, A._need, A._space = None, (None, 0), Space()
    A.n_heads, A.q_width = 1, 64
    A.desc = attention.moe_attn_desc(1, 1, 64, 16, 1)
    b = attention.Batch(1, T, 1, 9, None, None, None, 1.0)
    A.forward(b, None, None, None, 8)
    assert asked == [(T + 11, 8)]
    own = W.empty_on(500, None, "cpu")
    A.forward(b, None, None, None, 8, own)
    assert len(asked) == 1 and given[-1][0] == own.data_ptr() and given[-1][1:] == (500, 8)
