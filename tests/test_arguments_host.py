"""What the Python classes refuse before a pointer leaves them, and what they pass on (no GPU:
the C entry points are replaced by ones that record their arguments)."""
import pytest
import torch

H, KV, D, PAGE, PAGES = 4, 2, 64, 16, 3
bf16, i32 = torch.bfloat16, torch.int32


@pytest.fixture()
def A(monkeypatch):
    from mxfp4_routed_expert_03_gb300 import attention as m
    calls = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: calls.append(a) or 0
    monkeypatch.setattr(m, "lib", Lib)
    monkeypatch.setattr(m, "moe_attn_create", lambda *a: 0)
    monkeypatch.setattr(m, "moe_attn_destroy", lambda *a: None)
    m.calls = calls
    m.cache = m.alloc_kv_cache(KV, D, PAGE, PAGES, device="cpu")
    m.make = lambda **k: m.Attention(H, KV, D, PAGE, PAGES, {**m.cache, **k})
    m.ws = torch.empty(256, dtype=torch.uint8)
    return m


def _refused(A, call, *bad):
    """`call` refuses each of `bad` with a ValueError and reaches no entry point."""
    for args in bad:
        del A.calls[:]
        with pytest.raises(ValueError):
            call(*args)
        assert not A.calls


def test_cache_arrays(A):
    A.make()
    A.make(k_q=torch.zeros(2 * A.cache["k_q"].numel(), dtype=torch.int8))
    for n, t in A.cache.items():
        for bad in (t[:2], t.repeat(1, 2, *[1] * (t.dim() - 2))[:, ::2]):
            with pytest.raises(ValueError):
                A.make(**{n: bad})
    with pytest.raises(KeyError):
        A.Attention(H, KV, D, PAGE, PAGES, {"k_q": A.cache["k_q"]})


def test_append_and_read(A):
    a = A.make()
    x, slots = torch.zeros(5, KV * D, dtype=bf16), torch.zeros(5, dtype=i32)
    wide = torch.zeros(5, 3 * KV * D, dtype=bf16)[:, KV * D:2 * KV * D]
    bad = ((5, x.float(), x, slots), (5, x, x[:4], slots), (5, x, x[:, :-8], slots), (5, x, x, slots[:4]),
           (5, x, x, slots.long()), (5, x, x, slots.float()), (5, x, x, torch.zeros(10, dtype=i32)[::2]),
           (5, x[0], x, slots), (6, x, x, slots))
    for call, order in ((a.append, lambda n, k, v, s: (n, k, v, s)), (a.read, lambda n, k, v, s: (n, s, k, v))):
        _refused(A, call, *[order(*b) for b in bad])
        for good in ((5, x, x, slots), (3, wide, x, slots), (5, x.view(torch.int16), wide, slots), (0, None, None, None),
                     (-1, x, x, slots), (5, x, x, slots.data_ptr()), (5, x, x, None)):
            assert call(*order(*good)) == 0
    assert a.read(5, slots, x, None) == 0 and A.calls[-1][5] is None


def test_norm_rope(A):
    a = A.make()
    q, k, pos = torch.zeros(5, H * D, dtype=bf16), torch.zeros(5, KV * D, dtype=bf16), torch.zeros(5, dtype=i32)
    table, w = torch.zeros(7, D), torch.zeros(D, dtype=bf16)
    rope = A.Rope(table, D, q_weight=w, k_weight=w)
    _refused(A, a.norm_rope, (5, q, k, pos.long(), rope, q, k), (5, q, k, pos[:3], rope, q, k),
             (5, q.float(), k, pos, rope, q, k), (5, q[:3], k, pos, rope, q, k), (5, q, k, pos, rope, q[:3], k),
             (5, q, q[:, :64], pos, rope, q, k), (5, q, k, pos, rope, q, k[:, :64]),
             (5, q, k, pos, A.Rope(table, D, q_weight=w[:32]), q, k))
    for bad in (dict(cos_sin=table.double(), rope_dim=D), dict(cos_sin=table, rope_dim=32),
                dict(cos_sin=torch.zeros(7, 2 * D)[:, ::2], rope_dim=D),
                dict(cos_sin=table, rope_dim=D, q_weight=w.float()),
                dict(cos_sin=table, rope_dim=D, k_weight=torch.zeros(2 * D, dtype=bf16)[::2])):
        with pytest.raises(ValueError):
            A.Rope(**bad)
    assert a.norm_rope(5, q, k, pos, rope, q, k) == 0 and a.norm_rope(3, q, None, pos, rope, q, None) == 0
    assert a.norm_rope(5, q, k, None, A.Rope(None, 0), q, k) == 0
    A.Rope(table, 72), A.Rope(table, 24), A.Rope(None, 64)  # (the call refuses these)


def test_batch_and_forward(A):
    a = A.make()
    cu, kv, pages = torch.zeros(4, dtype=i32), torch.zeros(3, dtype=i32), torch.zeros(3, 2, dtype=i32)
    good = dict(n_seqs=3, n_tokens=6, max_q=2, max_kv=30, cu_q=cu, kv_len=kv, page_table=pages, scale=1.0)
    for k, v in (("cu_q", cu[:3]), ("cu_q", cu.long()), ("kv_len", kv[:2]), ("kv_len", kv.float()),
                 ("page_table", pages[:2]), ("page_table", pages.long()), ("page_table", pages[:, 0]),
                 ("page_table", torch.zeros(3, 4, dtype=i32)[:, ::2]), ("cu_q", torch.zeros(8, dtype=i32)[::2])):
        with pytest.raises(ValueError):
            A.Batch(**{**good, k: v})
    q, lse = torch.zeros(6, H * D, dtype=bf16), torch.zeros(6, H)
    b = A.Batch(**good)
    run = lambda *x: a.forward(*x, None, A.ws)  # noqa: E731
    _refused(A, run, (b, q[:5], q, None), (b, q, q[:5], None), (b, q.float(), q, None), (b, q, q[:, :-8], None),
             (b, q, q, lse[:5]), (b, q, q, lse.double()), (b, q, q, torch.zeros(6, 2 * H)[:, ::2]))
    assert run(b, q, q, lse) == 0 and run(b, torch.zeros(9, 2 * H * D, dtype=bf16)[:, H * D:], q, None) == 0
    # rows of a wider table: the entries between them are another's
    sliced = A.Batch(**{**good, "page_table": torch.zeros(3, 9, dtype=i32)[:, :2]})
    assert run(sliced, q, q, None) == 0
    short = A.Batch(**{**good, "max_kv": 33, "page_table": torch.zeros(3, 9, dtype=i32)[:, :2]})
    _refused(A, run, (short, q, q, None))
    for k in ("cu_q", "kv_len", "page_table"):  # (the call refuses these)
        assert run(A.Batch(**{**good, k: None}), q, q, None) == 0


def test_plan_scored(monkeypatch):
    from mxfp4_routed_expert_03_gb300 import MOE_ROUTER_XWR, layer as m
    calls = []
    monkeypatch.setattr(m, "moe_plan_scored", lambda *a: calls.append(a) or 0)
    L = m.Layer.__new__(m.Layer)
    L.h, L.D, L.E, L.k, L.router_mode, L.atoms = None, 256, 32, 4, 0, object()
    monkeypatch.setattr(m.Layer, "workspace", lambda self, T, op, stream=None: (torch.empty(1), 1))
    plan, lg, bias = m.Plan(5, 32, 4, device="cpu"), torch.zeros(5, 32), torch.zeros(32)
    x = torch.zeros(5, 256, dtype=bf16)
    for bad in ((5, lg.double(), None, plan, None, bias), (5, lg[:4], None, plan, None, bias),
                (5, lg, None, plan, None, bias[:31]), (5, lg, None, plan, None, bias.half()),
                (5, torch.zeros(5, 64)[:, ::2], None, plan, None, None), (6, torch.zeros(6, 32), None, plan, None, None)):
        with pytest.raises(ValueError):
            L.plan_scored(*bad)
    assert not calls
    assert L.plan_scored(5, lg, None, plan, None, bias) == 0 and L.plan_scored(3, lg, None, plan, None) == 0
    L.router_mode = MOE_ROUTER_XWR
    for bad in (x[:4], x.float(), torch.zeros(5, 512, dtype=bf16)[:, ::2]):
        with pytest.raises(ValueError):
            L.plan_scored(5, None, bad, plan, None)
    assert L.plan_scored(5, None, x, plan, None, bias) == 0 and L.plan_scored(5, None, None, plan, None) == 0
