"""Attention where rows, tiles or pages hold nothing, and where a NaN must or must not
reach a row. References and tolerances are test_gpu_attention's unless a test says
otherwise."""
import math

import pytest
import torch

from oracle.act_study import round_to_format
from test_gpu_attention import DEV, Setup, _randn
from test_gpu_attention_sizes import _refill

pytestmark = pytest.mark.gpu


def _evict():
    """The L2 cache holds none of the inputs afterwards."""
    torch.empty(1 << 28, dtype=torch.uint8, device=DEV).fill_(1)


@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_without_keys_are_zero_whatever_the_timing(d):
    """Column tiles of which no row sees a key: their queries come from HBM, each warp's at
    its own time, while other warps already write the rows' zeros."""
    from mxfp4_routed_expert_03_gb300 import check
    nq = [64] * 120 + [300] * 20
    kv = [0 if b % 3 else 5 for b in range(140)]
    s = Setup(8, 2, d, 16, nq, kv, seed=70)
    dead = torch.zeros(s.T, dtype=torch.bool, device=DEV)
    for b, (n, m) in enumerate(zip(nq, kv)):
        dead[s.cu[b]:s.cu[b + 1] - min(m, n)] = True
    for _ in range(20):
        s.out.fill_(7.0)
        s.lse.fill_(7.0)
        _evict()
        check(s.attn.forward(s.batch, s.q, s.out, s.lse), "forward")
        assert bool((s.out[dead] == 0).all()) and bool((s.lse[dead] == -math.inf).all())
        assert bool((s.lse[~dead] > -math.inf).all())
    assert s.attn.status() == 0


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("H,KV,nq,kv", [(4, 2, [6, 1], [2, 3]), (8, 2, [90, 40], [50, 0]), (8, 1, [200], [10]),
                                        (8, 2, [1200], [1100])])
def test_non_finite_query_that_sees_no_key_gives_zero(H, KV, nq, kv, bad):
    """Few rows, many rows, and many rows with the keys split over CTAs. Rows that see a key
    become NaN, all others stay within twice test_gpu_attention's bound of a run without."""
    s = Setup(H, KV, 64, 16, nq, kv, seed=71)
    clean, clean_lse = (t.double().clone() for t in s.run())
    hit = torch.zeros(s.T, H, dtype=torch.bool, device=DEV)
    empty = torch.zeros(s.T, H, dtype=torch.bool, device=DEV)
    for b, (n, m) in enumerate(zip(nq, kv)):
        first = s.cu[b] + max(n - m, 0)  # row that sees the first key
        empty[s.cu[b]:first] = True
        for r in {s.cu[b], max(first - 1, s.cu[b]), min(first, s.cu[b + 1] - 1), s.cu[b + 1] - 1}:
            s.q[r, 64 * (r % H) + 7] = bad
            hit[r, r % H] = True
    out, lse = s.run()
    assert s.attn.status() == 0
    out = out.double().view(s.T, H, 64)
    assert bool((out[empty] == 0).all()) and bool((lse[empty] == -math.inf).all())
    assert bool(torch.isnan(out[hit & ~empty]).all()) and bool(torch.isnan(lse[hit & ~empty]).all())
    rest = ~hit & ~empty
    top = max([float(v.abs().max()) for v in s.v if v.numel()])
    assert bool(((out - clean.view(s.T, H, 64))[rest].abs() <= 2 * top * (2.0 ** -8 + 2.0 ** -9)).all())
    assert bool(((lse - clean_lse)[rest].abs() <= 2.0 ** -10).all())


@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("H,KV,nq", [(4, 2, 1), (8, 1, 3), (8, 1, 40)])
def test_pages_before_the_window_are_not_looked_up(H, KV, nq, page):
    """A cache manager may have given the pages back that lie wholly before the window."""
    kv = [100 + i for i in range(0, 70, 3)]
    s = Setup(H, KV, 64, page, [nq] * len(kv), kv, seed=72, window=20)
    for b, n in enumerate(kv):
        s.table[b, :(n - nq + 1 - 20) // page] = -1
    s.check()


@pytest.mark.parametrize("nq", [1, 40])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nan_at,top_at", [(37, 250), (250, 37), (36, 37), (37, 36), (200, 201)])
@pytest.mark.parametrize("window", [0, 150])
def test_nan_value_reaches_rows_that_hardly_weigh_it(window, nan_at, top_at, d, nq):
    """One key's logit far above the others' (whose weights are below 2^-40 of it), a NaN value
    at another: every row that sees that key has it, and no other."""
    from mxfp4_routed_expert_03_gb300 import check
    n = 300
    s = Setup(8, 1, d, 16, [nq], [n], seed=73, window=window)
    s.q.copy_((3.0 * torch.sign(s.q)).bfloat16())
    k = torch.zeros(n, d, dtype=torch.bfloat16, device=DEV)
    v = _randn(n, d, seed=74)
    v[nan_at, d - 7] = math.nan
    j = torch.arange(n, device=DEV)
    slots = (s.table[0, j // 16] * 16 + j % 16).int()
    # head r % 8 of every row has the key of its own signs: 9 d scale
    for head in (0, 5):
        k[top_at] = s.q[nq - 1, head * d:(head + 1) * d]
        check(s.attn.append(n, k, v, slots), "append")
        out, lse = s.run()
        assert s.attn.status() == 0
        pos = n - nq + torch.arange(nq, device=DEV)
        sees = (pos >= nan_at) & ((pos - window < nan_at) | (window == 0))
        hit = torch.zeros(nq, 8, d, dtype=torch.bool, device=DEV)
        hit[sees, :, d - 32:] = True
        out = out.view(nq, 8, d)
        assert bool(torch.isnan(out[hit]).all()) and bool(torch.isfinite(out[~hit]).all())
        assert bool(torch.isfinite(lse).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("nq,seqs", [(64, 80), (1, 912)])
def test_small_weights_of_a_long_context_add_up(nq, seqs, d):
    """One key far above 2^20 others, whose weights are 2^-25.5 of its own and 2^-5.5 in all.
    Keys of 0 and 1, values of 0 (the one) and 1 (the others): out = W / (1 + W), with W the sum
    of the others' weights. Weights are rounded to fp16 after a factor of 2^5 at least, so they
    lose 2^-30 each; the bounds are otherwise test_gpu_attention's. Enough column tiles that the
    keys of one are not split (many rows), or CTAs that take whole sequences (one row); all
    sequences share the pages."""
    from mxfp4_routed_expert_03_gb300 import check
    from mxfp4_routed_expert_03_gb300.attention import Attention, Batch, alloc_kv_cache
    n, page, H = 1 << 20, 256, 8 if nq > 1 else 1
    a = Attention(H, 1, d, page, n // page, alloc_kv_cache(1, d, page, n // page))
    k, v = torch.zeros(n, d, device=DEV).bfloat16(), torch.ones(n, d, device=DEV).bfloat16()
    k[5], v[5] = 1.0, 0.0
    slots = torch.randperm(n // page, device=DEV)[:, None] * page + torch.arange(page, device=DEV)
    table = (slots[:, 0] // page).int().expand(seqs, -1).contiguous()
    check(a.append(n, k, v, slots.flatten().int()), "append")
    low = 25.5
    q = torch.ones(seqs * nq, H * d, device=DEV).bfloat16()
    cu = torch.arange(0, seqs * nq + 1, nq, device=DEV, dtype=torch.int32)
    kv = torch.full((seqs,), n, dtype=torch.int32, device=DEV)
    batch = Batch(seqs, seqs * nq, nq, n, cu, kv, table, low * math.log(2.0) / d)
    out, lse = torch.empty_like(q), torch.empty(seqs * nq, H, device=DEV)
    check(a.forward(batch, q, out, lse), "forward")
    assert a.status() == 0
    seen = (n - nq + 1 + torch.arange(nq, device=DEV, dtype=torch.float64)).repeat(seqs)
    W = ((seen - 1) * 2.0 ** -low)[:, None]
    want = W / (1 + W)
    bound = 2.0 ** -8 * want + 2.0 ** -9 * want + n * 2.0 ** -30 / (1 + W)
    assert bool(((out.double() - want).abs() <= bound).all())
    assert bool(((lse.double() - (low * math.log(2.0) + torch.log1p(W))).abs() <= 2.0 ** -17 * (1 + low)).all())


@pytest.mark.parametrize("nq", [1, 2, 40])
@pytest.mark.parametrize("d", [64, 128])
def test_keys_of_the_smallest_scale(d, nq):
    """All keys have scale byte 0 (2^-127), and queries are so large that the logits are of
    ordinary size: no key lies below another by enough to count as zero."""
    s = Setup(8, 1, d, 32, [nq], [200], seed=75, q_scale=1e37, scale=1.0)
    k = _randn(200, d, seed=76, scale=1e-38)
    _refill(s, 0, k)
    # (the reference's own quantisation has no smallest scale)
    s.k[0] = torch.from_numpy(round_to_format(k.double().cpu().numpy() * 2.0 ** 127, "e2m1") * 2.0 ** -127).to(DEV)
    s.k[0] = s.k[0].view(200, 1, d)
    assert bool((s.attn.cache["k_s"].view(-1, 32, d // 32)[s.table[0, 0].long()] == 0).all())
    assert float((s.q.double().view(-1, 8, d) @ s.k[0][:, 0].T).std()) > 0.3
    s.check()
