"""The attention operators against plain 64-bit references.

Tolerances. Outputs are rounded once to bf16 (2^-9 relative). norm_rope: fp32
arithmetic in between (a few 2^-24), so 2^-8 |y| bounds an element, plus the
cancellation of a rotation, 2^-20 of its pair. Attention: the weights p are
rounded to fp16 (2^-12 relative) and everything else is fp32, so an element
is within 2^-8 |out| + 2^-9 sum p |v|; weights below fp16's normal range are
off by 2^-25 of the largest, 4096 of them 2^-13. lse: 128-term fp32 sums,
2^-17 of the largest sum |q k|. The cache is exact."""
import math

import numpy as np
import pytest
import torch

import attn_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16_EPS = 2.0 ** -8


def _attn(H, KV, d, page, pages, zero=True):
    from mxfp4_routed_expert_03_gb300.attention import Attention, alloc_kv_cache
    cache = alloc_kv_cache(KV, d, page, pages)
    if not zero:  # what an unwritten cache may hold
        g = torch.Generator(device=DEV).manual_seed(9)
        for t in cache.values():
            t.copy_(torch.randint(256, t.shape, device=DEV, generator=g, dtype=torch.uint8))
    return Attention(H, KV, d, page, pages, cache)


def _randn(*shape, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (scale * torch.randn(*shape, device=DEV, generator=g)).bfloat16()


class Setup:
    """A filled paged cache, its fp64 contents and a batch over it."""

    def __init__(self, H, KV, d, page, nq, kv, seed=0, window=0, scale=None, q_scale=1.0,
                 v_scale=1.0, single=False, v_exp=0):
        from mxfp4_routed_expert_03_gb300 import check
        from mxfp4_routed_expert_03_gb300.attention import Batch
        self.H, self.KV, self.d, self.page, self.kv = H, KV, d, page, kv
        need = [-(-n // page) for n in kv]
        pages = sum(need) + 2
        self.attn = _attn(H, KV, d, page, pages, zero=False)
        g = torch.Generator(device="cpu").manual_seed(seed)
        order = torch.randperm(pages, generator=g).tolist()
        table = torch.full((len(kv), max(max(need), 1) + 1), -7, dtype=torch.int32)
        self.k, self.v = [], []
        for b, n in enumerate(kv):
            mine = [order.pop() for _ in range(need[b])]
            table[b, :len(mine)] = torch.tensor(mine, dtype=torch.int32)
            k = _randn(n, KV * d, seed=seed + 10 * b + 1)
            v = _randn(n, KV * d, seed=seed + 10 * b + 2, scale=v_scale)
            if v_exp and n:  # very different magnitudes from token to token
                v = (v.float() * torch.exp2(torch.arange(n, device=DEV) % (2 * v_exp) - v_exp)[:, None].float()).bfloat16()
            if n:
                j = torch.arange(n)
                slots = (table[b][j // page] * page + j % page).int().to(DEV)
                check(self.attn.append(n, k, v, slots), "append")
            self.k.append(ref.mxfp4(k).view(n, KV, d))
            self.v.append(ref.mxfp4(v).view(n, KV, d))
        self.table = table.to(DEV)
        self.cu = [0]
        for n in nq:
            self.cu.append(self.cu[-1] + n)
        self.T = self.cu[-1]
        self.q = _randn(self.T, H * d, seed=seed + 5, scale=q_scale)
        self.scale = d ** -0.5 if scale is None else scale
        self.window = window
        self.kv_t = torch.tensor(kv, dtype=torch.int32, device=DEV)
        self.cu_t = None if single else torch.tensor(self.cu, dtype=torch.int32, device=DEV)
        self.batch = Batch(len(kv), self.T, max(nq), max(max(kv), 1), self.cu_t, self.kv_t,
                           self.table, self.scale, window)
        self.out = torch.full((self.T, H * d), 7.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((self.T, H), 7.0, device=DEV)

    def run(self):
        from mxfp4_routed_expert_03_gb300 import check
        check(self.attn.forward(self.batch, self.q, self.out, self.lse), "forward")
        return self.out, self.lse

    def want(self, q=None):
        q = self.q if q is None else q
        return ref.attention(q.double().view(self.T, self.H, self.d), self.k, self.v, self.cu,
                             self.kv, self.scale, self.window)

    def check(self):
        out, lse = self.run()
        assert self.attn.status() == 0
        o, l_, mag, big = self.want()
        _close(out, lse, o.view(self.T, -1), l_, mag.view(self.T, -1), big)
        return out, lse


def _close(out, lse, o, l_, mag, big):
    err = (out.double() - o).abs()
    assert bool((err <= BF16_EPS * o.abs() + 2.0 ** -9 * mag + 1e-30).all()), float((err / (mag + 1e-30)).max())
    dead = torch.isinf(l_)
    assert bool((lse.double()[dead] == -math.inf).all())
    assert bool(((lse.double() - l_).abs()[~dead] <= 2.0 ** -17 * (1 + big)).all())


@pytest.mark.parametrize("H,KV,d,page", [(8, 1, 128, 16), (56, 8, 128, 64), (4, 4, 64, 32),
                                         (24, 2, 64, 16), (40, 8, 128, 128), (17, 1, 128, 256)])
def test_one_token_over_lengths_around_tiles_and_pages(H, KV, d, page):
    kv = [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 257, 300]
    Setup(H, KV, d, page, [1] * len(kv), kv, seed=H, single=True).check()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kv", [1, 40, 128])
def test_short_sequences_take_whole_items(d, kv):
    Setup(16, 2, d, 32, [1] * 5, [kv, 0, kv, 1, kv], seed=kv).check()


@pytest.mark.parametrize("window", [0, 1, 7, 32, 100])
@pytest.mark.parametrize("H,KV,d", [(8, 2, 64), (12, 1, 128)])
def test_several_queries_causal_and_window(H, KV, d, window):
    Setup(H, KV, d, 16, [3, 1, 9, 20, 5, 2], [3, 70, 9, 200, 0, 1], seed=window, window=window).check()


def test_rows_that_see_nothing():
    s = Setup(4, 2, 64, 16, [6, 4, 1], [2, 0, 0], seed=1)
    out, lse = s.check()  # the first 4 rows of sequence 0 lie before its first token
    for r in (0, 1, 2, 3, 6, 7, 8, 9, 10):
        assert bool((out[r] == 0).all()) and bool((lse[r] == -math.inf).all())
    assert bool((lse[4:6] > -math.inf).all())


def test_prefill_rows():
    Setup(8, 2, 128, 64, [70, 33], [150, 33], seed=3).check()


def test_long_sequence_split_over_the_gpu():
    s = Setup(8, 1, 128, 64, [1], [20000], seed=4)
    s.check()
    again = [s.run()[0].clone() for _ in range(3)]
    assert all(torch.equal(x, again[0]) for x in again)  # joined in a fixed order


def test_large_logits_and_value_magnitudes():
    Setup(8, 2, 128, 32, [1, 2], [500, 333], seed=5, q_scale=30.0).check()   # one key takes all
    Setup(8, 2, 64, 32, [1, 2], [300, 90], seed=6, v_scale=1e30).check()
    Setup(8, 2, 128, 32, [1, 2], [300, 90], seed=7, v_scale=1e-30).check()
    Setup(8, 2, 128, 32, [1, 2], [300, 90], seed=8, v_exp=5).check()         # 2^-5 .. 2^4 by token
    Setup(8, 2, 64, 32, [2], [100], seed=9, q_scale=1e-30).check()           # uniform weights
    Setup(8, 2, 64, 32, [2], [100], seed=10, scale=0.0).check()
    Setup(8, 2, 64, 32, [2], [100], seed=11, scale=-0.3).check()


def test_strided_queries_and_outputs_and_no_lse():
    from mxfp4_routed_expert_03_gb300 import check
    s = Setup(8, 2, 64, 32, [3, 1], [50, 90], seed=12)
    s.check()
    fused = torch.full((4, 8 * 64 + 264), 3.0, dtype=torch.bfloat16, device=DEV)
    fused[:, 8:8 + 512] = s.q
    wide = torch.full((4, 8 * 64 + 40), 5.0, dtype=torch.bfloat16, device=DEV)
    check(s.attn.forward(s.batch, fused[:, 8:8 + 512], wide[:, 16:16 + 512], None), "forward")
    assert torch.equal(wide[:, 16:528], s.out)
    assert bool((wide[:, :16] == 5.0).all()) and bool((wide[:, 528:] == 5.0).all())


def test_another_stream():
    s = Setup(8, 2, 128, 32, [1, 1], [700, 90], seed=13)
    from mxfp4_routed_expert_03_gb300 import check
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    check(s.attn.forward(s.batch, s.q, s.out, s.lse, st), "forward")
    assert s.attn.status(st) == 0
    o, l_, mag, big = s.want()
    _close(s.out, s.lse, o.view(s.T, -1), l_, mag.view(s.T, -1), big)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_non_finite_keys_and_values_reach_only_the_rows_that_see_them(bad):
    from mxfp4_routed_expert_03_gb300 import check
    s = Setup(4, 2, 64, 16, [10], [60], seed=14)
    o, l_, mag, big = s.want()
    page = s.table[0, 54 // 16] * 16 + 54 % 16
    k = _randn(1, 2 * 64, seed=99)
    v = _randn(1, 2 * 64, seed=98)
    s.k[0][54], s.v[0][54] = ref.mxfp4(k).view(2, 64), ref.mxfp4(v).view(2, 64)
    o, l_, mag, big = s.want()
    v[0, 64 + 40] = bad       # token 54, head 1, second block: rows 4.. see it
    check(s.attn.append(1, k, v, page.view(1).int()), "append")
    out, lse = s.run()
    hit = torch.zeros(10, 4, 64, dtype=torch.bool, device=DEV)
    hit[4:, 2:, 32:] = True
    hit = hit.view(10, -1)
    assert bool(torch.isnan(out[hit]).all())
    err = (out.double() - o.view(10, -1)).abs()
    ok = err <= BF16_EPS * o.view(10, -1).abs() + 2.0 ** -9 * mag.view(10, -1)
    assert bool(ok[~hit].all())
    k[0, 3] = bad             # head 0, first block of the key
    check(s.attn.append(1, k, v, page.view(1).int()), "append")
    out, lse = s.run()
    hit = hit.view(10, 4, 64)
    hit[4:, :2] = True
    hit = hit.view(10, -1)
    assert bool(torch.isnan(out[hit]).all()) and bool(torch.isnan(lse[4:, :2]).all())
    err = (out.double() - o.view(10, -1)).abs()
    ok = err <= BF16_EPS * o.view(10, -1).abs() + 2.0 ** -9 * mag.view(10, -1)
    assert bool(ok[~hit].all())
    assert s.attn.status() == 0


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_non_finite_query_stays_in_its_row(bad):
    s = Setup(4, 2, 64, 16, [3], [60], seed=15)
    o, l_, mag, big = s.want()
    s.q[1, 64 + 5] = bad
    out, lse = s.run()
    hit = torch.zeros(3, 4, 64, dtype=torch.bool, device=DEV)
    hit[1, 1] = True
    assert bool(torch.isnan(out.view(3, 4, 64)[hit]).all()) and bool(torch.isnan(lse[1, 1]))
    err = (out.double().view(3, 4, 64) - o).abs()
    assert bool((err <= BF16_EPS * o.abs() + 2.0 ** -9 * mag)[~hit].all())


def test_bad_lengths_and_pages_are_reported_and_left_out():
    from mxfp4_routed_expert_03_gb300 import MOE_ERR_BAD_INDEX
    s = Setup(4, 2, 64, 16, [1, 1], [60, 70], seed=16)
    s.check()
    s.table[0, 1] = 100000          # tokens 16 .. 31 of sequence 0 have no page
    s.run()
    assert s.attn.status() == MOE_ERR_BAD_INDEX
    keep = [j for j in range(60) if not 16 <= j < 32]
    s.k[0], s.v[0] = s.k[0][keep], s.v[0][keep]
    s.kv = [44, 70]
    o, l_, mag, big = s.want()
    _close(s.out, s.lse, o.view(2, -1), l_, mag.view(2, -1), big)
    s = Setup(4, 2, 64, 16, [1, 1], [60, 70], seed=17)
    s.kv_t[0] = 1000                # above max_kv: clamped to 70, whose fifth page is -7
    s.run()
    assert s.attn.status() == MOE_ERR_BAD_INDEX
    s.kv_t[0] = -3
    out, lse = s.run()
    assert s.attn.status() == MOE_ERR_BAD_INDEX
    assert bool((out[0] == 0).all())
    s.kv_t[0] = 60
    s.cu_t[1] = 9                   # beyond n_tokens
    s.run()
    assert s.attn.status() == MOE_ERR_BAD_INDEX
    assert s.attn.status() == 0     # cleared after reading


# ------------------------------------------------------------------ the cache
def _bytes_of(attn, d, page, KV, slot, head, is_v):
    """Codes (one per element) and scale bytes of a slot, by the documented address."""
    q = attn.cache["v_q" if is_v else "k_q"].cpu().numpy().ravel()
    s = attn.cache["v_s" if is_v else "k_s"].cpu().numpy().ravel()
    p, o, nb = slot // page, slot % page, d // 32
    codes, scales = [], []
    for x in range(d):
        at = ((((p * KV + head) * (page // 8) + o // 8) * nb + x // 32) * 8 + o % 8) * 16 + x % 32 // 2
        codes.append((q[at] >> (4 * (x % 2))) & 15)
    for b in range(nb):
        if is_v:
            scales.append(s[(((p * KV + head) * (page // 2) + o // 2) * nb + b) * 2 + o % 2])
        else:
            scales.append(s[((p * KV + head) * page + o) * nb + b])
    return np.array(codes), np.array(scales)


@pytest.mark.parametrize("KV,d,page", [(1, 64, 16), (3, 128, 32), (8, 128, 256)])
@pytest.mark.parametrize("T", [1, 7, 8, 9, 50])
def test_append_and_read_back(KV, d, page, T):
    from mxfp4_routed_expert_03_gb300 import check
    pages = -(-T // page) + 3
    a = _attn(KV, KV, d, page, pages)
    before = {n: t.clone() for n, t in a.cache.items()}
    fused = _randn(T, 2 * KV * d + 8, seed=T, scale=3.0)
    k, v = fused[:, :KV * d], fused[:, KV * d:2 * KV * d]
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(pages * page, generator=g)[:T].int()
    if T > 7:
        slots[3] = -1
    check(a.append(T, k, v, slots.to(DEV)), "append")
    back = torch.full((T, 2 * KV * d + 16), 7.0, dtype=torch.bfloat16, device=DEV)
    check(a.read(T, slots.to(DEV), back[:, 8:8 + KV * d], back[:, 8 + KV * d:8 + 2 * KV * d]), "read")
    assert a.status() == 0
    keep = (slots >= 0).nonzero().flatten().to(DEV)
    for x, y in ((k, back[:, 8:8 + KV * d]), (v, back[:, 8 + KV * d:8 + 2 * KV * d])):
        assert torch.equal(y[keep].double(), ref.mxfp4(x[keep].contiguous()))
    if T > 7:
        assert bool((back[3] == 7.0).all())
    assert bool((back[:, :8] == 7.0).all()) and bool((back[:, -8:] == 7.0).all())
    levels = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    for i in (0, T - 1):
        for head in (0, KV - 1):
            for x, is_v in ((k, False), (v, True)):
                codes, scales = _bytes_of(a, d, page, KV, int(slots[i]), head, is_v)
                val = np.where(codes > 7, -1.0, 1.0) * levels[codes % 8] * np.repeat(2.0 ** (scales.astype(float) - 127), 32)
                want = ref.mxfp4(x[i:i + 1, head * d:(head + 1) * d].contiguous()).cpu().numpy()[0]
                np.testing.assert_array_equal(val, want)
    # nothing but those slots changed: write zeros to them and compare
    check(a.append(T, torch.zeros_like(fused)[:, :KV * d], torch.zeros_like(fused)[:, :KV * d], slots.to(DEV)), "append")
    for n, t in a.cache.items():
        assert torch.equal(t, before[n]), n


def test_append_edges_of_the_format():
    """Ties, saturation, the smallest and largest bf16 values, signed zeros."""
    from mxfp4_routed_expert_03_gb300 import check
    a = _attn(1, 1, 64, 16, 1)
    rows = torch.zeros(6, 64, dtype=torch.bfloat16, device=DEV)
    rows[0, :9] = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0])
    rows[1, :3] = torch.tensor([7.9, -7.9, 5.1])
    rows[2, 0] = 2.0 ** -133
    rows[2, 32] = -2.0 ** -126
    rows[3, :2] = torch.tensor([3.3e38, -1e38])
    rows[4, 0] = -0.0
    rows[5, :4] = torch.tensor([1e-38, 2e-39, 0.0, -1e-38])
    slots = torch.arange(6, dtype=torch.int32, device=DEV)
    check(a.append(6, rows, rows, slots), "append")
    back = torch.empty(6, 64, dtype=torch.bfloat16, device=DEV)
    for pair in ((back, None), (None, back)):
        check(a.read(6, slots, *pair), "read")
        assert a.status() == 0
        want = ref.mxfp4(rows[:2])
        assert torch.equal(back[:2].double(), want)
        assert back[1, 0] == 6.0 and back[1, 1] == -6.0
        # scale 2^-127: 2^-133 rounds to zero, 2^-126 = 2 x 2^-127 stays
        assert back[2, 0] == 0 and back[2, 32].double() == -2.0 ** -126
        assert torch.equal(back[3].double(), ref.mxfp4(rows[3:4])[0])
        assert bool((back[4] == 0).all())
    assert int(a.cache["k_s"].view(-1)[4 * 2]) == 0


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_append_non_finite_block_reads_as_nan(bad):
    from mxfp4_routed_expert_03_gb300 import check
    a = _attn(1, 1, 128, 16, 1)
    x = _randn(2, 128, seed=3)
    x[1, 70] = bad
    slots = torch.tensor([3, 4], dtype=torch.int32, device=DEV)
    check(a.append(2, x, x, slots), "append")
    k, v = torch.empty_like(x), torch.empty_like(x)
    check(a.read(2, slots, k, v), "read")
    for y in (k, v):
        assert bool(torch.isnan(y[1, 64:96]).all())
        y[1, 64:96] = 0
        z = x.clone()
        z[1, 64:96] = 0
        assert torch.equal(y.double(), ref.mxfp4(z))


def test_bad_slots_are_reported_and_skipped():
    from mxfp4_routed_expert_03_gb300 import MOE_ERR_BAD_INDEX, check
    a = _attn(2, 2, 64, 16, 2)
    x = _randn(3, 128, seed=4)
    slots = torch.tensor([32, -2, 5], dtype=torch.int32, device=DEV)
    check(a.append(3, x, x, slots), "append")
    assert a.status() == MOE_ERR_BAD_INDEX
    y = torch.full_like(x, 7.0)
    check(a.read(3, slots, y, None), "read")
    assert a.status() == MOE_ERR_BAD_INDEX
    assert bool((y[:2] == 7.0).all()) and torch.equal(y[2].double(), ref.mxfp4(x[2:])[0])


# ------------------------------------------------------------------ norm and rotation
def _table(n_pos, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(n_pos, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


@pytest.mark.parametrize("H,KV,d,rot,inter", [(56, 8, 128, 128, False), (5, 1, 128, 64, True),
                                              (4, 4, 64, 64, True), (6, 2, 64, 48, False),
                                              (3, 1, 128, 16, False), (8, 2, 64, 0, False)])
@pytest.mark.parametrize("T", [1, 5, 700])
def test_norm_rope(H, KV, d, rot, inter, T):
    from mxfp4_routed_expert_03_gb300 import check
    from mxfp4_routed_expert_03_gb300.attention import Rope
    a = _attn(H, KV, d, 16, 1)
    fused = _randn(T, (H + 2 * KV) * d, seed=T, scale=2.0)
    q, k = fused[:, :H * d], fused[:, H * d:(H + KV) * d]
    wq, wk = 1 + 0.3 * _randn(d, seed=1), 1 + 0.3 * _randn(d, seed=2)
    table = _table(4096, rot) if rot else None
    pos = torch.randint(4096, (T,), device=DEV, dtype=torch.int32) if rot else None
    rope = Rope(table, rot, interleaved=inter, eps=1e-5, q_weight=wq, k_weight=wk)
    qo, ko = (torch.empty(T, n * d, dtype=torch.bfloat16, device=DEV) for n in (H, KV))
    check(a.norm_rope(T, q, k, pos, rope, qo, ko), "norm_rope")
    assert a.status() == 0
    for x, w, y, n in ((q, wq, qo, H), (k, wk, ko, KV)):
        want = ref.norm_rope(x.double().reshape(T, n, d), w, 1e-5, table, pos, rot, inter)
        size = want.abs().amax(-1, keepdim=True)
        err = (y.double().view(T, n, d) - want).abs()
        assert bool((err <= BF16_EPS * want.abs() + 2.0 ** -20 * size).all())
    # in place, without the keys, without the norm
    q2 = q.clone()
    check(a.norm_rope(T, q2, None, pos, rope, q2, None), "norm_rope")
    assert torch.equal(q2, qo)
    plain = Rope(table, rot, interleaved=inter)
    check(a.norm_rope(T, None, k, pos, plain, None, ko), "norm_rope")
    want = ref.norm_rope(k.double().reshape(T, KV, d), None, 0, table, pos, rot, inter)
    err = (ko.double().view(T, KV, d) - want).abs()
    assert bool((err <= BF16_EPS * want.abs() + 2.0 ** -20 * want.abs().amax(-1, keepdim=True)).all())


def test_norm_rope_bad_position_and_zero_row():
    from mxfp4_routed_expert_03_gb300 import MOE_ERR_BAD_INDEX, check
    from mxfp4_routed_expert_03_gb300.attention import Rope
    a = _attn(2, 1, 64, 16, 1)
    q = _randn(3, 128, seed=1)
    q[2] = 0
    rope = Rope(_table(10, 64), 64, q_weight=torch.ones(64, dtype=torch.bfloat16, device=DEV))
    out = torch.full_like(q, 7.0)
    pos = torch.tensor([10, -1, 3], dtype=torch.int32, device=DEV)
    check(a.norm_rope(3, q, None, pos, rope, out, None), "norm_rope")
    assert a.status() == MOE_ERR_BAD_INDEX
    assert bool((out[:2] == 7.0).all()) and bool((out[2] == 0).all())


# ------------------------------------------------------------------ refusals
def test_refusals():
    from mxfp4_routed_expert_03_gb300 import (MOE_ERR_INVALID_ARG, MOE_ERR_WORKSPACE, moe_attn_forward)
    from mxfp4_routed_expert_03_gb300.attention import Batch, Rope
    s = Setup(4, 2, 64, 16, [2], [200], seed=20)
    a, bad = s.attn, MOE_ERR_INVALID_ARG
    fwd = lambda batch, q=s.q, out=s.out: a.forward(batch, q, out)  # noqa: E731
    B = lambda **k: Batch(*[k.get(n, v) for n, v in (  # noqa: E731
        ("n_seqs", 1), ("n_tokens", 2), ("max_q", 2), ("max_kv", 200), ("cu_q", s.cu_t), ("kv_len", s.kv_t),
        ("page_table", s.table), ("scale", 1.0), ("window", 0))])
    assert fwd(B()) == 0
    assert fwd(B(scale=math.nan)) == bad and fwd(B(scale=math.inf)) == bad
    assert fwd(B(window=-1)) == bad and fwd(B(max_kv=-1)) == bad and fwd(B(n_seqs=-1)) == bad
    assert fwd(B(max_kv=100000)) == bad                 # more pages than the table has
    assert fwd(B(kv_len=None)) == bad and fwd(B(page_table=None)) == bad and fwd(B(max_q=0)) == bad
    assert fwd(B(cu_q=None)) == bad                     # one row per sequence needs n_tokens == n_seqs
    assert fwd(B(n_seqs=0)) == 0 and fwd(B(n_tokens=0)) == 0
    assert moe_attn_forward(a.h, s.batch.desc, s.q, 256 - 8, s.out, 256, None, None, 0) == bad
    assert moe_attn_forward(a.h, s.batch.desc, s.q, 260, s.out, 256, None, None, 0) == bad
    assert moe_attn_forward(a.h, s.batch.desc, s.q.data_ptr() + 2, 256, s.out, 256, None, None, 0) == bad
    assert moe_attn_forward(a.h, s.batch.desc, None, 256, s.out, 256, None, None, 0) == bad
    assert moe_attn_forward(a.h, s.batch.desc, s.q, 256, s.out, 256, None, None, 0) == MOE_ERR_WORKSPACE
    ws, n = a.workspace(s.batch)
    assert moe_attn_forward(a.h, s.batch.desc, s.q, 256, s.out, 256, None, ws.data_ptr() + 16, n, None) == MOE_ERR_WORKSPACE
    x = s.q[:, :128].contiguous()
    sl = torch.zeros(2, dtype=torch.int32, device=DEV)
    assert a.append(2, x, None, sl) == bad and a.append(2, x, x, None) == bad and a.append(-1, x, x, sl) == bad
    assert a.append(0, None, None, None) == 0 and a.read(0, None, None, None) == 0
    assert a.read(2, None, x, x) == bad
    pos = torch.zeros(2, dtype=torch.int32, device=DEV)
    for rope in (Rope(_table(4, 64), 72), Rope(_table(4, 64), 24), Rope(_table(4, 64), 64, eps=-1.0),
                 Rope(_table(4, 64), 64, eps=math.nan), Rope(None, 64)):
        assert a.norm_rope(2, s.q, None, pos, rope, s.q, None) == bad
    rope = Rope(_table(4, 64), 64)
    assert a.norm_rope(2, s.q, None, None, rope, s.q, None) == bad
    assert a.norm_rope(2, s.q, None, pos, rope, None, None) == bad
    assert a.status() == 0


# ------------------------------------------------------------------ many query rows
@pytest.mark.parametrize("H,KV,d,page", [(8, 1, 128, 16), (16, 2, 64, 64), (6, 2, 128, 128), (33, 1, 64, 32)])
@pytest.mark.parametrize("window", [0, 1, 100, 200])
def test_many_rows_per_sequence(H, KV, d, page, window):
    """Column tiles of 128 and 256 begun, filled and passed; sequences without
    keys, with fewer keys than rows, and with keys that split over the SMs."""
    Setup(H, KV, d, page, [64, 3, 31, 40], [130, 700, 31, 0], seed=window + H, window=window).check()


def test_many_rows_long_keys_split_over_the_gpu():
    s = Setup(8, 1, 128, 32, [10, 9], [5000, 2600], seed=30)
    s.check()
    first = s.out.clone()
    s.run()
    assert torch.equal(first, s.out)


def test_many_rows_large_logits_and_value_magnitudes():
    Setup(8, 2, 128, 32, [40], [500], seed=31, q_scale=30.0).check()
    Setup(8, 2, 64, 32, [40], [300], seed=32, v_scale=1e30).check()
    Setup(8, 2, 128, 32, [40], [300], seed=33, v_scale=1e-30).check()
    Setup(8, 2, 128, 32, [40], [300], seed=34, v_exp=5).check()
    Setup(8, 2, 64, 32, [40], [200], seed=35, scale=-0.3).check()
    Setup(8, 2, 64, 32, [40], [200], seed=36, scale=0.0).check()


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("window", [0, 20])
def test_many_rows_non_finite_keys_values_queries(bad, window):
    from mxfp4_routed_expert_03_gb300 import check
    s = Setup(8, 2, 64, 16, [40], [200], seed=37, window=window)
    at = 170                               # seen by rows from 10 on (and, windowed, before 30)
    slot = (s.table[0, at // 16] * 16 + at % 16).view(1).int()
    k, v = _randn(1, 128, seed=97), _randn(1, 128, seed=96)
    s.k[0][at], s.v[0][at] = ref.mxfp4(k).view(2, 64), ref.mxfp4(v).view(2, 64)
    v[0, 64 + 40] = bad
    check(s.attn.append(1, k, v, slot), "append")
    last = 10 + window if window else 40
    o, l_, mag, big = s.want()
    hit = torch.zeros(40, 8, 64, dtype=torch.bool, device=DEV)
    hit[10:last, 4:, 32:] = True
    for step in range(3):
        if step == 1:                      # a key of head 0: its rows
            k[0, 3] = bad
            check(s.attn.append(1, k, v, slot), "append")
            hit[10:last, :4] = True
        if step == 2:                      # a query row of one head
            s.q[5, 6 * 64 + 1] = bad
            hit[5, 6] = True
        out, lse = s.run()
        assert s.attn.status() == 0
        out = out.double().view(40, 8, 64)
        assert bool(torch.isnan(out[hit]).all())
        ok = (out - o).abs() <= BF16_EPS * o.abs() + 2.0 ** -9 * mag
        assert bool(ok[~hit].all())


def test_many_rows_bad_pages_are_left_out():
    from mxfp4_routed_expert_03_gb300 import MOE_ERR_BAD_INDEX
    s = Setup(8, 2, 64, 16, [40], [200], seed=38)
    s.check()
    s.table[0, 2] = -1                     # tokens 32 .. 47
    s.run()
    assert s.attn.status() == MOE_ERR_BAD_INDEX
    keep = [j for j in range(200) if not 32 <= j < 48]
    s.k[0], s.v[0], s.kv = s.k[0][keep], s.v[0][keep], [184]
    o, l_, mag, big = s.want()             # (every row sits behind token 47)
    _close(s.out, s.lse, o.view(40, -1), l_, mag.view(40, -1), big)


def test_both_kernels_agree_at_their_border():
    """63 and 64 columns of the same sequence: the rows they share are the
    same to the bounds of either kernel."""
    for n in (63, 64):
        Setup(1, 1, 128, 16, [n], [300], seed=39).check()
