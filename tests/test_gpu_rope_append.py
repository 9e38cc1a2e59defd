"""moe_rope_append: the same bits as moe_qk_norm_rope followed by moe_kv_append."""
import pytest
import torch

pytestmark = pytest.mark.gpu

NAMES = ("k_q", "k_s", "v_q", "v_s")


def table(n_pos, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


class Setup:
    def __init__(self, T, H, KV, d, page, rot, interleaved=False, weights=True, seed=0, pages=None):
        from mxfp4_routed_expert_03_gb300.attention import Attention, Rope, alloc_kv_cache
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.H, self.KV, self.d = T, H, KV, d
        x = torch.randn(T, (H + 2 * KV) * d + 8, device="cuda", generator=g).bfloat16()
        self.q, self.k, self.v, _ = x.split([H * d, KV * d, KV * d, 8], dim=1)
        w = [(1 + 0.2 * torch.randn(d, device="cuda", generator=g)).bfloat16() if weights else None for _ in range(2)]
        self.rope = Rope(table(500, rot) if rot else None, rot, interleaved, 1e-6, *w)
        self.pos = torch.randint(500, (T,), device="cuda", generator=g, dtype=torch.int32)
        self.pages = pages or -(-T // page) + 3
        self.slots = torch.randperm(self.pages * page, device="cuda", generator=g)[:T].int()
        self.attn, self.other = (Attention(H, KV, d, page, self.pages, alloc_kv_cache(KV, d, page, self.pages)) for _ in range(2))

    def two_calls(self, live=None):
        """q_out and the cache as the two calls leave them (`live`: tokens that they are called for)."""
        from mxfp4_routed_expert_03_gb300 import check
        at = slice(None) if live is None else live
        q, k, v = (t[at].contiguous() for t in (self.q, self.k, self.v))
        k_out, q_out, n = torch.empty_like(k), torch.empty_like(q), q.shape[0]
        check(self.other.norm_rope(n, q, k, self.pos[at].contiguous(), self.rope, q_out, k_out), "moe_qk_norm_rope")
        check(self.other.append(n, k_out, v, self.slots[at].contiguous()), "moe_kv_append")
        return q_out

    def one(self, q_out, stream=None, **kw):
        args = dict(q=self.q, k=self.k, v=self.v, positions=self.pos, slots=self.slots) | kw
        return self.attn.rope_append(self.T, args["q"], args["k"], args["v"], args["positions"], self.rope, q_out,
                                     args["slots"], stream)

    def same_cache(self):
        torch.cuda.synchronize()
        return all(torch.equal(self.attn.cache[n], self.other.cache[n]) for n in NAMES)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 100, 1003])
@pytest.mark.parametrize("H,KV,d,rot,interleaved", [
    (8, 2, 128, 128, False), (8, 2, 128, 64, True), (3, 3, 128, 48, False), (56, 8, 128, 128, False), (4, 1, 64, 64, True),
    (6, 2, 64, 16, False), (16, 4, 64, 64, False), (5, 1, 128, 16, True), (12, 1, 128, 112, False), (40, 8, 64, 48, True)])
def test_same_bits_as_the_two_calls(T, H, KV, d, rot, interleaved):
    s = Setup(T, H, KV, d, 16, rot, interleaved, seed=T + rot)
    want = s.two_calls()
    q_out = torch.full((T, H * d), 7.0, dtype=torch.bfloat16, device="cuda")
    assert s.one(q_out) == 0 and s.attn.status() == 0
    assert torch.equal(q_out, want) and s.same_cache()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d", [64, 128])
def test_pages_and_consecutive_slots(page, d):
    s = Setup(777, 8, 4, d, page, d, seed=page)
    s.slots = (torch.arange(777, device="cuda") + page // 2 + 3).int()
    want = s.two_calls()
    q_out = torch.empty_like(want)
    assert s.one(q_out) == 0
    assert torch.equal(q_out, want) and s.same_cache()


@pytest.mark.parametrize("rot,weights", [(0, True), (0, False), (64, False)])
def test_without_rotation_or_norm(rot, weights):
    s = Setup(50, 8, 2, 64, 32, rot, weights=weights, seed=1)
    want = s.two_calls()
    q_out = torch.empty_like(want)
    assert s.one(q_out, positions=s.pos if rot else None) == 0
    assert torch.equal(q_out, want) and s.same_cache()


@pytest.mark.parametrize("d,interleaved", [(64, False), (128, False), (128, True)])
def test_against_64_bits(d, interleaved):
    """The values that attention reads: the rotated key within bf16's rounding and half a step of its
    block's 4-bit grid, the value within the latter. A step is at most 2 scales (between 4 and 6), above 6
    (up to 8) the distance to 6; bf16 and fp32 add 2^-8 and 2^-16 of the value."""
    from mxfp4_routed_expert_03_gb300 import check
    s = Setup(300, 8, 2, d, 16, d, interleaved, seed=2)
    q_out = torch.empty(300, 8 * d, dtype=torch.bfloat16, device="cuda")
    check(s.one(q_out), "moe_rope_append")
    tab = s.rope.tensors[0].double()[s.pos.long()]
    turn = torch.complex(tab[:, :d // 2], tab[:, d // 2:])[:, None]
    k, v = torch.empty(300, 2 * d, dtype=torch.bfloat16, device="cuda"), torch.empty(300, 2 * d, dtype=torch.bfloat16, device="cuda")
    check(s.attn.read(300, s.slots, k, v), "moe_kv_read")
    for x, w, got in ((s.q, s.rope.tensors[1], q_out), (s.k, s.rope.tensors[2], k), (s.v, None, v)):
        y = x.double().reshape(300, -1, d)
        if w is not None:
            y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.double()
            a, b = (y[..., 0::2], y[..., 1::2]) if interleaved else y.chunk(2, -1)
            z = torch.complex(a, b) * turn
            y = torch.stack([z.real, z.imag], -1).flatten(-2) if interleaved else torch.cat([z.real, z.imag], -1)
        y = y.reshape(300, -1)
        tol = y.abs() * (2.0 ** -8 + 2.0 ** -16) + 1e-6
        if got is not q_out:
            unit = torch.exp2(torch.floor(torch.log2(y.unflatten(1, (-1, 32)).abs().amax(2, keepdim=True))) - 2)
            u = y.unflatten(1, (-1, 32)).abs() / unit
            step = torch.where(u >= 4, torch.maximum(torch.ones_like(u), u - 6), torch.where(u >= 2, 0.5, 0.25))
            # (a rounding of the largest element may move the block's scale by one power of two)
            tol = tol + (step * unit * 1.05).flatten(1) * 2
        assert bool(((got.double() - y).abs() <= tol).all())


def cache_values(x):
    """What the cache holds of x [n][w] (bf16), in 64 bits: per 32 elements the scale 2^(floor(log2 max) - 2), at
    least 2^-127, and the nearest of E2M1's values, of two equally near ones that with the even code."""
    b = x.double().unflatten(1, (-1, 32))
    exponent = torch.frexp(b.abs().amax(2, keepdim=True))[1] - 3  # (frexp's fraction is in [1/2, 1))
    unit = torch.exp2(exponent.clamp(min=-127).double())
    levels = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    off = ((b / unit).abs()[..., None] - levels).abs()
    near = off == off.amin(-1, keepdim=True)
    even = near & (torch.arange(8, device=x.device) % 2 == 0)
    code = torch.where(even.any(-1), even.int().argmax(-1), near.int().argmax(-1))
    return (torch.copysign(levels[code], b) * unit).flatten(1)


@pytest.mark.parametrize("T", [5, 300])
@pytest.mark.parametrize("H,KV,d,rot,interleaved", [(8, 2, 64, 64, False), (8, 2, 128, 128, False), (3, 1, 128, 48, True)])
def test_the_cache_holds_the_nearest_values(T, H, KV, d, rot, interleaved):
    """Element for element, from the key rounded to bf16 and the value. The key is within half a step of bf16
    (2^-8 of it) and fp32's errors (under 60 roundings of the row's terms) of 64 bits."""
    from mxfp4_routed_expert_03_gb300 import check
    s = Setup(T, H, KV, d, 16, rot, interleaved, seed=10 + T)
    g = torch.Generator(device="cuda").manual_seed(T)
    # half of the values on a coarse grid: many are half-way between two codes, many block maxima powers of two
    s.v[:, :KV * d // 2] = (torch.randint(-32, 33, (T, KV * d // 2), device="cuda", generator=g) / 4).bfloat16()
    q_out, key = torch.empty(T, H * d, dtype=torch.bfloat16, device="cuda"), torch.empty(T, KV * d, dtype=torch.bfloat16, device="cuda")
    check(s.one(q_out), "moe_rope_append")
    check(s.other.norm_rope(T, None, s.k, s.pos, s.rope, None, key), "moe_qk_norm_rope")
    x = s.k.double().reshape(T, KV, d)
    x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * s.rope.tensors[2].double()
    tab = s.rope.tensors[0].double()[s.pos.long()]
    turn = torch.complex(tab[:, :rot // 2], tab[:, rot // 2:])[:, None]
    first, second = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, rot // 2), slice(rot // 2, rot))
    z, size = torch.complex(x[..., first], x[..., second]) * turn, x.abs()
    size[..., first] = size[..., second] = z.abs()
    x[..., first], x[..., second] = z.real, z.imag
    assert bool(((key.double().view_as(x) - x).abs() <= 2.0 ** -8 * x.abs() + 60 * 2.0 ** -24 * size).all())
    k, v = (torch.empty(T, KV * d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    check(s.attn.read(T, s.slots, k, v), "moe_kv_read")
    assert torch.equal(k.double(), cache_values(key)) and torch.equal(v.double(), cache_values(s.v))


@pytest.mark.parametrize("T", [200, 1300])
def test_skipped_tokens(T):
    s = Setup(T, 8, 2, 128, 16, 128, seed=3)
    s.slots[[0, 5, 77, T - 1]] = -1  # padding: the query is still turned
    live = s.slots >= 0
    s.two_calls(live)
    want = torch.empty(T, 8 * 128, dtype=torch.bfloat16, device="cuda")
    s.other.norm_rope(T, s.q, None, s.pos, s.rope, want, None)
    q_out = torch.full_like(want, 7.0)
    assert s.one(q_out) == 0 and s.attn.status() == 0
    assert torch.equal(q_out, want) and s.same_cache()


@pytest.mark.parametrize("T", [60, 1300])
def test_bad_slots_and_positions(T):
    """Slots outside the cache and positions outside the table: reported, left out."""
    from mxfp4_routed_expert_03_gb300 import MOE_ERR_BAD_INDEX
    for bad_slot in (-2, (-(-T // 16) + 3) * 16, 2 ** 31 - 1, -2 ** 31):
        t = Setup(T, 8, 2, 128, 16, 128, seed=4)
        t.slots[[3, 40]] = bad_slot
        ok = torch.ones(T, dtype=torch.bool, device="cuda")
        ok[[3, 40]] = False
        want = torch.empty(T, 8 * 128, dtype=torch.bfloat16, device="cuda")
        t.other.norm_rope(T, t.q, None, t.pos, t.rope, want, None)
        t.two_calls(ok)
        q_out = torch.full_like(want, 7.0)
        assert t.one(q_out) == 0 and t.attn.status() == MOE_ERR_BAD_INDEX and t.attn.status() == 0
        assert torch.equal(q_out, want) and t.same_cache()
    for bad_pos in (-1, 500, 2 ** 31 - 1, -2 ** 31):
        t = Setup(T, 8, 2, 64, 16, 64, seed=5)
        t.pos[[0, 33, T - 1]] = bad_pos
        ok = torch.ones(T, dtype=torch.bool, device="cuda")
        ok[[0, 33, T - 1]] = False
        want = torch.full((T, 8 * 64), 7.0, dtype=torch.bfloat16, device="cuda")
        want[ok] = t.two_calls(ok)
        q_out = torch.full_like(want, 7.0)
        assert t.one(q_out) == 0 and t.attn.status() == MOE_ERR_BAD_INDEX
        assert torch.equal(q_out, want) and t.same_cache()


def test_not_finite_values_stay_in_their_blocks():
    s = Setup(40, 4, 2, 64, 16, 32, seed=6)
    s.k[3, 70], s.v[4, 5], s.v[9, 100] = float("nan"), float("inf"), float("nan")
    want = s.two_calls()
    q_out = torch.empty_like(want)
    assert s.one(q_out) == 0
    assert torch.equal(q_out, want) and s.same_cache()


@pytest.mark.parametrize("T", [90, 1300])
def test_in_place_keys_alone_streams_and_graphs(T):
    s = Setup(T, 8, 2, 128, 32, 64, True, seed=7)
    s.two_calls()
    assert s.one(None, q=None) == 0 and s.same_cache()  # keys and values alone
    want = s.two_calls()
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    q = s.q.contiguous()
    keep = q.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        assert s.one(q, torch.cuda.current_stream(), q=q) == 0  # queries in place
    for n in NAMES:
        s.attn.cache[n].zero_()
    for _ in range(2):
        q.copy_(keep)
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q, want) and s.same_cache()


def test_untouched_memory():
    """Slots of other tokens, columns beside and rows behind the output stay as they were."""
    s = Setup(30, 4, 2, 64, 16, 64, seed=8)
    for c in (s.attn.cache, s.other.cache):
        for n in NAMES:
            c[n].fill_(0x31)
    want = s.two_calls()
    wide = torch.full((33, 4 * 64 + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    assert s.one(wide[:, 8:264]) == 0
    assert s.same_cache() and torch.equal(wide[:30, 8:264], want)
    wide[:30, 8:264] = 7.0
    assert bool((wide == 7.0).all())


def test_no_tokens_and_refusals():
    from mxfp4_routed_expert_03_gb300 import MOE_ERR_INVALID_ARG
    s = Setup(20, 4, 2, 64, 16, 64, seed=9)
    q_out = torch.full((20, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    assert s.attn.rope_append(0, s.q, s.k, s.v, s.pos, s.rope, q_out, s.slots) == 0
    for kw in (dict(k=None), dict(v=None), dict(slots=None), dict(positions=None), dict(q=None)):
        assert s.one(q_out, **kw) == MOE_ERR_INVALID_ARG
    assert s.one(None) == MOE_ERR_INVALID_ARG
    for kw in (dict(q=s.q[:19]), dict(k=s.k[:, :64]), dict(v=s.v.float()), dict(slots=s.slots.long()), dict(slots=s.slots[:19]),
               dict(positions=s.pos[:5]), dict(q=s.q.half()), dict(k=s.k.half()), dict(k=s.k.cpu()), dict(v=s.v.cpu()), dict(slots=s.slots.cpu()), dict(positions=s.pos.cpu())):
        with pytest.raises(ValueError):
            s.one(q_out, **kw)
    for bad in (q_out.cpu(), q_out.half(), q_out[:19]):
        with pytest.raises(ValueError):
            s.one(bad)
    from mxfp4_routed_expert_03_gb300.attention import Rope
    half = Rope(s.rope.tensors[0], 64, False, 1e-6, s.rope.tensors[1].half(), s.rope.tensors[2])
    with pytest.raises(ValueError):
        s.attn.rope_append(20, s.q, s.k, s.v, s.pos, half, q_out, s.slots)
    torch.cuda.synchronize()
    assert bool((q_out == 7.0).all()) and all(bool((s.attn.cache[n] == 0).all()) for n in NAMES)
