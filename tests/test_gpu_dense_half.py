"""The dense half of a decoder layer as it is used: norm, projection, rotation into the cache, attention,
output projection, norm with the residual; against the same steps in 64 bits.

Each step is compared at the library's own inputs (codes and scales, rounded rows, the cache as it reads
back), so the bounds are those of the single calls; the whole is one captured graph, replayed with new inputs."""
import pytest
import torch

import attn_ref
from linear_ref import U, bound, decode, product, weights

pytestmark = pytest.mark.gpu


class Half:
    """One sequence of `past` cached tokens to which T more come."""

    def __init__(self, T, past, d=512, H=8, KV=2, W=64, page=16, seed=0):
        from mxfp4_routed_expert_03_gb300.attention import Attention, Batch, Rope, alloc_kv_cache
        from mxfp4_routed_expert_03_gb300.linear import Fp8Rows, Linear, Norm
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.past, self.d, self.H, self.KV, self.W, self.g = T, past, d, H, KV, W, g
        self.n_qkv = (H + 2 * KV) * W
        self.w_qkv, self.w_out = weights(self.n_qkv, d, g), weights(d, H * W, g)
        self.qkv, self.out = Linear(d, self.n_qkv, *self.w_qkv), Linear(H * W, d, *self.w_out)
        self.gain = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).bfloat16()
        self.norm, self.to8, self.last = Norm(d, weight=self.gain), Norm(H * W), Norm(d, weight=self.gain)
        pages = -(-(past + T) // page)
        self.attn = Attention(H, KV, W, page, pages, alloc_kv_cache(KV, W, page, pages))
        f = 10000.0 ** (-torch.arange(0, W, 2, dtype=torch.float64, device="cuda") / W)
        a = torch.arange(past + T, dtype=torch.float64, device="cuda")[:, None] * f
        self.rope = Rope(torch.cat([a.cos(), a.sin()], 1).float(), W, q_weight=self.gain[:W].clone(), k_weight=self.gain[W:2 * W].clone())
        self.table = torch.randperm(pages, device="cuda", generator=g).int()[None].contiguous()
        tok = torch.arange(past + T, device="cuda")
        self.all_slots = (self.table[0, tok // page] * page + tok % page).int()
        bf = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        if past:
            k, v = (torch.randn(past, KV * W, device="cuda", generator=g).bfloat16() for _ in range(2))
            assert self.attn.append(past, k, v, self.all_slots) == 0
        self.pos = torch.arange(past, past + T, device="cuda", dtype=torch.int32)
        self.slots = self.all_slots[past:].contiguous()
        cu = torch.tensor([0, T], device="cuda", dtype=torch.int32)
        self.kv = torch.tensor([past + T], device="cuda", dtype=torch.int32)
        self.batch = Batch(1, T, T, past + T, cu, self.kv, self.table, W ** -0.5)
        self.x, self.x8, self.o8 = bf(T, d), Fp8Rows.empty(T, d), Fp8Rows.empty(T, H * W)
        self.rows, self.q, self.att, self.proj, self.total, self.y = bf(T, self.n_qkv), bf(T, H * W), bf(T, H * W), bf(T, d), bf(T, d), bf(T, d)

    def fill(self):
        self.x.copy_(torch.randn(self.T, self.d, device="cuda", generator=self.g))

    def run(self, st):
        from mxfp4_routed_expert_03_gb300 import check
        T, w = self.T, [self.H * self.W, self.KV * self.W, self.KV * self.W]
        check(self.norm.forward(T, self.x, y8=self.x8, stream=st))
        check(self.qkv.forward(T, self.x8, self.rows, st))
        q, k, v = self.rows.split(w, dim=1)
        check(self.attn.rope_append(T, q, k, v, self.pos, self.rope, self.q, self.slots, st))
        check(self.attn.forward(self.batch, self.q, self.att, None, st))
        check(self.to8.forward(T, self.att, y8=self.o8, stream=st))
        check(self.out.forward(T, self.o8, self.proj, st))
        check(self.last.forward(T, self.proj, self.x, self.total, self.y, stream=st))

    def verify(self):
        torch.cuda.synchronize()
        assert self.attn.status() == 0 and self.qkv.status() == 0 and self.out.status() == 0
        T, H, KV, W, d = self.T, self.H, self.KV, self.W, self.d
        norm = lambda h: h.double() / torch.sqrt(h.double().square().mean(1, keepdim=True) + 1e-6) * self.gain.double()  # noqa: E731
        # 8-bit rows: half a step of E4M3 (2^-4 of the value, 2^-10 of the scale near zero), beside fp32's errors
        for rows, want in ((self.x8, norm(self.x)), (self.o8, self.att.double())):
            got = decode(rows.q, rows.s)
            step = torch.maximum(want.abs() * 2.0 ** -4, rows.s.double().repeat_interleave(128, 1)[:, :want.shape[1]] * 2.0 ** -10)
            assert bool(((got - want).abs() <= step * (1 + 2.0 ** -10) + 100 * U * want.abs()).all())
        for rows, (wq, ws), got, k in ((self.x8, self.w_qkv, self.rows, d), (self.o8, self.w_out, self.proj, H * W)):
            ref, mag = product(rows.q, rows.s, wq, ws)
            assert bool(((got.double() - ref).abs() <= bound(ref, mag, k, torch.bfloat16)).all())
        n = self.past + T
        k, v = (torch.empty(n, KV * W, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        assert self.attn.read(n, self.all_slots, k, v) == 0
        o, _, mag, _ = attn_ref.attention(self.q.double().view(T, H, W), [k.double().view(n, KV, W)], [v.double().view(n, KV, W)],
                                          [0, T], [n], W ** -0.5)
        assert bool(((self.att.double().view(T, H, W) - o).abs() <= 2.0 ** -8 * o.abs() + 2.0 ** -9 * mag).all())
        assert torch.equal(self.total, (self.proj.float() + self.x.float()).bfloat16())
        want = norm(self.total)
        assert bool(((self.y.double() - want).abs() <= (2.0 ** -8 + 120 * U) * want.abs() + 1e-30).all())


@pytest.mark.parametrize("T,past", [(1, 0), (1, 300), (7, 40), (90, 0), (200, 77)])
def test_steps_in_a_graph(T, past):
    h = Half(T, past, seed=T)
    st = torch.cuda.Stream()
    h.fill()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        h.run(st)  # (sizes the attention's workspace of this stream)
    torch.cuda.synchronize()
    h.verify()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        h.run(torch.cuda.current_stream())
    for _ in range(3):
        h.fill()
        graph.replay()
        h.verify()
