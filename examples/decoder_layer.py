"""One decoder layer served by the library: attention over a 4-bit cache, then routed experts.

A batch of prompts is taken in (many rows per sequence), then decoded token by token (one row
per sequence), every step through the same calls:

  fused q/k/v projection (torch) -> moe_qk_norm_rope -> moe_kv_append -> moe_attn_forward ->
  output projection (torch) -> moe_plan_scored -> moe_forward

    python examples/decoder_layer.py [--seqs 8] [--prompt 512] [--steps 64]

Weights are random; the layer's own norms are left out to keep the calls in view.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from mxfp4_routed_expert_03_gb300 import MOE_ROUTER_XWR, MOE_SCORE_SIGMOID, check, moe_route_desc
from mxfp4_routed_expert_03_gb300.attention import Attention, Batch, Rope, alloc_kv_cache
from mxfp4_routed_expert_03_gb300.layer import Layer, Plan, alloc_weights


def rope_table(n_pos: int, dim: int, base: float = 10000.0) -> torch.Tensor:
    """cos then sin of position x frequency, made in 64 bits: fp32 [n_pos][dim]."""
    f = base ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    a = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


class DecoderLayer:
    """n_seqs sequences of up to max_len tokens; page p of sequence b is b * pages + p."""

    def __init__(self, d_model=1024, heads=16, kv_heads=4, head_dim=64, d_ff=256, experts=64, top_k=6,
                 n_seqs=8, max_len=1024, page=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s, std: (std * torch.randn(*s, device="cuda", generator=g)).bfloat16()  # noqa: E731
        self.d, self.H, self.KV, self.hd, self.n_seqs, self.page = d_model, heads, kv_heads, head_dim, n_seqs, page
        self.w_qkv = rand(d_model, (heads + 2 * kv_heads) * head_dim, std=d_model ** -0.5)
        self.w_out = rand(heads * head_dim, d_model, std=(heads * head_dim) ** -0.5)
        self.rope = Rope(rope_table(max_len, head_dim), head_dim, q_weight=1 + rand(head_dim, std=0.1),
                         k_weight=1 + rand(head_dim, std=0.1))
        self.pages = -(-max_len // page)
        self.attn = Attention(heads, kv_heads, head_dim, page, n_seqs * self.pages,
                              alloc_kv_cache(kv_heads, head_dim, page, n_seqs * self.pages))
        self.table = torch.arange(n_seqs * self.pages, device="cuda", dtype=torch.int32).view(n_seqs, -1)
        weights = alloc_weights(experts, d_model, d_ff)
        for name, t in weights.items():
            lo, hi = (0, 256) if name.endswith("_q") else (117, 121)  # codes; scales 2^-10 .. 2^-7
            t.copy_(torch.randint(lo, hi, t.shape, device="cuda", generator=g, dtype=torch.uint8))
        self.w_router = torch.randn(experts, d_model, device="cuda", generator=g) * d_model ** -0.5
        self.moe = Layer(d_model, d_ff, experts, top_k, weights, router_mode=MOE_ROUTER_XWR, w_router=self.w_router)
        # groups of 8 experts, half of them open to a token, weights that sum to 1
        self.route = moe_route_desc(MOE_SCORE_SIGMOID, experts // 8, experts // 16, 2, 1, 1.0)
        self.bias = 0.02 * torch.randn(experts, device="cuda", generator=g)
        self.k_len = torch.zeros(n_seqs, dtype=torch.int32, device="cuda")
        self.length = 0

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        """x: bf16 [n_seqs][n][d_model], the next n tokens of every sequence. Returns the same shape."""
        B, n, _ = x.shape
        T, W = B * n, self.hd
        rows = x.reshape(T, self.d)
        st = torch.cuda.current_stream()
        qkv = rows @ self.w_qkv
        q, k, v = qkv.split([self.H * W, self.KV * W, self.KV * W], dim=1)
        pos = (self.length + torch.arange(n, device="cuda", dtype=torch.int32)).repeat(B)
        check(self.attn.norm_rope(T, q, k, pos, self.rope, q, k, st), "moe_qk_norm_rope")  # in place
        seq = torch.arange(B, device="cuda").repeat_interleave(n)
        slots = (self.table[seq, (pos // self.page).long()] * self.page + pos % self.page).int()
        check(self.attn.append(T, k, v, slots, st), "moe_kv_append")
        self.length += n
        self.k_len.fill_(self.length)
        cu = None if n == 1 else torch.arange(0, T + 1, n, device="cuda", dtype=torch.int32)
        batch = Batch(B, T, n, self.length, cu, self.k_len, self.table, W ** -0.5)
        out = torch.empty(T, self.H * W, dtype=torch.bfloat16, device="cuda")
        check(self.attn.forward(batch, q, out, None, st), "moe_attn_forward")
        h = rows + out @ self.w_out
        plan = Plan(T, self.moe.E, self.moe.k)
        check(self.moe.plan_scored(T, None, h, plan, self.route, self.bias, st), "moe_plan_scored")
        y = torch.empty_like(h)
        check(self.moe.forward(T, h, plan, y, st), "moe_forward")
        return (h + y).view(B, n, self.d)

    def status(self) -> None:
        check(self.attn.status(torch.cuda.current_stream()), "attention")
        check(self.moe.status(torch.cuda.current_stream()), "experts")


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--seqs", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=512)
    ap.add_argument("--steps", type=int, default=64)
    a = ap.parse_args()
    layer = DecoderLayer(n_seqs=a.seqs, max_len=a.prompt + a.steps)
    x = torch.randn(a.seqs, a.prompt, layer.d, device="cuda").bfloat16()
    e = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
    layer.forward(x[:, :1])  # loads the kernels
    layer.length = 0
    e[0].record()
    y = layer.forward(x)[:, -1:]
    e[1].record()
    for _ in range(a.steps):
        y = layer.forward(y)
    e[2].record()
    layer.status()
    print(f"prompt: {a.seqs} x {a.prompt} tokens in {e[0].elapsed_time(e[1]):.2f} ms; "
          f"decode: {e[1].elapsed_time(e[2]) / a.steps * 1e3:.0f} us a step; |y| {float(y.float().norm()):.3f}")


if __name__ == "__main__":
    main()
