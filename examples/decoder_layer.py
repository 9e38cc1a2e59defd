"""One decoder layer served by the library: projections in 8 bits, attention over a 4-bit cache,
then routed experts.

A batch of prompts is taken in (many rows per sequence), then decoded token by token (one row
per sequence), every step through the same calls:

  moe_add_norm (8-bit rows) -> moe_linear_forward (fused q/k/v) -> moe_rope_append ->
  moe_attn_forward -> moe_add_norm (8-bit rows, no norm) -> moe_linear_forward (output) ->
  moe_add_norm (residual, norm) -> moe_plan_scored -> moe_forward

    python examples/decoder_layer.py [--seqs 8] [--prompt 512] [--steps 64]

Weights are random.
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
from mxfp4_routed_expert_03_gb300.linear import Fp8Rows, Linear, Norm


def rope_table(n_pos: int, dim: int, base: float = 10000.0) -> torch.Tensor:
    """cos then sin of position x frequency, made in 64 bits: fp32 [n_pos][dim]."""
    f = base ** (-torch.arange(0, dim, 2, dtype=torch.float64, device="cuda") / dim)
    a = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def fp8_linear(w: torch.Tensor) -> Linear:
    """A projection of w [d_out][d_in], quantised to E4M3 with a scale per 128 x 128 block."""
    n, k = w.shape
    full = torch.nn.functional.pad(w.float(), (0, -k % 128, 0, -n % 128)).view(-(-n // 128), 128, -(-k // 128), 128)
    scale = (full.abs().amax((1, 3)) / 448).clamp(min=2.0 ** -126)
    codes = (full / scale[:, None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(-(-n // 128) * 128, -1)[:n, :k]
    return Linear(k, n, codes.contiguous(), scale.contiguous())


class DecoderLayer:
    """n_seqs sequences of up to max_len tokens; page p of sequence b is b * pages + p."""

    def __init__(self, d_model=1024, heads=16, kv_heads=4, head_dim=64, d_ff=256, experts=64, top_k=6,
                 n_seqs=8, max_len=1024, page=64, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda *s, std: (std * torch.randn(*s, device="cuda", generator=g)).bfloat16()  # noqa: E731
        self.d, self.H, self.KV, self.hd, self.n_seqs, self.page = d_model, heads, kv_heads, head_dim, n_seqs, page
        self.qkv = fp8_linear(rand((heads + 2 * kv_heads) * head_dim, d_model, std=d_model ** -0.5))
        self.out = fp8_linear(rand(d_model, heads * head_dim, std=(heads * head_dim) ** -0.5))
        self.norm_attn, self.norm_ffn = (Norm(d_model, weight=1 + rand(d_model, std=0.1)) for _ in range(2))
        self.to_8bit = Norm(heads * head_dim)  # (no weight: no norm)
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
        y8, qkv = Fp8Rows.empty(T, self.d), torch.empty(T, (self.H + 2 * self.KV) * W, dtype=torch.bfloat16, device="cuda")
        check(self.norm_attn.forward(T, rows, y8=y8, stream=st), "moe_add_norm")
        check(self.qkv.forward(T, y8, qkv, st), "moe_linear_forward")
        q, k, v = qkv.split([self.H * W, self.KV * W, self.KV * W], dim=1)
        pos = (self.length + torch.arange(n, device="cuda", dtype=torch.int32)).repeat(B)
        seq = torch.arange(B, device="cuda").repeat_interleave(n)
        slots = (self.table[seq, (pos // self.page).long()] * self.page + pos % self.page).int()
        check(self.attn.rope_append(T, q, k, v, pos, self.rope, q, slots, st), "moe_rope_append")  # q in place
        self.length += n
        self.k_len.fill_(self.length)
        cu = None if n == 1 else torch.arange(0, T + 1, n, device="cuda", dtype=torch.int32)
        batch = Batch(B, T, n, self.length, cu, self.k_len, self.table, W ** -0.5)
        out = torch.empty(T, self.H * W, dtype=torch.bfloat16, device="cuda")
        check(self.attn.forward(batch, q, out, None, st), "moe_attn_forward")
        o8, proj = Fp8Rows.empty(T, self.H * W), torch.empty_like(rows)
        check(self.to_8bit.forward(T, out, y8=o8, stream=st), "moe_add_norm")
        check(self.out.forward(T, o8, proj, st), "moe_linear_forward")
        h, z = torch.empty_like(rows), torch.empty_like(rows)
        check(self.norm_ffn.forward(T, proj, rows, total=h, y=z, stream=st), "moe_add_norm")
        plan = Plan(T, self.moe.E, self.moe.k)
        check(self.moe.plan_scored(T, None, z, plan, self.route, self.bias, st), "moe_plan_scored")
        y = torch.empty_like(h)
        check(self.moe.forward(T, z, plan, y, st), "moe_forward")
        return (h + y).view(B, n, self.d)

    def status(self) -> None:
        check(self.attn.status(torch.cuda.current_stream()), "attention")
        check(self.moe.status(torch.cuda.current_stream()), "experts")
        for linear in (self.qkv, self.out):
            check(linear.status(torch.cuda.current_stream()), "projections")


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
