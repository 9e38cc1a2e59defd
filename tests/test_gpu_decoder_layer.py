"""The example decoder layer: prompt and decode steps through the library's calls against the
same layer computed in 64 bits from the same (cached, quantised) values.

The steps in between round to bf16 as the library does, so the attention output and the
routing are compared at the library's own inputs; the bounds are those of the single calls."""
import os
import sys

import numpy as np
import pytest
import torch

import attn_ref as ref
from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture()
def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import decoder_layer
    yield decoder_layer
    sys.path.remove(os.path.join(ROOT, "examples"))


def test_prompt_and_steps(example, monkeypatch):
    B, n, steps = 3, 37, 3
    layer = example.DecoderLayer(d_model=256, heads=8, kv_heads=2, head_dim=64, d_ff=128, experts=32, top_k=4,
                                 n_seqs=B, max_len=64, page=16)
    seen = []
    real = layer.attn.forward

    def forward(batch, q, out, lse=None, stream=None):
        rc = real(batch, q, out, lse, stream)
        seen.append((q.clone(), out.clone()))
        return rc
    monkeypatch.setattr(layer.attn, "forward", forward)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(B, n, 256, device="cuda", generator=g).bfloat16()
    y = layer.forward(x)
    outs = [y]
    for _ in range(steps):
        y = layer.forward(y[:, -1:])
        outs.append(y)
    layer.status()
    assert all(bool(torch.isfinite(o.float()).all()) for o in outs)
    # the cache after all steps, read back, holds what every step attended to
    total = n + steps
    slots = (layer.table[:, torch.arange(total) // 16] * 16 + torch.arange(total, device="cuda") % 16).int()
    k, v = (torch.empty(B * total, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert layer.attn.read(B * total, slots.flatten().contiguous(), k, v) == 0
    k, v = (t.double().view(B, total, 2, 64) for t in (k, v))
    at = n
    for i, (q, out) in enumerate(seen):
        rows = n if i == 0 else 1
        cu = [b * rows for b in range(B + 1)]
        o, _, mag, _ = ref.attention(q.double().reshape(B * rows, 8, 64), [k[b, :at] for b in range(B)],
                                     [v[b, :at] for b in range(B)], cu, [at] * B, 64 ** -0.5)
        err = (out.double().view(B * rows, 8, 64) - o).abs()
        assert bool((err <= 2.0 ** -8 * o.abs() + 2.0 ** -9 * mag).all())
        at += 1


def test_split_prompt_gives_the_whole_prompts_rows(example):
    """A prompt taken in as one piece and as two: the same cache, and outputs within rounding."""
    def run(parts):
        layer = example.DecoderLayer(d_model=256, heads=8, kv_heads=2, head_dim=64, d_ff=128, experts=32, top_k=4,
                                     n_seqs=2, max_len=64, page=16)
        g = torch.Generator(device="cuda").manual_seed(2)
        x = torch.randn(2, 48, 256, device="cuda", generator=g).bfloat16()
        out = [layer.forward(p) for p in x.split(parts, dim=1)]
        layer.status()
        return torch.cat(out, 1), {n: t.clone() for n, t in layer.attn.cache.items()}
    a, ca = run([48])
    b, cb = run([20, 27, 1])
    # (the projections' sums may round differently by shape: a few codes may differ)
    same = np.mean([float((ca[n] == cb[n]).float().mean()) for n in ca])
    assert same > 0.99
    scale = float(a.float().abs().max())
    # a token whose experts' scores lie within that rounding may be routed elsewhere
    close = ((a.float() - b.float()).abs().amax(-1) <= 2.0 ** -4 * scale)
    assert float(close.float().mean()) >= 0.9
