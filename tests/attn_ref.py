"""Plain 64-bit references of the attention operators (tests only)."""
from __future__ import annotations

import numpy as np
import torch

from oracle.act_study import mx_quantise

DEV = "cuda"


def bf16(x):
    return x.to(torch.bfloat16)


def mxfp4(x: torch.Tensor) -> torch.Tensor:
    """The fp64 values that bf16 rows x [..., multiple of 32] have in MXFP4."""
    v = x.detach().double().cpu().numpy()
    return torch.from_numpy(np.ascontiguousarray(mx_quantise(v, "e2m1"))).to(x.device)


def attention(q, k, v, cu, kv, scale, window=0):
    """q fp64 [T][H][d]; k, v: per sequence fp64 [kv_b][KV][d]. Returns out,
    lse and, for error bounds, sum p |v| and the largest scale * sum |q_i k_i|."""
    T, H, d = q.shape
    out = torch.zeros(T, H, d, dtype=torch.float64, device=q.device)
    mag = torch.zeros_like(out)
    lse = torch.full((T, H), -float("inf"), dtype=torch.float64, device=q.device)
    big = 0.0
    for b, n in enumerate(kv):
        nq = cu[b + 1] - cu[b]
        for i in range(nq):
            p = n - nq + i
            lo = max(0, p - window + 1) if window else 0
            if p < 0:
                continue
            for h in range(H):
                g = h // (H // k[b].shape[1])
                kk, vv, qq = k[b][lo:p + 1, g], v[b][lo:p + 1, g], q[cu[b] + i, h]
                s = (kk @ qq) * scale
                w = torch.softmax(s, 0)
                out[cu[b] + i, h] = w @ vv
                # sum p |v|, and the 2^-25 that a weight below fp16's normal range may be off
                # by, carried at the weight of a 2^-9 error (see the callers' bounds)
                mag[cu[b] + i, h] = w @ vv.abs() + 2.0 ** -16 * vv.abs().sum(0)
                lse[cu[b] + i, h] = torch.logsumexp(s, 0)
                big = max(big, float((kk.abs() @ qq.abs()).max() * abs(scale)))
    return out, lse, mag, big


def norm_rope(x, w, eps, cos_sin, pos, rot, interleaved):
    """x fp64 [T][heads][d]."""
    y = x
    if w is not None:
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    y = y.clone()
    if rot:
        c, s = cos_sin.double()[pos.long()][:, None].chunk(2, -1)
        r = y[..., :rot].clone()
        a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else r.chunk(2, -1)
        u, v = a * c - b * s, b * c + a * s
        if interleaved:
            y[..., 0:rot:2], y[..., 1:rot:2] = u, v
        else:
            y[..., :rot] = torch.cat([u, v], -1)
    return y
