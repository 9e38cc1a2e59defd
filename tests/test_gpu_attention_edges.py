"""Attention where rows, tiles or pages hold nothing, and where a NaN must or must not
reach a row. References and tolerances are test_gpu_attention's unless a test says
otherwise."""
import math

import pytest
import torch

from test_gpu_attention import DEV, Setup

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
