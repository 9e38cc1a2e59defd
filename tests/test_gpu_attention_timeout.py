"""The device-side timeout path of the attention kernels, driven on purpose.

With the test hook MOE_INJECT_ATTN_STALL the warp that copies the cache (few query rows) or
the first tile's MMA issuer (many) waits on a barrier that nothing signals, under a limit of 2e6
SM cycles (about a millisecond). The kernel must record MOE_ERR_DEVICE_TIMEOUT, wind down
(copies and products in flight end, tensor memory is freed) and return; the next call on the
same handle, with the hook off, must be right. No GPU fault is involved: the wait that runs
out is an ordinary bounded one."""
import pytest
import torch

from test_gpu_attention import Setup

pytestmark = pytest.mark.gpu

SHORT_LIMIT = 2_000_000


@pytest.mark.parametrize("H,KV,d,nq,kv", [
    (8, 1, 64, [1], [20000]), (8, 1, 128, [2, 2], [9000, 30000]), (8, 2, 128, [1] * 20, [700 + 90 * b for b in range(20)]),
    (8, 1, 64, [40], [5000]), (8, 2, 128, [64, 300, 20], [700, 900, 20]), (16, 1, 128, [20], [300])])
def test_stall_times_out_then_recovers(H, KV, d, nq, kv):
    from mxfp4_routed_expert_03_gb300 import (MOE_ERR_DEVICE_TIMEOUT, MOE_INJECT_ATTN_STALL, MOE_INJECT_NONE, check,
                                              moe_attn_set_fault_injection)
    s = Setup(H, KV, d, 32, nq, kv, seed=90)
    s.run()
    assert s.attn.status() == 0
    clean = s.out.clone()
    check(moe_attn_set_fault_injection(s.attn.h, MOE_INJECT_ATTN_STALL, SHORT_LIMIT), "inject")
    for _ in range(2):
        s.run()
        assert s.attn.status() == MOE_ERR_DEVICE_TIMEOUT
    check(moe_attn_set_fault_injection(s.attn.h, MOE_INJECT_NONE, 0), "inject off")
    s.out.fill_(7.0)
    s.check()
    assert torch.equal(s.out, clean)


def test_injection_arguments_are_checked():
    from mxfp4_routed_expert_03_gb300 import (MOE_ERR_INVALID_ARG, MOE_INJECT_ATTN_STALL, MOE_INJECT_GEMM_STALL,
                                              MOE_INJECT_NONE, moe_attn_set_fault_injection)
    s = Setup(4, 2, 64, 16, [1], [20], seed=91)
    for mode, limit in ((7, 0), (MOE_INJECT_GEMM_STALL, 0), (MOE_INJECT_ATTN_STALL, 1000), (MOE_INJECT_NONE, 99999)):
        assert moe_attn_set_fault_injection(s.attn.h, mode, limit) == MOE_ERR_INVALID_ARG
    assert moe_attn_set_fault_injection(None, MOE_INJECT_NONE, 0) == MOE_ERR_INVALID_ARG
    assert moe_attn_set_fault_injection(s.attn.h, MOE_INJECT_NONE, 0) == 0
    s.check()
