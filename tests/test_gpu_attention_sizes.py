"""Attention of many query rows at the sizes where its kernel changes: columns
between the two kernels' ranges, lengths around a unit (64 keys) and a step
(128 keys), and maxima that rise at chosen keys. References and tolerances are
test_gpu_attention's."""
import pytest
import torch

import attn_ref as ref
from test_gpu_attention import DEV, Setup, _randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,KV,d,nq", [(48, 2, 128, 1), (32, 2, 128, 1), (20, 2, 64, 2), (34, 2, 128, 1),
                                       (9, 1, 64, 7)])
@pytest.mark.parametrize("window", [0, 300])
def test_few_columns_in_a_large_batch(H, KV, d, nq, window):
    """16 to 63 columns, with fewer and with more than 4e6 logits."""
    kv = [3000, 1, 2999, 64, 0, 777] * 5
    Setup(H, KV, d, 64, [nq] * len(kv), [max(n, nq) if n else 0 for n in kv], seed=H + d, window=window).check()


@pytest.mark.parametrize("kv", [1, 2, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 640])
@pytest.mark.parametrize("d,page", [(128, 16), (64, 128)])
def test_lengths_around_a_unit_of_keys(kv, d, page):
    s = Setup(16, 1, d, page, [min(kv, 20), 9], [kv, kv + 9], seed=kv + d)
    s.check()
    first = s.out.clone()
    s.run()
    assert torch.equal(first, s.out)


def _refill(s, b, k):
    """Sequence b's keys again, as k (its values stay)."""
    from mxfp4_routed_expert_03_gb300 import check
    n = s.kv[b]
    j = torch.arange(n, device=DEV)
    slots = (s.table[b, j // s.page].long() * s.page + j % s.page).int()
    v = torch.empty(n, s.KV * s.d, dtype=torch.bfloat16, device=DEV)
    old = torch.empty_like(v)
    check(s.attn.read(n, slots, old, v), "read")
    check(s.attn.append(n, k, v, slots), "append")
    s.k[b] = ref.mxfp4(k).view(n, s.KV, s.d)


@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", ["rising", "falling", 63, 64, 130, 299])
def test_maximum_that_moves(at, d, window):
    """Keys that grow along the sequence, shrink along it, or stand out at one
    token, in a unit's last and first place and in the last unit."""
    s = Setup(8, 1, d, 32, [40], [300], seed=50, window=window)
    k = _randn(300, d, seed=51)
    if at == "rising":
        f = torch.linspace(0.01, 12, 300)
    elif at == "falling":
        f = torch.linspace(12, 0.01, 300)
    else:
        f = torch.full((300,), 0.1)
        f[at] = 20.0
    _refill(s, 0, (k.float() * f.to(DEV)[:, None]).bfloat16())
    s.check()


def test_workspace_of_the_bounds_serves_every_batch_within_them():
    from mxfp4_routed_expert_03_gb300 import moe_attn_workspace_bytes as need
    s = Setup(8, 1, 128, 64, [2], [4000], seed=60)
    sizes = [(n, n * q, q, kv) for n in (1, 16, 300) for q in (1, 2, 3, 8, 200) for kv in (100, 1000, 4000, 100000)]
    for small in sizes:
        for large in sizes:
            if all(a <= b for a, b in zip(small, large)):
                assert need(s.attn.h, *small) <= need(s.attn.h, *large)
    # 2 rows a sequence with the workspace of bounds that the other kernel serves
    s.attn._ws = torch.empty(need(s.attn.h, 300, 900, 3, 4000), dtype=torch.uint8, device=DEV)
    held = s.attn._ws.data_ptr()
    s.check()
    assert s.attn._ws.data_ptr() == held


def test_prompts_among_many_single_rows():
    """More than 32 sequences, few of which have many rows (most tiles of the
    longest sequence's number do not exist in the others)."""
    nq, kv = [1] * 40, [33 + b for b in range(40)]
    nq[3], kv[3] = 150, 333
    nq[38], kv[38] = 300, 301
    nq[39], kv[39] = 2, 0
    Setup(8, 2, 64, 32, nq, kv, seed=61).check()
    nq, kv = [33] * 34, [40 + 3 * b for b in range(34)]   # most tiles exist
    Setup(16, 2, 64, 32, nq, kv, seed=62).check()


@pytest.mark.parametrize("B", [160, 161, 333, 500])
@pytest.mark.parametrize("longest", [100, 129, 700])
def test_more_sequences_than_threads(B, longest):
    """Batches of one row and of a few rows a sequence that a block has to scan in rounds of
    160 sequences: whole items (up to 128 keys), and pieces of the line of all tiles. Lengths
    repeat irregularly, with empty sequences beside the rounds' ends."""
    kv = [1 + (37 * b * b + 11 * b) % longest for b in range(B)]
    for b in (0, 159, 160, 161, 319, 320, 332, 479, 480, B - 1):
        if b < B and b != 1:
            kv[b] = 0 if b % 2 else longest
    Setup(4, 2, 64, 32, [1] * B, kv, seed=B, single=True).check()
    nq = [1 + b % 3 for b in range(B)]
    Setup(4, 2, 64, 32, nq, kv, seed=B + 1, window=50).check()
