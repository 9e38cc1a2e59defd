"""moe_linear_forward: E4M3 rows times E4M3 weights with block scales, against 64 bits."""
import pytest
import torch

from linear_ref import bound, product, quantised, weights

pytestmark = pytest.mark.gpu

E4M3 = torch.float8_e4m3fn


class Setup:
    def __init__(self, T, K, N, seed=0, dtype=torch.bfloat16):
        from mxfp4_routed_expert_03_gb300.linear import Fp8Rows, Linear
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.K, self.N, self.dtype = T, K, N, dtype
        self.wq, self.ws = weights(N, K, g)
        self.xq, self.xs = quantised(T, K, g)
        self.linear = Linear(K, N, self.wq, self.ws)
        self.rows = Fp8Rows(self.xq, self.xs)
        self.out = torch.full((T, N), 7.0, dtype=dtype, device="cuda")

    def run(self, stream=None):
        from mxfp4_routed_expert_03_gb300 import check
        check(self.linear.forward(self.T, self.rows, self.out, stream), "moe_linear_forward")

    def verify(self, out=None):
        assert self.linear.status() == 0
        ref, mag = product(self.xq, self.xs, self.wq, self.ws)
        off = ((self.out if out is None else out).double() - ref).abs()
        assert bool((off <= bound(ref, mag, self.K, self.dtype)).all()), float((off / bound(ref, mag, self.K, self.dtype)).max())


# tokens around every tile's edge, from one to several tiles
TOKENS = [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 255, 256, 257, 300, 511, 513, 1000]


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("K,N", [(256, 384), (1040, 776)])
def test_tokens(T, K, N):
    s = Setup(T, K, N, seed=T)
    s.run()
    s.verify()


@pytest.mark.parametrize("K,N", [(16, 8), (32, 16), (112, 120), (128, 128), (144, 136), (2048, 8), (16, 2000),
                                 (7168, 264), (4096, 1000), (1536, 4096), (7168, 7168), (65536, 128), (128, 20000)])
@pytest.mark.parametrize("T,dtype", [(1, torch.bfloat16), (5, torch.float32), (40, torch.bfloat16),
                                     (140, torch.float32), (600, torch.bfloat16)])
def test_shapes(T, K, N, dtype):
    s = Setup(T, K, N, seed=1, dtype=dtype)
    s.run()
    s.verify()


@pytest.mark.parametrize("T,K,N", [(3000, 7168, 9216), (2049, 4096, 1000), (4100, 512, 2560)])
def test_prefill(T, K, N):
    s = Setup(T, K, N, seed=2, dtype=torch.float32)
    s.run()
    s.verify()


# K shared by 2 to 8 CTAs; rows that these do not divide, or fewer of them
@pytest.mark.parametrize("T", [1, 3, 13, 27, 61])
@pytest.mark.parametrize("K,N", [(1040, 13000), (2304, 10240), (1536, 7168), (2560, 5120), (4096, 5120), (4096, 4864), (4096, 4096)])
def test_shared_by_any_number(T, K, N):
    s = Setup(T, K, N, seed=15)
    s.run()
    s.verify()


# tiles of fewer rows than there are, the last one cut
@pytest.mark.parametrize("T", [18, 33, 47, 64, 67, 95, 97, 128, 131, 200, 257, 350])
@pytest.mark.parametrize("K,N,dtype", [(1040, 776, torch.bfloat16), (4096, 1000, torch.float32), (7168, 264, torch.bfloat16),
                                       (512, 4096, torch.bfloat16), (2048, 2048, torch.float32)])
def test_tiles_of_fewer_rows(T, K, N, dtype):
    s = Setup(T, K, N, seed=18, dtype=dtype)
    s.run()
    s.verify()


@pytest.mark.parametrize("T,K,N", [(209, 7168, 896), (257, 7168, 896), (245, 8192, 1408), (385, 4096, 1000), (260, 4096, 2048),
                                   (129, 4096, 4096), (100, 4096, 5120), (127, 2560, 5000), (70, 4096, 6400)])
def test_many_rows_shared_by_any_number(T, K, N):
    s = Setup(T, K, N, seed=16, dtype=torch.float32)
    s.run()
    s.verify()


@pytest.mark.parametrize("T", [1, 20, 70, 200, 700])
def test_whole_numbers_are_exact(T):
    """Small whole codes and scales that are powers of two: every sum is a whole number of at most 24
    bits, so nothing is rounded, wherever a row, a column or a block of 128 lies."""
    from mxfp4_routed_expert_03_gb300 import check
    from mxfp4_routed_expert_03_gb300.linear import Fp8Rows, Linear
    K, N = 1296, 392
    g = torch.Generator(device="cuda").manual_seed(T)
    whole = lambda *s: torch.randint(-3, 4, s, device="cuda", generator=g).float()  # noqa: E731
    pow2 = lambda *s: torch.randint(0, 3, s, device="cuda", generator=g).float().exp2()  # noqa: E731
    xq, wq, kb = whole(T, K).to(E4M3), whole(N, K).to(E4M3), -(-K // 128)
    xs, ws = pow2(T, kb), pow2(-(-N // 128), kb)
    out = torch.empty(T, N, device="cuda")
    linear = Linear(K, N, wq, ws)
    check(linear.forward(T, Fp8Rows(xq, xs), out), "moe_linear_forward")
    assert torch.equal(out.double(), product(xq, xs, wq, ws)[0])


@pytest.mark.parametrize("T", [1, 6, 50, 130, 400])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_rows_and_untouched_memory(T, dtype):
    """Rows cut out of wider ones, more rows than tokens: what lies around the output stays."""
    from mxfp4_routed_expert_03_gb300 import check
    from mxfp4_routed_expert_03_gb300.linear import Fp8Rows
    s = Setup(T, 400, 264, seed=3, dtype=dtype)
    codes = torch.full((T + 3, 512), 0x7F, dtype=torch.uint8, device="cuda")  # NaN wherever it is not a row
    codes[:T, 16:416] = s.xq.view(torch.uint8)
    scales = torch.full((T + 3, 9), float("nan"), device="cuda")
    scales[:T, 2:6] = s.xs
    out = torch.full((T + 2, 296), 7.0, dtype=dtype, device="cuda")
    rows = Fp8Rows(codes.view(E4M3)[:, 16:416], scales[:, 2:6])
    check(s.linear.forward(T, rows, out[:, 16:280]), "moe_linear_forward")
    s.verify(out[:T, 16:280])
    out[:T, 16:280] = 7.0
    assert bool((out == 7.0).all())


@pytest.mark.parametrize("T", [1, 12, 60, 150, 500])
def test_what_is_not_finite_stays_where_it_belongs(T):
    s = Setup(T, 640, 520, seed=4, dtype=torch.float32)
    t, n = T // 2, 300
    s.xq.view(torch.uint8)[t, 77] = 0x7F
    s.wq.view(torch.uint8)[n, 130] = 0xFF
    s.xs[T - 1, 4] = float("inf")
    s.ws[3, 2] = float("nan")  # columns 384 .. 511
    s.run()
    ref, mag = product(s.xq, s.xs, s.wq, s.ws)
    assert torch.equal(s.out.isfinite(), ref.isfinite())
    fine = ref.isfinite()
    assert bool(((s.out.double() - ref).abs() <= bound(ref, mag, 640, s.dtype))[fine].all())


@pytest.mark.parametrize("T", [1, 16, 64, 333])
def test_zero_scales_and_zero_codes(T):
    s = Setup(T, 384, 256, seed=5)
    s.xs.zero_()
    s.run()
    assert bool((s.out == 0).all())
    s.xs.fill_(1.0)
    s.xq.view(torch.uint8).fill_(0x80)  # negative zeros
    s.run()
    assert bool((s.out == 0).all())


@pytest.mark.parametrize("T", [1, 8, 48, 100, 260, 900])
def test_same_bits_again_and_in_any_batch(T):
    """Repeated calls give the same bits; so do calls on two streams at a time."""
    a = Setup(T, 2048, 1024, seed=6)
    a.run()
    first = a.out.clone()
    other = Setup(T, 2048, 1024, seed=7)
    other.run()
    want = other.out.clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        a.out.fill_(0)
        other.out.fill_(0)
        torch.cuda.synchronize()
        for _ in range(4):
            a.run(streams[0])
            other.run(streams[1])
        torch.cuda.synchronize()
        assert torch.equal(a.out, first) and torch.equal(other.out, want)


@pytest.mark.parametrize("T", [1, 33, 300])
def test_captured_and_replayed_with_changed_inputs(T):
    """A graph reads the codes, scales and weights of the time of its replay."""
    s = Setup(T, 1152, 640, seed=8)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        s.run(st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        s.run(torch.cuda.current_stream())
    new = Setup(T, 1152, 640, seed=9)
    for mine, fresh in ((s.xq, new.xq), (s.xs, new.xs), (s.wq, new.wq), (s.ws, new.ws)):
        mine.view(torch.uint8).copy_(fresh.view(torch.uint8))
    s.out.fill_(0)
    graph.replay()
    torch.cuda.synchronize()
    s.verify()


# several waves of tiles: a pair of CTAs on 256 x 256, one and several tiles a pair, ragged in both directions
LARGE = [(400, 2064, 6000), (512, 2048, 5120), (1500, 2048, 7000), (3000, 1552, 5008)]


@pytest.mark.parametrize("T,K,N", LARGE)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large(T, K, N, dtype):
    s = Setup(T, K, N, seed=20, dtype=dtype)
    s.run()
    s.verify()
    first = s.out.clone()
    s.out.fill_(0)
    s.run()
    assert torch.equal(s.out, first)


@pytest.mark.parametrize("T,K,N", LARGE)
def test_large_whole_numbers_are_exact(T, K, N):
    from mxfp4_routed_expert_03_gb300 import check
    from mxfp4_routed_expert_03_gb300.linear import Fp8Rows, Linear
    g = torch.Generator(device="cuda").manual_seed(T)
    xq = torch.randint(-3, 4, (T, K), device="cuda", generator=g).float().to(E4M3)
    wq = torch.randint(-3, 4, (N, K), device="cuda", generator=g).float().to(E4M3)
    xs = torch.randint(0, 3, (T, -(-K // 128)), device="cuda", generator=g).float().exp2()
    ws = torch.randint(0, 3, (-(-N // 128), -(-K // 128)), device="cuda", generator=g).float().exp2()
    out = torch.empty(T, N, device="cuda")
    linear = Linear(K, N, wq, ws)
    check(linear.forward(T, Fp8Rows(xq, xs), out), "moe_linear_forward")
    assert torch.equal(out.double(), product(xq, xs, wq, ws)[0])


@pytest.mark.parametrize("T,K,N", [(512, 1408, 9728), (500, 1536, 9704), (1000, 1024, 9728), (8192, 384, 4864), (8000, 512, 4800)])
def test_pairs_with_few_blocks_end_and_start_again(T, K, N):
    """11 to 32 blocks of K for a pair of CTAs, odd and even, in one and several tiles. The last blocks of a
    pair have none behind them that would use their accumulators again, and tell nobody that they have read them;
    the next call's CTAs come to the same SMs right behind. Whole numbers, so every call is exact."""
    from mxfp4_routed_expert_03_gb300 import check
    from mxfp4_routed_expert_03_gb300.linear import Fp8Rows, Linear
    g = torch.Generator(device="cuda").manual_seed(K)
    xq = torch.randint(-3, 4, (T, K), device="cuda", generator=g).float().to(E4M3)
    wq = torch.randint(-3, 4, (N, K), device="cuda", generator=g).float().to(E4M3)
    xs, ws = torch.ones(T, -(-K // 128), device="cuda"), torch.ones(-(-N // 128), -(-K // 128), device="cuda")
    out = [torch.empty(T, N, device="cuda") for _ in range(2)]
    linear, rows = Linear(K, N, wq, ws), Fp8Rows(xq, xs)
    want = product(xq, xs, wq, ws)[0]
    for k in range(40):
        check(linear.forward(T, rows, out[k % 2]), "moe_linear_forward")
    assert linear.status() == 0 and all(torch.equal(o.double(), want) for o in out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_large_strided_and_not_finite(dtype):
    from mxfp4_routed_expert_03_gb300 import check
    T, K, N = 700, 2064, 6008
    s = Setup(T, K, N, seed=21, dtype=dtype)
    s.xq.view(torch.uint8)[333, 77] = 0x7F
    s.wq.view(torch.uint8)[5000, 130] = 0xFF
    s.xs[T - 1, 4] = float("inf")
    s.ws[3, 2] = float("nan")
    out = torch.full((T + 2, N + 40), 7.0, dtype=dtype, device="cuda")
    check(s.linear.forward(T, s.rows, out[:, 16:16 + N]), "moe_linear_forward")
    got = out[:T, 16:16 + N].clone()
    ref, mag = product(s.xq, s.xs, s.wq, s.ws)
    fine = ref.isfinite()
    assert torch.equal(got.isfinite(), fine)
    assert bool(((got.double() - ref).abs() <= bound(ref, mag, K, dtype))[fine].all())
    out[:T, 16:16 + N] = 7.0
    assert bool((out == 7.0).all())


def test_large_on_two_streams_and_in_a_graph():
    a, b = Setup(600, 2048, 6000, seed=22), Setup(600, 2048, 6000, seed=23)
    a.run()
    b.run()
    want = a.out.clone(), b.out.clone()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[1]):
        b.run(torch.cuda.current_stream())
    for _ in range(5):
        a.out.fill_(0)
        b.out.fill_(0)
        torch.cuda.synchronize()
        for _ in range(3):
            a.run(streams[0])
            with torch.cuda.stream(streams[1]):
                graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])


def test_weights_written_right_before_the_call_count():
    """The weights' last writer may be the call before in the same stream."""
    T, K, N = 4, 7168, 7168
    s = Setup(T, K, N, seed=10)
    new = Setup(T, K, N, seed=11)
    new.run()
    for _ in range(3):
        s.wq.view(torch.uint8).zero_()
        s.run()
        assert bool((s.out == 0).all())
        s.wq.view(torch.uint8).copy_(new.wq.view(torch.uint8))
        s.ws.copy_(new.ws)
        s.xq.view(torch.uint8).copy_(new.xq.view(torch.uint8))
        s.xs.copy_(new.xs)
        s.run()
        torch.cuda.synchronize()
        assert torch.equal(s.out, new.out)


def test_as_many_rows_as_are_taken():
    """2^31 - 513 rows of 16 (77 GB); one more is refused."""
    from mxfp4_routed_expert_03_gb300 import MOE_ERR_UNSUPPORTED, check, moe_linear_forward
    from mxfp4_routed_expert_03_gb300.linear import Fp8Rows
    T = 2 ** 31 - 1 - 512
    if torch.cuda.mem_get_info()[0] < 90e9:
        pytest.skip("needs 90 GB")
    s = Setup(5, 16, 8, seed=17)
    rows = Fp8Rows(torch.zeros(T, 16, dtype=torch.uint8, device="cuda"), torch.ones(T, 1, device="cuda"))
    some = torch.tensor([0, 2 ** 27 + 1, 2 ** 30, T - 129, T - 1], device="cuda")
    rows.q[some], rows.s[some] = s.xq.view(torch.uint8), s.xs
    out = torch.empty(T, 8, dtype=torch.bfloat16, device="cuda")
    assert moe_linear_forward(s.linear.h, T + 1, rows.desc, out, 8, 0) == MOE_ERR_UNSUPPORTED
    check(s.linear.forward(T, rows, out), "moe_linear_forward")
    s.verify(out[some])
    out[some] = 0
    for part in (out[:1000], out[2 ** 30 - 500:2 ** 30 + 500], out[-1000:]):
        assert bool((part == 0).all())
    del rows, out, part
    torch.cuda.empty_cache()


@pytest.mark.parametrize("T,K,N", [(3, 512, 512), (100, 512, 512), (300, 1536, 7168)])
def test_the_kernel_before_may_take_long(T, K, N):
    """A product that starts beside a long one on the SMs that this leaves free, and waits for its end,
    counts none of that as a wait that ran out (limit: 1e5 cycles, 48 us or more; the long one reads 671 MB on
    80 SMs, so it takes over 80 us)."""
    from mxfp4_routed_expert_03_gb300 import MOE_INJECT_NONE, check, moe_linear_set_fault_injection
    from mxfp4_routed_expert_03_gb300.linear import Fp8Rows, Linear
    n, k = 10240, 65536
    codes = torch.randint(0, 0x40, (n + 100, k), device="cuda", dtype=torch.uint8)
    scales = torch.ones(100, k // 128, device="cuda")
    long = Linear(k, n, codes[:n], torch.ones(n // 128, k // 128, device="cuda"))
    long_x, long_out = Fp8Rows(codes[n:], scales), torch.empty(100, n, dtype=torch.bfloat16, device="cuda")
    s = Setup(T, K, N, seed=14)
    s.run()
    want = s.out.clone()
    check(moe_linear_set_fault_injection(s.linear.h, MOE_INJECT_NONE, 100_000), "limit")
    for _ in range(3):
        s.out.fill_(0)
        check(long.forward(100, long_x, long_out), "moe_linear_forward")
        s.run()
        assert long.status() == 0 and s.linear.status() == 0
        assert torch.equal(s.out, want)


def test_no_tokens_and_refusals():
    from mxfp4_routed_expert_03_gb300 import MOE_ERR_INVALID_ARG, moe_linear_forward
    from mxfp4_routed_expert_03_gb300.linear import Fp8Rows, Linear
    s = Setup(4, 256, 128, seed=12)
    assert s.linear.forward(0, s.rows, s.out) == 0
    assert bool((s.out == 7.0).all())
    for bad in (s.out[:3], s.out[:, :64], s.out.half(), s.out.double(), s.out.cpu(), s.out.t()):
        with pytest.raises(ValueError):
            s.linear.forward(4, s.rows, bad)
    with pytest.raises(ValueError):
        s.linear.forward(5, s.rows, torch.empty(5, 128, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        s.linear.forward(4, Fp8Rows.empty(4, 240), s.out)
    with pytest.raises(ValueError):
        Fp8Rows(s.xq, s.xs[:, :1])
    with pytest.raises(ValueError):
        Fp8Rows(s.xq, s.xs.double())
    with pytest.raises(ValueError):
        Fp8Rows(s.xq.float(), s.xs)
    with pytest.raises(ValueError):
        Fp8Rows(s.xq, s.xs.cpu())
    with pytest.raises(ValueError):
        Linear(256, 128, s.wq[:, :128], s.ws)
    with pytest.raises(ValueError):
        Linear(256, 128, s.wq.cpu(), s.ws.cpu())
    wide = torch.empty(4, 300, dtype=torch.bfloat16, device="cuda")
    for out in (wide[:, 1:129], wide[:, :128]):  # unaligned base, row stride 300
        assert s.linear.forward(4, s.rows, out) == MOE_ERR_INVALID_ARG
    assert moe_linear_forward(s.linear.h, 4, s.rows.desc, s.out, 128, 2) == MOE_ERR_INVALID_ARG
    assert s.linear.forward(4, None, s.out) == MOE_ERR_INVALID_ARG and s.linear.forward(4, s.rows, None) == MOE_ERR_INVALID_ARG
    assert s.linear.forward(-1, s.rows, s.out) == MOE_ERR_INVALID_ARG
    s.run()
    s.verify()


@pytest.mark.parametrize("T,K,N", [(1, 2048, 1400), (40, 2048, 1400), (40, 2048, 5120), (100, 2048, 1400), (140, 2048, 1400),
                                   (200, 2048, 1400), (245, 8192, 1408), (100, 4096, 5120), (600, 2048, 1400),
                                   (500, 2048, 5120), (1500, 2048, 7000)])
def test_stall_times_out_then_recovers(T, K, N):
    """With the test hook an MMA issuer waits, under a limit of 2e6 SM cycles, on a barrier that
    nothing signals: the status is recorded, copies and products in flight end, tensor memory is
    freed, and the next call is right. No GPU fault is involved."""
    from mxfp4_routed_expert_03_gb300 import (MOE_ERR_DEVICE_TIMEOUT, MOE_ERR_INVALID_ARG, MOE_INJECT_ATTN_STALL,
                                              MOE_INJECT_LINEAR_STALL, MOE_INJECT_NONE, check, moe_linear_set_fault_injection)
    s = Setup(T, K, N, seed=13)
    s.run()
    clean = s.out.clone()
    for mode, limit in ((7, 0), (MOE_INJECT_ATTN_STALL, 0), (MOE_INJECT_LINEAR_STALL, 1000)):
        assert moe_linear_set_fault_injection(s.linear.h, mode, limit) == MOE_ERR_INVALID_ARG
    check(moe_linear_set_fault_injection(s.linear.h, MOE_INJECT_LINEAR_STALL, 2_000_000), "inject")
    for _ in range(2):
        s.run()
        assert s.linear.status() == MOE_ERR_DEVICE_TIMEOUT
    check(moe_linear_set_fault_injection(s.linear.h, MOE_INJECT_NONE, 0), "inject off")
    s.out.fill_(7.0)
    s.run()
    s.verify()
    assert torch.equal(s.out, clean)


@pytest.mark.parametrize("T,K,N", [(1, 7168, 9216), (1, 4096, 4096), (3, 2304, 4096), (40, 2048, 1400), (61, 4096, 5120),
                                   (200, 2048, 1400), (129, 4096, 4096), (245, 8192, 1408), (100, 4096, 5120), (129, 4096, 1000)])
@pytest.mark.parametrize("last", [False, True])
def test_one_cta_of_a_cluster_gives_up(T, K, N, last):
    """The issuer of one CTA of each cluster stalls: the first, which has rows to join (with one row it is the
    only one), or the last, whose part the others wait for. The other CTAs send their parts, which have to end
    before any of them leaves: the call right behind takes their place and is right."""
    from mxfp4_routed_expert_03_gb300 import (MOE_ERR_DEVICE_TIMEOUT, MOE_INJECT_LINEAR_STALL_FIRST, MOE_INJECT_LINEAR_STALL_LAST,
                                              MOE_INJECT_NONE, check, moe_linear_set_fault_injection)
    s = Setup(T, K, N, seed=24)
    s.run()
    want, lost = s.out.clone(), torch.empty_like(s.out)
    mode = MOE_INJECT_LINEAR_STALL_LAST if last else MOE_INJECT_LINEAR_STALL_FIRST
    for _ in range(3):
        check(moe_linear_set_fault_injection(s.linear.h, mode, 2_000_000), "inject")
        check(s.linear.forward(T, s.rows, lost), "moe_linear_forward")
        check(moe_linear_set_fault_injection(s.linear.h, MOE_INJECT_NONE, 0), "inject off")
        s.out.fill_(7.0)
        s.run()
        assert s.linear.status() == MOE_ERR_DEVICE_TIMEOUT and s.linear.status() == 0
        assert torch.equal(s.out, want)


def test_transposed_weights_are_refused():
    from mxfp4_routed_expert_03_gb300.linear import Linear
    s = Setup(4, 256, 640, seed=25)
    for wq, ws in ((s.wq.t().contiguous(), s.ws), (s.wq, s.ws.t().contiguous()), (s.wq.view(1280, 128), s.ws)):
        with pytest.raises(ValueError):
            Linear(256, 640, wq, ws)
    Linear(256, 640, s.wq.flatten(), s.ws[:, None, :, None])
    s.run()
    s.verify()


@pytest.mark.parametrize("K,N", [(7168, 6912), (7168, 7040), (7168, 7168), (2048, 7168), (7168, 9216), (4096, 4096), (1040, 776)])
def test_a_row_has_the_same_bits_in_any_batch_of_up_to_16(K, N):
    from mxfp4_routed_expert_03_gb300 import check
    from mxfp4_routed_expert_03_gb300.linear import Fp8Rows
    s = Setup(16, K, N, seed=26, dtype=torch.float32)
    s.run()
    for T in (1, 2, 3, 5, 8, 15):
        out = torch.empty(T, N, device="cuda")
        check(s.linear.forward(T, Fp8Rows(s.xq[16 - T:], s.xs[16 - T:]), out), "moe_linear_forward")
        assert torch.equal(out, s.out[16 - T:])
