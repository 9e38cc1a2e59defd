"""moe_add_norm: residual addition, norm and rows in 8 bits, against 64 bits."""
import pytest
import torch

from linear_ref import U, blocks, decode, distance, grid

pytestmark = pytest.mark.gpu

# fp32 error of y, relative: at most 64 squares a thread, 5 + 16 sums across threads (all of one
# sign), halved by the root, then mean, eps, the root's 2 ulp and two products: under 60 roundings
Y = 60 * U
BF16 = 2.0 ** -8


def make(T, d, seed, residual=True, weight=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    scale = torch.exp(torch.randn(d, device="cuda", generator=g))
    rand = lambda: (torch.randn(T, d, device="cuda", generator=g) * scale).bfloat16()  # noqa: E731
    return rand(), rand() if residual else None, (1 + 0.3 * torch.randn(d, device="cuda", generator=g)).bfloat16() if weight else None


def reference(x, r, w, eps):
    """h exactly, y in 64 bits."""
    h = x if r is None else (x.float() + r.float()).bfloat16()
    y = h.double()
    if w is not None:
        y = y / torch.sqrt(y.square().mean(1, keepdim=True) + eps) * w.double()
    return h, y


def check_rows8(q, s, y):
    """Codes and scales of y [T][d] (fp64, finite)."""
    top = blocks(y).abs().amax(2)
    want = (top / 448).clamp(min=2.0 ** -126)
    kb = want.shape[1]
    assert bool(((s[:, :kb].double() - want).abs() <= (Y + 2 * U) * want).all())
    # the code is as near to y / s as any (up to the fp32 error of y / s)
    u = (blocks(y) / s[:, :kb].double()[:, :, None]).flatten(1)[:, :y.shape[1]]
    off = (q.float().double() - u).abs()
    assert bool((off <= distance(u.clamp(-448, 448)) + (u.abs() - 448).clamp(min=0) + (2 * Y + 4 * U) * u.abs()).all())


def run(x, r, w, total=True, y=True, y8=True, eps=1e-6, stream=None):
    from mxfp4_routed_expert_03_gb300 import check
    from mxfp4_routed_expert_03_gb300.linear import Fp8Rows, Norm
    T, d = x.shape
    norm = Norm(d, eps, w)
    out = [torch.full_like(x, 7.0) if on else None for on in (total and r is not None, y)]
    rows = Fp8Rows.empty(T, d) if y8 else None
    check(norm.forward(T, x, r, *out, rows, stream), "moe_add_norm")
    torch.cuda.synchronize()
    return out[0], out[1], rows


def verify(x, r, w, got, eps=1e-6):
    total, y, rows = got
    h, ref = reference(x, r, w, eps)
    if total is not None:
        assert torch.equal(total, h)
    if y is not None:
        assert bool(((y.double() - ref).abs() <= (BF16 + 2 * Y) * ref.abs() + 1e-38).all())
    if rows is not None:
        check_rows8(rows.q, rows.s, ref)


@pytest.mark.parametrize("d", [16, 32, 128, 144, 1008, 1536, 2048, 2064, 4096, 5120, 7168, 8192, 16384])
@pytest.mark.parametrize("T", [1, 2, 3, 17, 200])
def test_sizes(T, d):
    x, r, w = make(T, d, seed=T + d)
    verify(x, r, w, run(x, r, w, y8=d % 16 == 0))


@pytest.mark.parametrize("d", [8, 24, 1000, 3000, 16376])
def test_odd_widths_in_bf16(d):
    x, r, w = make(9, d, seed=d)
    verify(x, r, w, run(x, r, w, y8=False))


@pytest.mark.parametrize("T,d", [(5000, 256), (3001, 1536), (1400, 7168), (40000, 64)])
def test_many_rows(T, d):
    x, r, w = make(T, d, seed=1)
    verify(x, r, w, run(x, r, w))


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("total,y,y8", [(True, False, False), (False, True, False), (False, False, True), (True, True, True)])
def test_parts(residual, weight, total, y, y8):
    x, r, w = make(37, 2048, seed=2, residual=residual, weight=weight)
    verify(x, r, w, run(x, r, w, total, y, y8))


@pytest.mark.parametrize("eps", [0.0, 1e-5, 3.0])
def test_eps(eps):
    x, r, w = make(5, 1024, seed=3)
    verify(x, r, w, run(x, r, w, eps=eps), eps)


@pytest.mark.parametrize("d", [256, 4096])
def test_zero_rows_and_small_values(d):
    x, r, w = make(6, d, seed=4, residual=False)
    x[1] = 0
    x[2] *= 2.0 ** -60
    x[3] *= 2.0 ** -120
    x[4, 128:256] = 0
    x[5, :128] = 2.0 ** -130
    verify(x, r, None, run(x, r, None))  # as they are: scales of 2^-126 at least
    verify(x, r, w, run(x, r, w))        # eps decides
    _, _, rows = run(x, r, None)
    assert bool((decode(rows.q, rows.s)[1] == 0).all()) and float(rows.s[1, 0]) == 2.0 ** -126


@pytest.mark.parametrize("T", [3, 2000])
def test_a_sum_beyond_its_range_gives_zeros(T):
    x, r, w = make(T, 1024, seed=12)
    x[1] = 1e30
    total, y, rows = run(x, r, w)
    assert torch.equal(total[1], x[1]) and bool((y[1] == 0).all()) and bool((decode(rows.q, rows.s)[1] == 0).all())
    others = torch.arange(T, device="cuda") != 1
    verify(x[others], r[others], w, (total[others], y[others], type(rows)(rows.q.view(torch.uint8)[others].view(rows.q.dtype), rows.s[others])))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("d", [384, 7168])
def test_not_finite(bad, d):
    x, r, w = make(4, d, seed=5, residual=False)
    x[1, 130] = bad
    _, y, rows = run(x, None, None)
    assert bool(rows.s[1, 1].isnan()) and bool(rows.s[:, 0].isfinite().all()) and bool(rows.s[1, 2:].isfinite().all())
    keep = torch.ones(4, d, dtype=torch.bool, device="cuda")
    keep[1, 128:256] = False
    assert bool(decode(rows.q, rows.s)[~keep].isnan().all()) and bool(decode(rows.q, rows.s)[keep].isfinite().all())
    assert torch.equal(y[keep], x[keep])
    _, y, rows = run(x, None, w)  # a norm spreads it over its row and no other
    others = [0, 2, 3]
    verify(x[others], None, w, (None, y[others], type(rows)(rows.q.view(torch.uint8)[others].view(rows.q.dtype), rows.s[others])))
    assert bool(y[1, 130].isnan()) and bool(rows.s[1, 1].isnan())
    assert bool((y[1].isnan() | (y[1] == 0)).all())


@pytest.mark.parametrize("T", [1, 50])
def test_strided_rows_in_place_and_untouched_memory(T):
    from mxfp4_routed_expert_03_gb300 import check
    from mxfp4_routed_expert_03_gb300.linear import Fp8Rows, Norm
    d = 400
    x, r, w = make(T, d, seed=6)
    h, ref = reference(x, r, w, 1e-6)
    wide = torch.full((T + 2, 1024), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:T, 8:408], wide[:T, 512:912] = x, r
    codes = torch.full((T + 2, 448), 9, dtype=torch.uint8, device="cuda")
    scales = torch.full((T + 2, 7), 9.0, device="cuda")
    rows = Fp8Rows(codes.view(torch.float8_e4m3fn)[:, 32:432], scales[:, 1:5])
    norm = Norm(d, 1e-6, w)
    # y over x, total over the residual
    check(norm.forward(T, wide[:, 8:408], wide[:, 512:912], wide[:, 512:912], wide[:, 8:408], rows), "moe_add_norm")
    verify(x, r, w, (wide[:T, 512:912].contiguous(), wide[:T, 8:408].contiguous(), Fp8Rows(rows.q[:T].contiguous(), rows.s[:T].contiguous())))
    wide[:T, 8:408] = 7.0
    wide[:T, 512:912] = 7.0
    codes[:T, 32:432] = 9
    scales[:T, 1:5] = 9.0
    assert bool((wide == 7.0).all()) and bool((codes == 9).all()) and bool((scales == 9.0).all())


def test_many_rows_in_place_on_a_stream_and_in_a_graph():
    """Rows on their way while others are written: outputs over the inputs of the same rows."""
    from mxfp4_routed_expert_03_gb300 import check
    from mxfp4_routed_expert_03_gb300.linear import Fp8Rows, Norm
    T, d = 3001, 1008
    x, r, w = make(T, d, seed=10)
    norm, rows = Norm(d, 1e-6, w), Fp8Rows.empty(T, d)
    wide = torch.full((T + 1, 2 * d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    a, b = wide[:, :d], wide[:, d + 8:]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        check(norm.forward(T, a, b, b, a, rows, torch.cuda.current_stream()), "moe_add_norm")
    for _ in range(3):
        a[:T], b[:T] = x, r
        graph.replay()
        torch.cuda.synchronize()
        verify(x, r, w, (b[:T].contiguous(), a[:T].contiguous(), rows))
    assert bool((wide[T] == 7.0).all()) and bool((wide[:, d:d + 8] == 7.0).all())


def test_as_many_rows_as_the_count_holds():
    """2^31 - 1 rows of 8, in place (34 GB)."""
    from mxfp4_routed_expert_03_gb300 import check
    from mxfp4_routed_expert_03_gb300.linear import Norm
    T, d = 2 ** 31 - 1, 8
    if torch.cuda.mem_get_info()[0] < 40e9:
        pytest.skip("needs 40 GB")
    x = torch.zeros(T, d, dtype=torch.bfloat16, device="cuda")
    some = torch.tensor([0, 2 ** 28 + 1, 2 ** 30, T - 9, T - 1], device="cuda")
    few, _, w = make(5, d, seed=13, residual=False)
    x[some] = few
    check(Norm(d, 1e-6, w).forward(T, x, y=x), "moe_add_norm")
    got = x[some]
    x[some] = 0
    assert int(torch.count_nonzero(x[:1000])) == 0 and int(torch.count_nonzero(x[-1000:])) == 0
    verify(few, None, w, (None, got, None))
    del x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_many_rows_not_finite(bad):
    T, d = 2000, 1024
    x, r, w = make(T, d, seed=11)
    x[77, 500], r[1999, 3] = bad, bad
    total, y, rows = run(x, r, w)
    others = torch.ones(T, dtype=torch.bool, device="cuda")
    others[[77, 1999]] = False
    verify(x[others], r[others], w, (total[others], y[others], type(rows)(rows.q.view(torch.uint8)[others].view(rows.q.dtype), rows.s[others])))
    assert bool(rows.s[77, 3].isnan()) and bool(rows.s[1999, 0].isnan())


def test_streams_and_graphs():
    from mxfp4_routed_expert_03_gb300 import check
    from mxfp4_routed_expert_03_gb300.linear import Fp8Rows, Norm
    x, r, w = make(33, 7168, seed=7)
    norm, rows, y, total = Norm(7168, 1e-6, w), Fp8Rows.empty(33, 7168), torch.empty_like(x), torch.empty_like(x)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    check(norm.forward(33, x, r, total, y, rows, st), "moe_add_norm")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        check(norm.forward(33, x, r, total, y, rows, torch.cuda.current_stream()), "moe_add_norm")
    x2, r2, _ = make(33, 7168, seed=8)
    x.copy_(x2)
    r.copy_(r2)
    graph.replay()
    torch.cuda.synchronize()
    verify(x, r, w, (total, y, rows))


def test_no_rows_and_refusals():
    from mxfp4_routed_expert_03_gb300 import MOE_ERR_INVALID_ARG
    from mxfp4_routed_expert_03_gb300.linear import Fp8Rows, Norm
    x, r, w = make(4, 256, seed=9)
    norm, y, rows = Norm(256, 1e-6, w), torch.full_like(x, 7.0), Fp8Rows.empty(4, 256)
    assert norm.forward(0, x, r, None, y, rows) == 0 and bool((y == 7.0).all())
    assert norm.forward(4, x, r) == 0  # nothing asked for
    assert norm.forward(-1, x, r, None, y) == MOE_ERR_INVALID_ARG and norm.forward(4, None, r, None, y) == MOE_ERR_INVALID_ARG
    assert norm.forward(4, x, None, y) == MOE_ERR_INVALID_ARG  # a total without a residual
    for bad in (x[:3], x[:, :128], x.half(), x.float(), x.cpu(), x.t()):
        with pytest.raises(ValueError):
            norm.forward(4, bad, None, None, y)
        with pytest.raises(ValueError):
            norm.forward(4, x, bad, None, y)
        with pytest.raises(ValueError):
            norm.forward(4, x, r, None, bad)
    with pytest.raises(ValueError):
        norm.forward(4, x, r, None, y, Fp8Rows.empty(3, 256))
    with pytest.raises(ValueError):
        norm.forward(4, x, r, None, y, Fp8Rows.empty(4, 128))
    for bad in (w[:100], w.float(), w.cpu(), torch.stack([w, w], 1)[:, 0]):
        with pytest.raises(ValueError):
            Norm(256, 1e-6, bad)
    wide = torch.empty(4, 300, dtype=torch.bfloat16, device="cuda")
    assert norm.forward(4, wide[:, 1:257], None, None, y) == MOE_ERR_INVALID_ARG
    assert norm.forward(4, wide[:, :256], None, None, y) == MOE_ERR_INVALID_ARG  # row stride 300
    odd = Norm(248, 1e-6)
    assert odd.forward(4, x, None, None, None, Fp8Rows.empty(4, 256)) == MOE_ERR_INVALID_ARG  # 8 bits: multiples of 16


@pytest.mark.parametrize("T,d", [(1, 7168), (40, 4096), (777, 4096), (9, 144), (3001, 1536), (4099, 8192)])
@pytest.mark.parametrize("residual", [True, False])
def test_half_way_codes_go_to_the_even_one(T, d, residual):
    """Code for code: with a norm a block's quotients y / s are h weight / (largest |h weight| / 448), in which the row's
    factor does not occur. In 64 bits a quotient that is half-way between two codes is exactly that, and any
    other is at least 2^-21 of its size away from it (16-bit numerators and denominators), so that rounding it
    to fp32 first changes no code. A code or so in 8000 is half-way."""
    x, r, w = make(T, d, seed=14, residual=residual)
    _, _, rows = run(x, r, w, y=False)
    h, _ = reference(x, r, None, 0.0)
    p = blocks(h.double() * w.double())
    u = (448 * p / p.abs().amax(2, keepdim=True)).flatten(1)[:, :d]
    if T * d > 2 ** 20:
        g = grid("cuda")
        at = torch.searchsorted(g, u.contiguous()).clamp(1, g.numel() - 1)
        assert int((u * 2 == g[at - 1] + g[at]).sum()) > 20
    assert torch.equal(rows.q.float(), u.float().to(torch.float8_e4m3fn).float())


@pytest.mark.parametrize("few", [False, True])
def test_codes_without_a_norm_are_those_of_a_division(few):
    """Bit for bit, signs of zeros too: s = max (1 / 448) and h / s in fp32, then the nearest code. Every significand of
    a block's largest element with every one of the others, at several sizes."""
    m = torch.arange(128, 256, dtype=torch.float64)[:, None, None]  # a row for each
    e = torch.tensor([0, -1, -2, -3, -5, -8, -12, -17]).double()     # two blocks of the row for each
    h = torch.arange(128, 256, dtype=torch.float64) * torch.exp2(e)[None, :, None] * (1 - 2.0 * (torch.arange(128) % 3 == 1))
    h = torch.where(h.abs() > m, h / 2, h)
    ends = torch.cat([m, -m, 0 * m, -0.0 * m], 2).expand(128, 8, 4)
    x = torch.stack([torch.cat([ends, h[..., :124]], 2), torch.cat([ends, h[..., 4:]], 2)], 2).reshape(128, 2048)
    x = torch.cat([x * 2.0 ** k for k in ((0,) if few else range(-50, 60, 2))]).bfloat16()
    b = x.float().unflatten(1, (16, 128))
    want_s = b.abs().amax(2) * torch.tensor(1 / 448)  # (on the CPU)
    want = (b / want_s[..., None]).flatten(1).clamp(-448, 448).to(torch.float8_e4m3fn)
    _, _, got = run(x.cuda(), None, None, y=False)
    assert torch.equal(got.s.cpu(), want_s)
    assert torch.equal(got.q.cpu().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("d", [8, 24, 136, 248, 1000, 4104, 16376])
@pytest.mark.parametrize("T,residual,weight", [(1, True, True), (9, False, False), (700, True, True), (1500, False, True)])
def test_packed_code_rows_of_odd_widths(d, T, residual, weight):
    """Widths that are multiples of 8 alone: code rows one behind the other; nothing around them is written."""
    from mxfp4_routed_expert_03_gb300 import MOE_ERR_INVALID_ARG, check
    from mxfp4_routed_expert_03_gb300.linear import Fp8Rows, Norm
    x, r, w = make(T, d, seed=d, residual=residual, weight=weight)
    norm, y, rows = Norm(d, 1e-6, w), torch.empty_like(x), Fp8Rows.empty(T + 1, d)
    rows.q.view(torch.uint8).fill_(9)
    rows.s.fill_(9.0)
    check(norm.forward(T, x, r, None, y, rows), "moe_add_norm")
    assert bool((rows.q.view(torch.uint8)[T] == 9).all()) and bool((rows.s[T] == 9.0).all())
    verify(x, r, w, (None, y, Fp8Rows(rows.q[:T], rows.s[:T])))
    wide = Fp8Rows.empty(T, d + 8)  # (rows that the product would take for whole ones of 16)
    assert norm.forward(T, x, r, None, y, wide) == MOE_ERR_INVALID_ARG
