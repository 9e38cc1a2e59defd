"""Workspaces of the Python classes under captured graphs and on several streams."""
import pytest
import torch

from test_gpu_attention import DEV, Setup, _close

pytestmark = pytest.mark.gpu


def _check(s):
    o, l_, mag, big = s.want()
    _close(s.out, s.lse, o.view(s.T, -1), l_, mag.view(s.T, -1), big)


def test_a_captured_step_keeps_its_workspace():
    from mxfp4_routed_expert_03_gb300 import check
    from mxfp4_routed_expert_03_gb300.attention import Batch
    s = Setup(8, 1, 128, 64, [1], [5000], seed=80)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    check(s.attn.forward(s.batch, s.q, s.out, s.lse, st), "forward")
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        check(s.attn.forward(s.batch, s.q, s.out, s.lse, torch.cuda.current_stream()), "forward")
    need = s.attn.workspace_bytes(s.batch)
    # a prompt on the same stream needs more; what it frees is taken by others
    rows = 40
    cu = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    large = Batch(1, rows, rows, 5000, cu, s.kv_t, s.table, s.scale)
    assert s.attn.workspace_bytes(large) > need
    q = torch.randn(rows, 8 * 128, device=DEV).bfloat16()
    out = torch.empty_like(q)
    st.wait_stream(torch.cuda.current_stream())
    check(s.attn.forward(large, q, out, None, st), "forward")
    with torch.cuda.stream(st):
        others = [torch.full((need,), 42, dtype=torch.uint8, device=DEV) for _ in range(8)]
    st.synchronize()
    s.out.fill_(7.0)
    s.lse.fill_(7.0)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert s.attn.status() == 0
    assert all(bool((t == 42).all()) for t in others)
    _check(s)


def test_calls_on_two_streams_at_a_time():
    from mxfp4_routed_expert_03_gb300 import check
    s = Setup(8, 1, 128, 64, [1], [20000], seed=81)
    check(s.attn.forward(s.batch, s.q, s.out, s.lse), "forward")
    _check(s)
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [torch.empty_like(s.out) for _ in streams]
    own = torch.empty(s.attn.workspace_bytes(s.batch), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    for _ in range(50):
        for i, (st, out) in enumerate(zip(streams, outs)):
            check(s.attn.forward(s.batch, s.q, out, None, st, own if i == 2 else None), "forward")
    torch.cuda.synchronize()
    assert s.attn.status() == 0
    assert all(torch.equal(out, s.out) for out in outs)


def test_own_workspace_that_is_too_small_is_refused():
    from mxfp4_routed_expert_03_gb300 import MOE_ERR_WORKSPACE
    s = Setup(8, 1, 128, 64, [1], [2000], seed=82)
    small = torch.empty(s.attn.workspace_bytes(s.batch) - 256, dtype=torch.uint8, device=DEV)
    assert s.attn.forward(s.batch, s.q, s.out, s.lse, None, small) == MOE_ERR_WORKSPACE


def test_scored_plan_in_a_graph_and_on_its_own_stream():
    from mxfp4_routed_expert_03_gb300 import MOE_SCORE_SIGMOID, check, moe_route_desc
    from mxfp4_routed_expert_03_gb300.layer import Layer, Plan, alloc_weights
    T, E, k = 3000, 128, 8
    layer = Layer(256, 128, E, k, alloc_weights(E, 256, 128))
    route = moe_route_desc(MOE_SCORE_SIGMOID, 1, 1, 1, 1, 1.0)
    lg = torch.randn(4 * T, E, device=DEV)
    want, plan, large = Plan(T, E, k), Plan(T, E, k), Plan(4 * T, E, k)
    check(layer.plan_scored(T, lg, None, want, route), "plan")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    check(layer.plan_scored(T, lg, None, plan, route, None, st), "plan")
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        check(layer.plan_scored(T, lg, None, plan, route, None, torch.cuda.current_stream()), "plan")
    check(layer.plan_scored(4 * T, lg, None, large, route, None, st), "plan")
    n = layer.workspace(T, 0)[1]
    with torch.cuda.stream(st):
        others = [torch.full((n,), 42, dtype=torch.uint8, device=DEV) for _ in range(8)]
    for t in (plan.topk_idx, plan.counts, plan.offsets, plan.perm, plan.inv):
        t.fill_(-1)
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert layer.status() == 0
    assert all(bool((t == 42).all()) for t in others)
    for name in ("topk_idx", "topk_w", "counts", "offsets", "perm", "inv"):
        assert torch.equal(getattr(plan, name), getattr(want, name)), name
