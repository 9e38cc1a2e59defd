"""Scored routing against a plain 64-bit reference.

Scores in fp32 are within 2^-21 of their value (an exponential of 1 ulp, a
sum rounded once, a divide), and the bias adds one rounding, 2^-24 of the sum:
where the 64-bit selection values that decide a token lie further apart than
GAP = 2^-20 of a token's largest score plus bias magnitude, the selection must
be the reference's; where they are equal bit for bit (equal logits and
biases), ties must go to the lower index. Weights: a few fp32 roundings, 2e-6
relative."""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu
GAP = 2.0 ** -20


def _layer(E, k):
    from mxfp4_routed_expert_03_gb300.layer import Layer, alloc_weights
    return Layer(256, 128, E, k, alloc_weights(E, 256, 128))


def _run(lg, k, bias=None, **kw):
    from mxfp4_routed_expert_03_gb300 import check
    from mxfp4_routed_expert_03_gb300.layer import Plan
    T, E = lg.shape
    layer, plan = _layer(E, k), Plan(T, E, k)
    dev = lambda a: None if a is None else torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()  # noqa: E731
    lg_d, b_d = dev(lg), dev(bias)
    check(layer.plan_scored(T, lg_d, None, plan, _route(**kw), b_d), "moe_plan_scored")
    st = layer.status()
    layer.close()
    return plan, st


def _route(sigmoid=False, groups=1, keep=None, top=1, renorm=True, scale=1.0):
    from mxfp4_routed_expert_03_gb300 import moe_route_desc
    return moe_route_desc(int(sigmoid), groups, keep or groups, top, int(renorm), scale)


def _reference(lg, k, bias=None, sigmoid=False, groups=1, keep=None, top=1, renorm=True, scale=1.0):
    """idx, weights, and per token whether every decision was further apart than GAP."""
    x = np.asarray(lg, np.float64)
    T, E = x.shape
    with np.errstate(over="ignore"):
        if sigmoid:
            p = 1 / (1 + np.exp(-x))
        else:
            e = np.exp(x - x.max(1, keepdims=True))
            p = e / e.sum(1, keepdims=True)
    s = p + (0 if bias is None else np.asarray(bias, np.float32).astype(np.float64))
    finite = 0.0 if bias is None else np.abs(bias[np.isfinite(bias)], dtype=np.float64).max(initial=0.0)
    gap = GAP * (p.max(1) + finite)
    sure = np.ones(T, bool)
    if groups > 1:
        by = np.sort(s.reshape(T, groups, -1), 2)[:, :, ::-1]
        gs = by[:, :, :top].sum(2)
        order = np.argsort(-gs, 1, kind="stable")
        if keep < groups:
            sg = np.take_along_axis(gs, order, 1)
            sure &= sg[:, keep - 1] - sg[:, keep] > 2 * gap
        open_ = np.zeros((T, groups), bool)
        np.put_along_axis(open_, order[:, :keep], True, 1)
        s = np.where(np.repeat(open_, E // groups, 1), s, -np.inf)
    order = np.argsort(-s, 1, kind="stable")
    ss = np.take_along_axis(s, order, 1)[:, :k + 1]
    with np.errstate(invalid="ignore"):
        sure &= (-np.diff(ss, axis=1) > gap[:, None]).all(1)
    idx = order[:, :k]
    w = np.take_along_axis(p, idx, 1)
    if renorm:
        w = w / w.sum(1, keepdims=True)
    return idx, w * scale, sure


def _check_plan(plan, E):
    idx = plan.topk_idx.cpu().numpy()
    T, k = idx.shape
    p = oracle.plan(idx, E)
    for name in ("counts", "offsets"):
        np.testing.assert_array_equal(getattr(plan, name).cpu().numpy(), p[name])
    for name in ("perm", "inv"):
        np.testing.assert_array_equal(getattr(plan, name).cpu().numpy()[:T * k], p[name])
    act = plan.active.cpu().numpy()
    np.testing.assert_array_equal(act[:1 + act[0]], p["active"])


def _compare(lg, k, bias=None, least=0.9, **kw):
    plan, st = _run(lg, k, bias, **kw)
    assert st == 0
    idx, w, sure = _reference(lg, k, bias, **kw)
    assert sure.mean() >= least
    np.testing.assert_array_equal(plan.topk_idx.cpu().numpy()[sure], idx[sure])
    np.testing.assert_allclose(plan.topk_w.cpu().numpy()[sure], w[sure], rtol=2e-6, atol=1e-30)
    _check_plan(plan, lg.shape[1])
    return plan


def _normal(T, E, seed):
    return np.random.default_rng(seed).standard_normal((T, E)).astype(np.float32)


@pytest.mark.parametrize("T", [1, 2, 16, 17, 64, 65, 300])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_896_experts(T, sigmoid):
    bias = 0.05 * _normal(1, 896, 7)[0] * (1.0 if sigmoid else 0.02)
    _compare(_normal(T, 896, T), 16, bias, sigmoid=sigmoid, scale=2.5)
    _compare(_normal(T, 896, T + 1), 16, None, sigmoid=sigmoid, renorm=False)


@pytest.mark.parametrize("E,k,groups,keep,top", [(256, 8, 8, 4, 2), (160, 6, 8, 3, 1), (64, 6, 4, 1, 2),
                                                 (1000, 12, 8, 7, 2), (32, 32, 32, 32, 1),
                                                 (1024, 32, 32, 5, 2), (7, 3, 7, 4, 1), (96, 1, 3, 1, 2)])
@pytest.mark.parametrize("T", [3, 70])
def test_groups(E, k, groups, keep, top, T):
    bias = 0.05 * _normal(1, E, 3)[0]
    for sigmoid in (True, False):
        _compare(_normal(T, E, E + T), k, bias if sigmoid else bias / 50, sigmoid=sigmoid, groups=groups,
                 keep=keep, top=top, least=0.5)


@pytest.mark.parametrize("T", [5, 90])
def test_ties_go_to_the_lower_index(T):
    E, k = 96, 9
    lg = np.zeros((T, E), np.float32)
    lg[:, 1::2] = -0.0
    lg[::3, ::7] = 1.0
    for sigmoid in (True, False):
        for groups, keep, top in ((1, 1, 1), (8, 3, 2), (8, 2, 1)):
            plan, st = _run(lg, k, None, sigmoid=sigmoid, groups=groups, keep=keep, top=top)
            assert st == 0
            idx, w, _ = _reference(lg + 0.0, k, None, sigmoid=sigmoid, groups=groups, keep=keep, top=top)
            np.testing.assert_array_equal(plan.topk_idx.cpu().numpy(), idx)
            np.testing.assert_allclose(plan.topk_w.cpu().numpy(), w, rtol=2e-6)


@pytest.mark.parametrize("T", [4, 80])
def test_infinite_and_extreme_logits(T):
    E, k = 40, 4
    lg = _normal(T, E, 1)
    lg[0, 5:8] = np.inf                      # softmax: the infinite ones share the weight
    lg[1] = -np.inf                          # all equal: uniform
    lg[2] = -np.inf
    lg[2, 30] = 2.0                          # one finite
    lg[3, 0], lg[3, 1] = 3e38, -3e38
    plan, st = _run(lg, k)
    assert st == 0
    idx, w = plan.topk_idx.cpu().numpy(), plan.topk_w.cpu().numpy()
    np.testing.assert_array_equal(idx[0], [5, 6, 7, 0])
    np.testing.assert_allclose(w[0], [1 / 3, 1 / 3, 1 / 3, 0], rtol=1e-6)
    np.testing.assert_array_equal(idx[1], [0, 1, 2, 3])
    np.testing.assert_allclose(w[1], 0.25, rtol=1e-6)
    np.testing.assert_array_equal(idx[2], [30, 0, 1, 2])
    np.testing.assert_array_equal(w[2], [1, 0, 0, 0])
    assert idx[3, 0] == 0 and w[3, 0] == 1
    plan, st = _run(lg, k, sigmoid=True)
    idx, w = plan.topk_idx.cpu().numpy(), plan.topk_w.cpu().numpy()
    assert st == 0 and np.isfinite(w).all()
    np.testing.assert_array_equal(idx[0][:3], [5, 6, 7])
    np.testing.assert_array_equal(w[1], 0)   # all scores 0: their sum is 0
    _check_plan(plan, E)


@pytest.mark.parametrize("T", [4, 80])
def test_minus_infinite_bias_takes_experts_out(T):
    E, k = 64, 8
    lg = _normal(T, E, 2)
    bias = np.zeros(E, np.float32)
    bias[::2] = -np.inf
    for kw in (dict(sigmoid=True), dict(), dict(sigmoid=True, groups=4, keep=2, top=2)):
        plan = _compare(lg, k, bias, least=0.5, **kw)
        assert (plan.topk_idx.cpu().numpy() % 2 == 1).all()
    bias[:] = -np.inf                        # nothing left: still k distinct experts
    plan, st = _run(lg, k, bias, sigmoid=True)
    np.testing.assert_array_equal(plan.topk_idx.cpu().numpy(), np.tile(np.arange(k), (T, 1)))
    assert st == 0


@pytest.mark.parametrize("T", [4, 200])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_nan_logit_or_bias_is_reported(T, sigmoid):
    from mxfp4_routed_expert_03_gb300 import MOE_ERR_NAN_LOGIT
    lg = _normal(T, 64, 4)
    lg[1, 3] = np.nan
    plan, st = _run(lg, 4, sigmoid=sigmoid)
    assert st == MOE_ERR_NAN_LOGIT
    lg[1, 3] = -np.inf
    idx, w, _ = _reference(lg, 4, sigmoid=sigmoid)
    np.testing.assert_array_equal(plan.topk_idx.cpu().numpy(), idx)
    _check_plan(plan, 64)
    for bad in (np.nan, np.inf):
        bias = np.zeros(64, np.float32)
        bias[9] = bad
        plan, st = _run(_normal(T, 64, 5), 4, bias, sigmoid=sigmoid)
        assert st == MOE_ERR_NAN_LOGIT and 9 not in plan.topk_idx.cpu().numpy()


def test_scores_do_not_depend_on_the_order_of_the_sum():
    """The softmax's denominator is the exact sum of the fp32 exponentials,
    rounded once: a permutation of the experts gives the same weights bit for bit."""
    E, k = 896, 16
    lg = _normal(70, E, 6)
    perm = np.random.default_rng(1).permutation(E)
    a, _ = _run(lg, k, renorm=False)
    b, _ = _run(lg[:, perm], k, renorm=False)
    np.testing.assert_array_equal(a.topk_w.cpu().numpy(), b.topk_w.cpu().numpy())
    np.testing.assert_array_equal(a.topk_idx.cpu().numpy(), perm[b.topk_idx.cpu().numpy()])


def test_router_mode_and_the_experts_products():
    """In router mode the logits come from x . W_r; the plan drives moe_forward."""
    import synth
    from harness import assert_close, bf16_dev_to_f64, host_layer_weights, to_dev_bf16
    from mxfp4_routed_expert_03_gb300 import MOE_ROUTER_XWR, check
    from mxfp4_routed_expert_03_gb300.layer import Layer, Plan
    w = synth.WORKLOADS["tiny"]
    wr = torch.from_numpy(0.1 * _normal(w.E, w.D, 8)).cuda()
    layer = Layer(w.D, w.F, w.E, w.k, host_layer_weights(w), router_mode=MOE_ROUTER_XWR, w_router=wr)
    x_np = synth.make_x(w)
    x = to_dev_bf16(x_np)
    plan = Plan(w.T, w.E, w.k)
    check(layer.plan_scored(w.T, None, x, plan, _route(sigmoid=True, scale=2.0)), "plan")
    lg = torch.empty(w.T, w.E, device="cuda")
    check(layer.router_logits(w.T, x, lg), "router")
    out, ref = (torch.empty((w.T, w.D), dtype=torch.int16, device="cuda") for _ in range(2))
    check(layer.forward(w.T, x, plan, out), "forward")
    assert layer.status() == 0
    idx, wt, sure = _reference(lg.cpu().numpy(), w.k, sigmoid=True, scale=2.0)
    assert sure.all()
    np.testing.assert_array_equal(plan.topk_idx.cpu().numpy(), idx)
    # the same experts with the softmax's weights, through the plan that was there
    host = lg.cpu().numpy()
    same = Layer(w.D, w.F, w.E, w.k, layer.weights)
    plan2 = Plan(w.T, w.E, w.k)
    forced = np.full((w.T, w.E), -1e30, np.float32)
    np.put_along_axis(forced, idx, np.log(wt / 2.0).astype(np.float32), 1)
    check(same.plan(w.T, torch.from_numpy(forced).cuda(), None, plan2), "plan")
    check(same.forward(w.T, x, plan2, ref), "forward")
    assert same.status() == 0 and np.isfinite(host).all()
    assert_close(bf16_dev_to_f64(out), 2.0 * bf16_dev_to_f64(ref))


def test_refusals():
    from mxfp4_routed_expert_03_gb300 import MOE_ERR_INVALID_ARG, MOE_ERR_WORKSPACE, MOE_OK, moe_plan_scored
    from mxfp4_routed_expert_03_gb300.layer import Plan
    layer, plan = _layer(64, 6), Plan(4, 64, 6)
    lg = torch.zeros(4, 64, device="cuda")
    run = lambda r: layer.plan_scored(4, lg, None, plan, r)  # noqa: E731
    assert run(_route()) == MOE_OK
    bad = [_route(groups=5), _route(groups=0), _route(groups=64, keep=64), _route(groups=8, keep=9),
           _route(groups=16, keep=1), _route(top=3), _route(top=0), _route(scale=math.nan), _route(scale=math.inf)]
    r = _route()
    r.score = 2
    q = _route()
    q.renormalise = 2
    for d in bad + [r, q]:
        assert run(d) == MOE_ERR_INVALID_ARG
    assert moe_plan_scored(layer.h, 4, None, None, _route(), None, plan.buf, None, 0) == MOE_ERR_INVALID_ARG
    assert moe_plan_scored(layer.h, 100, lg, None, _route(), None, plan.buf, None, 0) == MOE_ERR_WORKSPACE
    assert moe_plan_scored(layer.h, 0, None, None, _route(), None, plan.buf, None, 0) == MOE_OK
    assert layer.status() == 0
    layer.close()
