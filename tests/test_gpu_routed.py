"""The layer on a given routing (moe_fwd_routed, moe_bwd_routed), alone and
together with moe_route and moe_route_bwd.

The experts' kernels are moe_fwd's and moe_bwd's: with the routing that the
built-in router made, the results are the same bits.  Against the plain fp64
layer the tolerances are the parity tests' (rel-L2 1e-2: h, the activation
gradients and the outputs are rounded to bf16, per-route rows to fp16)."""
import numpy as np
import pytest
import torch

import moe_inputs as mi
import routing_grouped_expert_gemm_gb300 as rg

pytestmark = pytest.mark.gpu


def layer_of(name="tiny", **kw):
    import gpu_util
    inp = mi.make_inputs(name)
    return inp, gpu_util.Layer(inp, **{**dict(minibatch=512, ring_slots=2, gather_ctas=2), **kw}), gpu_util.to_dev_bf16(inp.x)


def fwd_routed(layer, x, idx, w, **kw):
    out = torch.full((x.shape[0], layer.shape.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    layer.ws.fill_(0xFF)
    weights = {k: v for k, v in layer.w.items() if k not in ("W_router", "b_router")}
    rg.moe_fwd_routed(layer.plan, x.shape[0], x, weights, idx, w, out, layer.ws, layer.ws_bytes, **kw)
    return out, rg.moe_get_status(layer.plan, layer.ws)


def plain_layer(x, w, idx, wt):
    """fp64: shared expert + sum over the slots; idx < 0 is an empty slot."""
    f = lambda u, g, d, v: (torch.nn.functional.silu(v @ g.T) * (v @ u.T)) @ d.T
    out = f(w["Ws_up"], w["Ws_gate"], w["Ws_down"], x) if "Ws_up" in w else torch.zeros_like(x)
    for e in range(w["W_up"].shape[0]):
        t, s = torch.nonzero(idx == e, as_tuple=True)
        if len(t):
            out = out.index_add(0, t, wt[t, s, None] * f(w["W_up"][e], w["W_gate"][e], w["W_down"][e], x[t]))
    return out


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


@pytest.mark.parametrize("kw", [dict(), dict(mma_pair=1, dispatch="spread"), dict(dispatch="direct", gather_ctas=0)])
@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
def test_the_built_in_routers_routing_gives_the_same_bits(precision, kw):
    inp, layer, x = layer_of(mi.custom_shape(300, 256, 128, 16, 4, 128, precision=precision), **kw)
    res = layer.run(x)
    assert res["status"] == 0
    cnt = torch.empty_like(res["expert_counts"])
    sched = torch.empty_like(res["sched"])
    out, status = fwd_routed(layer, x, res["topk_idx"], res["topk_w"], expert_counts=cnt, sched=sched)
    assert status == rg.MOE_STATUS_OK
    assert torch.equal(out, res["out"]) and torch.equal(cnt, res["expert_counts"]) and torch.equal(sched, res["sched"])


def some_routing(T, E, k, seed=0, empty=0.3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    idx = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32)
    idx[torch.rand(T, k, generator=g, device="cuda") < empty] = -1
    idx[::11] = -1
    return idx, torch.rand(T, k, generator=g, device="cuda") + 0.1


@pytest.mark.parametrize("T", [1, 127, 256])
@pytest.mark.parametrize("pair", [0, 1])
def test_any_routing_with_empty_slots(T, pair):
    inp, layer, x = layer_of(mma_pair=pair)
    s, x = inp.shape, x[:T]
    idx, w = some_routing(T, s.E, s.k)
    out, status = fwd_routed(layer, x, idx, w)
    assert status == rg.MOE_STATUS_OK
    ref = plain_layer(x.double(), {k: v.double() for k, v in layer.w.items() if v is not None}, idx.long(), w.double())
    assert rel(out, ref) <= 1e-2


def test_invalid_slots_are_reported_and_harmless():
    inp, layer, x = layer_of()
    s = inp.shape
    idx, w = some_routing(inp.T, s.E, s.k, empty=0.0)
    ref, status = fwd_routed(layer, x, idx, w)
    assert status == rg.MOE_STATUS_OK
    for bad in (s.E, -2, 1 << 30):
        i2 = idx.clone()
        i2[5, 1] = bad
        out, status = fwd_routed(layer, x, i2, w)
        assert status == rg.MOE_STATUS_SCHEDULE_INVALID
        assert torch.equal(out[:5], ref[:5]) and torch.equal(out[6:], ref[6:])
    i2 = idx.clone()
    i2[7, 2] = i2[7, 0]
    out, status = fwd_routed(layer, x, i2, w)
    assert status == rg.MOE_STATUS_SCHEDULE_INVALID
    i2[7, 2] = -1
    ref2, status = fwd_routed(layer, x, i2, w)
    assert status == rg.MOE_STATUS_OK and torch.equal(out, ref2)


def grads_of(layer, T):
    s = layer.shape
    bf = lambda *d: torch.full(d, float("nan"), dtype=torch.bfloat16, device="cuda")
    return {"dx": bf(T, s.D), "dW_up": bf(s.E, s.I, s.D), "dW_gate": bf(s.E, s.I, s.D), "dW_down": bf(s.E, s.D, s.I),
            "dWs_up": bf(s.I_s, s.D), "dWs_gate": bf(s.I_s, s.D), "dWs_down": bf(s.D, s.I_s)}


def bwd_layer(pair):
    """A layer whose sizes the backward supports (multiples of 256)."""
    import gpu_util
    inp = mi.make_inputs(mi.custom_shape(300, 256, 256, 12, 3, 256))
    return inp, gpu_util.Layer(inp, minibatch=512, ring_slots=2, gather_ctas=2, mma_pair=pair), gpu_util.to_dev_bf16(inp.x)


@pytest.mark.parametrize("pair", [0, 1])
def test_gradients_match_fp64_and_moe_bwd(pair):
    inp, layer, x = bwd_layer(pair)
    s, T = inp.shape, inp.T
    g = torch.Generator(device="cuda").manual_seed(1)
    dO = torch.randn(T, s.D, generator=g, device="cuda").bfloat16()
    idx, w = some_routing(T, s.E, s.k, seed=3)
    out, status = fwd_routed(layer, x, idx, w)
    bws = torch.full((rg.moe_bwd_workspace_bytes(layer.plan, T),), 0xFF, dtype=torch.uint8, device="cuda")
    gr, dw = grads_of(layer, T), torch.full((T, s.k), float("nan"), device="cuda")
    weights = {k: v for k, v in layer.w.items() if k not in ("W_router", "b_router")}
    rg.moe_bwd_routed(layer.plan, T, x, weights, dO, layer.ws, gr, dw, bws)
    assert rg.moe_get_status(layer.plan, bws) == rg.MOE_STATUS_OK
    p = {k: v.double().requires_grad_(True) for k, v in layer.w.items() if v is not None and k not in ("W_router", "b_router")}
    xd, wd = x.double().requires_grad_(True), w.double().requires_grad_(True)
    plain_layer(xd, p, idx.long(), wd).backward(dO.double())
    assert rel(gr["dx"], xd.grad) <= 1e-2
    ref = torch.where(idx >= 0, wd.grad, torch.zeros_like(wd.grad))
    assert rel(dw, ref) <= 1e-2 and bool((dw[idx < 0] == 0).all())
    for k in ("W_up", "W_gate", "W_down", "Ws_up", "Ws_gate", "Ws_down"):
        assert rel(gr["d" + k], p[k].grad) <= 1e-2, k
    # the built-in router's routing: the experts' gradients are moe_bwd's, bit for bit
    res = layer.run(x)
    g0 = grads_of(layer, T)
    g0["dW_router"] = torch.empty(s.E, s.D, device="cuda")
    rg.moe_bwd(layer.plan, T, x, layer.w, dO, layer.ws, g0, bws)
    fwd_routed(layer, x, res["topk_idx"], res["topk_w"])
    rg.moe_bwd_routed(layer.plan, T, x, weights, dO, layer.ws, gr, dw, bws)
    for k in gr:
        if k != "dx":
            assert torch.equal(gr[k], g0[k]), k


def test_router_experts_and_back_give_moe_bwds_router_gradient():
    """logits -> moe_route -> moe_fwd_routed -> moe_bwd_routed -> moe_route_bwd
    -> dW_router, dx: the built-in router's, which does the same in one call."""
    inp, layer, x = bwd_layer(0)
    s, T = inp.shape, inp.T
    Wr = layer.w["W_router"]
    b = layer.w["b_router"]
    logits = x.float() @ Wr.float().T + (b if b is not None else 0.0)
    plan = rg.moe_route_plan_create(s.E, s.k, score_fn=s.score)
    idx = torch.empty(T, s.k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, s.k, device="cuda")
    rg.moe_route(plan, T, logits, None, idx, w)
    res = layer.run(x)
    assert torch.equal(idx, res["topk_idx"])
    dO = torch.randn(T, s.D, device="cuda").bfloat16()
    bws = torch.empty(rg.moe_bwd_workspace_bytes(layer.plan, T), dtype=torch.uint8, device="cuda")
    g0 = grads_of(layer, T)
    g0["dW_router"] = torch.empty(s.E, s.D, device="cuda")
    rg.moe_bwd(layer.plan, T, x, layer.w, dO, layer.ws, g0, bws)
    out, status = fwd_routed(layer, x, idx, w)
    assert rel(out, res["out"].double()) <= 1e-2
    gr, dw = grads_of(layer, T), torch.empty(T, s.k, device="cuda")
    rg.moe_bwd_routed(layer.plan, T, x, layer.w, dO, layer.ws, gr, dw, bws)
    dl = torch.empty(T, s.E, device="cuda")
    rg.moe_route_bwd(plan, T, logits, idx, dw, dl)
    assert rel(dl.T @ x.float(), g0["dW_router"].double()) <= 1e-2
    assert rel(gr["dx"].float() + dl @ Wr.float(), g0["dx"].double()) <= 1e-2


def test_refusals():
    inp, layer, x = layer_of()
    s, T = inp.shape, inp.T
    idx, w = some_routing(T, s.E, s.k)
    out = torch.empty(T, s.D, dtype=torch.bfloat16, device="cuda")

    def code(f, *a, **kw):
        with pytest.raises(rg.MoEError) as ei:
            f(*a, **kw)
        return ei.value.code

    bad = rg.MOE_ERR_INVALID_ARG
    assert code(rg.moe_fwd_routed, layer.plan, T, x, layer.w, None, w, out, layer.ws) == bad
    assert code(rg.moe_fwd_routed, layer.plan, T, x, layer.w, idx, None, out, layer.ws) == bad
    assert code(rg.moe_fwd_routed, layer.plan, T, x, layer.w, idx.data_ptr() + 2, w, out, layer.ws) == bad
    assert code(rg.moe_fwd_routed, layer.plan, layer.T_max + 1, x, layer.w, idx, w, out, layer.ws) == bad
    assert code(rg.moe_fwd_routed, layer.plan, T, None, layer.w, idx, w, out, layer.ws) == bad
    assert code(rg.moe_fwd_routed, layer.plan, T, x, layer.w, idx, w, out, layer.ws, workspace_bytes=256) == \
        rg.MOE_ERR_WORKSPACE_TOO_SMALL
    inp, layer, x = bwd_layer(0)
    gr = grads_of(layer, inp.T)
    assert code(rg.moe_bwd_routed, layer.plan, inp.T, x, layer.w, x, layer.ws, gr, None, layer.ws) == bad


@pytest.mark.parametrize("pair", [0, 1])
def test_a_backward_of_the_other_forward_is_reported(pair):
    """moe_bwd after moe_fwd_routed, and moe_bwd_routed after moe_fwd: the status
    says so, and what would be wrong is NaN."""
    inp, layer, x = bwd_layer(pair)
    s, T = inp.shape, inp.T
    dO = torch.randn(T, s.D, device="cuda").bfloat16()
    bws = torch.zeros(rg.moe_bwd_workspace_bytes(layer.plan, T), dtype=torch.uint8, device="cuda")

    def built_in():
        gr = grads_of(layer, T)
        gr["dW_router"] = torch.zeros(s.E, s.D, device="cuda")
        rg.moe_bwd(layer.plan, T, x, layer.w, dO, layer.ws, gr, bws)
        return rg.moe_get_status(layer.plan, bws), gr

    def routed():
        gr, dw = grads_of(layer, T), torch.zeros(T, s.k, device="cuda")
        rg.moe_bwd_routed(layer.plan, T, x, layer.w, dO, layer.ws, gr, dw, bws)
        return rg.moe_get_status(layer.plan, bws), dw

    res = layer.run(x)
    status, ref = built_in()
    assert status == rg.MOE_STATUS_OK
    status, dw = routed()
    assert status == rg.MOE_STATUS_SCHEDULE_INVALID and bool(torch.isnan(dw).all())
    fwd_routed(layer, x, res["topk_idx"], res["topk_w"])
    status, gr = built_in()
    assert status == rg.MOE_STATUS_SCHEDULE_INVALID
    hit = torch.bincount(res["topk_idx"].flatten().long(), minlength=s.E) > 0
    assert bool(torch.isnan(gr["dW_router"][hit]).all()) and bool(torch.isnan(gr["dx"]).all())
    status, dw = routed()
    assert status == rg.MOE_STATUS_OK and bool(torch.isfinite(dw).all())
    # the next forward decides again
    layer.run(x)
    status, again = built_in()
    assert status == rg.MOE_STATUS_OK and all(torch.equal(ref[k], again[k]) for k in ref)


@pytest.mark.parametrize("kw", [dict(), dict(mma_pair=1, dispatch="spread"), dict(dispatch="direct", gather_ctas=0)])
@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
def test_an_empty_slots_expert_does_not_reach_the_status(precision, kw):
    """Expert 0 runs in every empty slot; its outputs leave fp16's range, which
    concerns only tokens that were routed to it."""
    inp, layer, x = layer_of(mi.custom_shape(300, 256, 128, 16, 4, 128, precision=precision), **kw)
    s, T = inp.shape, inp.T
    g = torch.Generator(device="cuda").manual_seed(4)
    idx = 1 + torch.rand(T, s.E - 1, generator=g, device="cuda").argsort(1)[:, :s.k].to(torch.int32)
    idx[torch.rand(T, s.k, generator=g, device="cuda") < 0.3] = -1
    w = torch.rand(T, s.k, generator=g, device="cuda") + 0.1
    ref, status = fwd_routed(layer, x, idx, w)
    assert status == rg.MOE_STATUS_OK
    if precision == "mxfp8":
        big = layer.w_bf16["W_down"].clone()
        big[0] *= 2.0 ** 40
        rg.moe_quantize_mxfp8(layer.plan, big, s.E * s.D, s.I, layer.w["W_down"], layer.w["W_down_scale"])
    else:
        layer.w["W_down"][0] *= 2.0 ** 40
    out, status = fwd_routed(layer, x, idx, w)
    assert status == rg.MOE_STATUS_OK and torch.equal(out, ref)
    for t in (0, 130, T - 1):  # one route to expert 0 is enough
        i2 = idx.clone()
        i2[t, 1] = 0
        assert fwd_routed(layer, x, i2, w)[1] == rg.MOE_STATUS_STAGING_OVERFLOW
