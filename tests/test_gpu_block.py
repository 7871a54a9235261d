"""A block's feed-forward half put together: norm, the MoE layer, and the norm
behind it, as a serving loop (moe_norm, moe_decode) and a training step
(moe_norm, moe_fwd, moe_norm, moe_norm_bwd, moe_bwd, moe_norm_bwd) run them.

Tolerances, relative in the 2-norm: a rounding to bf16 is off by at most 2^-8
of an element, u = 2^-8 / sqrt(3) of the norm.  On the longest way of the
forward y and h of the first norm are rounded, which the product of gate and up
at most triples (2 x 3u), then the hidden row, the layer's output and the
second norm's y and h (4u): in quadrature sqrt(2 9 + 4) u = 4.7 u = 1.06e-2; two
layers in a row twice that many, 1.5e-2.  The backward adds the gradients at
four borders and two inside the layer, which its products of gradient and
activation take in beside the forward's: sqrt(22 + 2 9 + 6) u = 6.8 u = 1.5e-2.
Bounds of 2e-2 and 2.5e-2 leave the rest to weights of the routing, whose
logits see h's roundings.
"""
import pytest
import torch

import routing_grouped_expert_gemm_gb300 as rg

pytestmark = pytest.mark.gpu

D, I, E, K, I_S = 256, 256, 16, 4, 256
EPS = 1e-6


def rel(got, ref):
    assert torch.isfinite(got).all()
    return float((got.double() - ref).norm() / ref.norm())


def weights(g):
    rnd = lambda *s: (torch.randn(*s, generator=g, device="cuda") * s[-1] ** -0.5).bfloat16()  # noqa: E731
    return {"W_router": rnd(E, D), "W_up": rnd(E, I, D), "W_gate": rnd(E, I, D), "W_down": rnd(E, D, I),
            "Ws_up": rnd(I_S, D), "Ws_gate": rnd(I_S, D), "Ws_down": rnd(D, I_S)}


def norm_params(g):
    return {"post_weight": 1 + 0.2 * torch.randn(D, generator=g, device="cuda"),
            "pre_weight": 1 + 0.2 * torch.randn(D, generator=g, device="cuda"),
            "gate": 0.5 + 0.5 * torch.randn(D, generator=g, device="cuda")}


def norm64(v, w):
    return v * (v.square().mean(1, keepdim=True) + EPS) ** -0.5 * w


def silu_mlp(x, up, gate, down):
    return (torch.nn.functional.silu(x @ gate.T) * (x @ up.T)) @ down.T


def moe64(x, w, idx):
    """The layer in 64 bits, its selection given (which a rounding of x may decide)."""
    s = torch.sigmoid((x @ w["W_router"].T).gather(1, idx))
    s = s / s.sum(1, keepdim=True)
    out = silu_mlp(x, w["Ws_up"], w["Ws_gate"], w["Ws_down"])
    for e in range(E):
        t, j = (idx == e).nonzero(as_tuple=True)
        out = out.index_add(0, t, silu_mlp(x[t], w["W_up"][e], w["W_gate"][e], w["W_down"][e]) * s[t, j, None])
    return out


def norms64(p, x, o):
    y = x + p["gate"] * norm64(o, p["post_weight"])
    return y, norm64(y, p["pre_weight"])


def selection_fits(h, w, idx):
    """idx are the K largest logits of the stored h."""
    v = h.double() @ w["W_router"].double().T
    held = torch.zeros_like(v, dtype=torch.bool).scatter_(1, idx.long(), True)
    assert (v.masked_fill(~held, float("inf")).amin(1) >= v.masked_fill(held, float("-inf")).amax(1)).all()
    assert (held.sum(1) == K).all()


@pytest.mark.parametrize("T", [1, 13, 64])
def test_serving(T):
    """Two blocks for a few tokens: plans, workspace and streams as one loop keeps them, run, captured and replayed."""
    g = torch.Generator(device="cuda").manual_seed(T)
    plan = rg.moe_plan_create(64, D, I, E, K, I_S)
    norm = rg.moe_norm_plan_create(D, eps=EPS)
    layers = [(norm_params(g), weights(g)) for _ in range(2)]
    last = norm_params(g)
    ws = torch.full((rg.moe_decode_workspace_bytes(plan, T),), 0xFF, dtype=torch.uint8, device="cuda")
    new = lambda *s, t=torch.bfloat16: torch.empty(*s, dtype=t, device="cuda")  # noqa: E731
    x, o = torch.randn(T, D, generator=g, device="cuda").bfloat16(), torch.randn(T, D, generator=g, device="cuda").bfloat16()
    y, h, out = [[new(T, D) for _ in range(3)] for _ in range(3)]
    idx = [new(T, K, t=torch.int32) for _ in layers]
    x0, o0 = x.clone(), o.clone()

    def loop():
        a, b = x, o
        for i, (p, w) in enumerate(layers):
            rg.moe_norm(norm, T, p, x=a, o=b, y=y[i], h=h[i])
            rg.moe_decode(plan, T, h[i], w, out[i], ws, topk_idx=idx[i])
            a, b = y[i], out[i]
        rg.moe_norm(norm, T, last, x=a, o=b, y=y[2], h=h[2])

    def check():
        torch.cuda.synchronize()
        assert rg.moe_get_status(plan, ws) == rg.MOE_STATUS_OK
        a, b = x.double(), o.double()
        for i, (p, w) in enumerate(layers):
            selection_fits(h[i], w, idx[i])
            a, b = norms64(p, a, b)
            b = moe64(b, {n: v.double() for n, v in w.items()}, idx[i].long())
        a, b = norms64(last, a, b)
        assert rel(y[2], a) <= 2e-2 and rel(h[2], b) <= 2e-2

    loop()
    check()
    first = y[2].clone(), h[2].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        loop()
    x.copy_(o0)
    o.copy_(x0)
    graph.replay()
    check()
    x.copy_(x0)
    o.copy_(o0)
    graph.replay()
    loop()  # behind the replay, in the same buffers
    graph.replay()
    check()
    assert torch.equal(first[0], y[2]) and torch.equal(first[1], h[2])


@pytest.mark.parametrize("T", [2, 300])
def test_training_step(T):
    """Forward and backward through norm, layer and norm against differentiation in 64 bits."""
    g = torch.Generator(device="cuda").manual_seed(T)
    plan = rg.moe_plan_create(T, D, I, E, K, I_S, minibatch=1024, ring_slots=2, gather_ctas=2)
    norm = rg.moe_norm_plan_create(D, eps=EPS)
    w, p = weights(g), [norm_params(g), norm_params(g)]
    rnd = lambda s=1.0: (torch.randn(T, D, generator=g, device="cuda") * s).bfloat16()  # noqa: E731
    x, o, dy2, dh2 = rnd(), rnd(), rnd(), rnd()
    new = lambda *s, t=torch.bfloat16: torch.full(s, float("nan"), dtype=t, device="cuda")  # noqa: E731
    y, h, out, y2, h2 = [new(T, D) for _ in range(5)]
    st = [new(T, 4, t=torch.float32) for _ in range(2)]
    idx = torch.empty(T, K, dtype=torch.int32, device="cuda")
    ws = torch.empty(rg.moe_workspace_bytes(plan, T), dtype=torch.uint8, device="cuda")
    bws = torch.empty(rg.moe_bwd_workspace_bytes(plan, T), dtype=torch.uint8, device="cuda")
    nws = torch.empty(rg.moe_norm_workspace_bytes(norm, T), dtype=torch.uint8, device="cuda")
    dy, dout, dh, dx, do = [new(T, D) for _ in range(5)]
    gw = {"d" + n: new(*v.shape, t=torch.float32 if n == "W_router" else torch.bfloat16) for n, v in w.items()}
    gp = [{n: new(D, t=torch.float32) for n in q} for q in p]

    def step():
        rg.moe_norm(norm, T, p[0], x=x, o=o, y=y, h=h, stats=st[0])
        rg.moe_fwd(plan, T, h, w, out, ws, topk_idx=idx)
        rg.moe_norm(norm, T, p[1], x=y, o=out, y=y2, h=h2, stats=st[1])
        rg.moe_norm_bwd(norm, T, p[1], st[1], gp[1], o=out, y=y2, dy=dy2, dh=dh2, dx=dy, do=dout, workspace=nws)
        rg.moe_bwd(plan, T, h, w, dout, ws, {**gw, "dx": dh}, bws)
        rg.moe_norm_bwd(norm, T, p[0], st[0], gp[0], o=o, y=y, dy=dy, dh=dh, dx=dx, do=do, workspace=nws)

    step()
    assert rg.moe_get_status(plan, ws) == rg.MOE_STATUS_OK and rg.moe_get_status(plan, bws) == rg.MOE_STATUS_OK
    selection_fits(h, w, idx)
    leaf = lambda t: t.double().requires_grad_()  # noqa: E731
    x64, o64, w64 = leaf(x), leaf(o), {n: leaf(v) for n, v in w.items()}
    p64 = [{n: leaf(v) for n, v in q.items()} for q in p]
    a, b = norms64(p64[0], x64, o64)
    a, b = norms64(p64[1], a, moe64(b, w64, idx.long()))
    assert rel(y2, a.detach()) <= 2e-2 and rel(h2, b.detach()) <= 2e-2
    ((a * dy2.double()).sum() + (b * dh2.double()).sum()).backward()
    got = {"dx": (dx, x64), "do": (do, o64), **{"d" + n: (gw["d" + n], w64[n]) for n in w}}
    for i in range(2):
        got.update({f"d{n} {i}": (gp[i][n], p64[i][n]) for n in p[i]})
    far = {n: r for n, (v, t) in got.items() if not (r := rel(v, t.grad)) <= 2.5e-2}
    assert not far, far

    eager = {n: v.clone() for n, (v, _) in got.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for v, _ in got.values():
        v.fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(eager[n], v) for n, (v, _) in got.items())
