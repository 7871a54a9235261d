"""moe_route and moe_route_bwd against a plain fp64 implementation.

Tolerances: the selection and the counts are exact.  Weights: exp (2 ulp), a
sum of k terms, a quotient and a product, each half an ulp of fp32 or a few of
them: 16 * 2^-24 relative covers sigmoid; softmax adds the rounding of x - m,
|x - m| 2^-24 relative, at most 32 for these logits.  The gradient is rounded
once to its type, and its terms cancel (a - q sum a): the fp32 error counts
against the largest term of the row, not against the result."""
import numpy as np
import pytest
import torch

import routing_grouped_expert_gemm_gb300 as rg

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
U32 = 2.0 ** -24
HALF_ULP = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


def scores(x, fn):
    if fn == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(np.isneginf(x), 0.0, 1.0 / (1.0 + np.exp(-x)))
    m = x.max(1, keepdims=True)
    e = np.exp(x - np.where(np.isneginf(m), 0.0, m))
    z = e.sum(1, keepdims=True)
    return e / np.where(z == 0, 1.0, z)


def log_scores(x, fn):
    """Up to a constant per row (what a renormalised weight needs, without underflow)."""
    with np.errstate(over="ignore"):
        return x if fn == "softmax" else np.where(np.isneginf(x), -np.inf, -np.logaddexp(0.0, -x))


def plain_route(x, bias, k, fn, n_group, topk_group, group_top, renorm, scale):
    """Row by row, from the definition."""
    T, E = x.shape
    s, ls = scores(x, fn), log_scores(x, fn)
    idx = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    counts = np.zeros(E, np.int64)
    gs = E // n_group
    for t in range(T):
        live = [e for e in range(E) if x[t, e] > -np.inf]
        key = x[t] if bias is None else s[t] + bias
        val = s[t] if bias is None else key
        if n_group > 1:
            rank = []
            for g in range(n_group):
                v = sorted((val[e] for e in live if e // gs == g), reverse=True)[:group_top]
                rank.append((-sum(v) if v else np.inf, g))
            keep = {g for _, g in sorted(rank)[:topk_group]}
            live = [e for e in live if e // gs in keep]
        sel = sorted(sorted(live, key=lambda e: (-key[e], e))[:k])
        for i, e in enumerate(sel):
            idx[t, i] = e
            counts[e] += 1
        if sel:
            if renorm:
                l = ls[t, sel]
                u = np.exp(l - l.max())
                w[t, :len(sel)] = scale * u / u.sum()
            else:
                w[t, :len(sel)] = scale * s[t, sel]
    l = np.exp(ls - np.where(np.isneginf(ls.max(1, keepdims=True)), 0.0, ls.max(1, keepdims=True)))
    tot = l.sum(1, keepdims=True)
    return idx, w, counts, (l / np.where(tot == 0, 1.0, tot)).sum(0)


def run_route(x, bias, cfg, sums=True, stride=0, stream=None):
    T, E = x.shape[0], cfg["E"]
    plan = rg.moe_route_plan_create(**cfg)
    k = cfg["k"]
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    cnt = torch.full((E,), -7, dtype=torch.int32, device="cuda") if sums else None
    ps = torch.full((E,), float("nan"), device="cuda") if sums else None
    ws = torch.full((rg.moe_route_workspace_bytes(plan, T),), 0xFF, dtype=torch.uint8, device="cuda")
    rg.moe_route(plan, T, x, bias, idx, w, expert_counts=cnt, prob_sum=ps, workspace=ws, logits_stride=stride, stream=stream)
    return plan, idx, w, cnt, ps


def cfg_of(E, k, fn="sigmoid", dtype="fp32", n_group=1, topk_group=1, group_top=2, renorm=True, scale=1.0):
    return dict(E=E, k=k, score_fn=fn, logits_dtype=dtype, n_group=n_group, topk_group=topk_group, group_top=group_top,
                renormalize=renorm, scale=scale)


def check_route(x, bias, cfg, stride=0):
    """x: device logits [T, >= E]."""
    plan, idx, w, cnt, ps = run_route(x, bias, cfg, stride=stride)
    xe = x[:, :cfg["E"]].double().cpu().numpy()
    b = None if bias is None else bias.double().cpu().numpy()
    ri, rw, rc, rp = plain_route(xe, b, cfg["k"], cfg["score_fn"], cfg["n_group"], cfg["topk_group"], cfg["group_top"],
                                 cfg["renormalize"], cfg["scale"])
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert np.array_equal(cnt.cpu().numpy(), rc)
    tol = (16 + 32 * (cfg["score_fn"] == "softmax")) * U32
    assert np.abs(w.double().cpu().numpy() - rw).max(initial=0.0) <= tol * cfg["scale"]
    # a sum over T rows in fp32, in runs of at most T / 8 rows per lane and then per CTA
    assert np.all(np.abs(ps.double().cpu().numpy() - rp) <= (tol + 2e-6) * np.maximum(rp, 1e-3))
    return idx, w


CASES = [
    # T, E, k, kwargs
    (1, 256, 8, dict(n_group=8, topk_group=4, scale=2.5)),
    (1, 1, 1, {}),
    (3, 2, 2, dict(fn="softmax", renorm=False)),
    (7, 33, 5, dict(fn="softmax")),
    (130, 64, 6, dict(fn="softmax", n_group=4, topk_group=2, group_top=1)),
    (65, 100, 16, dict(n_group=5, topk_group=3)),
    (50, 100, 6, dict(n_group=25, topk_group=2, group_top=1, fn="softmax", renorm=False, scale=2.5)),
    (40, 96, 3, dict(n_group=32, topk_group=1)),
    (200, 256, 8, dict(n_group=8, topk_group=4, renorm=False, scale=2.5)),
    (77, 384, 8, dict(scale=2.5)),
    (64, 384, 6, dict(n_group=12, topk_group=5)),
    (33, 512, 16, dict(fn="softmax", n_group=16, topk_group=16)),
    (2500, 128, 8, dict(fn="softmax")),
    (5000, 60, 4, dict(n_group=4, topk_group=2)),
]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,k,kw", CASES)
def test_route_matches_fp64(T, E, k, kw, with_bias, dtype):
    g = torch.Generator(device="cuda").manual_seed(T * 1000 + E)
    x = (torch.randn(T, E, generator=g, device="cuda") * 1.5).to(DTYPES[dtype])
    bias = (torch.rand(E, generator=g, device="cuda") - 0.5) * 0.2 if with_bias else None
    check_route(x, bias, cfg_of(E, k, dtype=dtype, **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masked_experts_and_empty_rows(fn, with_bias):
    g = torch.Generator(device="cuda").manual_seed(5)
    T, E = 300, 48
    x = torch.randn(T, E, generator=g, device="cuda")
    x[torch.rand(T, E, generator=g, device="cuda") < 0.8] = -float("inf")
    x[::7] = -float("inf")
    bias = torch.randn(E, generator=g, device="cuda") if with_bias else None
    for kw in (dict(), dict(n_group=6, topk_group=2), dict(n_group=6, topk_group=3, group_top=1, renorm=False)):
        idx, w = check_route(x, bias, cfg_of(E, 9, fn=fn, **kw))
        assert bool((idx[::7] == -1).all()) and bool((w[::7] == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
def test_ties_go_to_the_lowest_id(fn):
    """Few distinct logits and biases: equal keys everywhere; and biases that
    make different logits nearly equal in key (decided as in fp64)."""
    g = torch.Generator(device="cuda").manual_seed(9)
    T, E = 257, 128
    x = torch.randint(-2, 3, (T, E), generator=g, device="cuda").float()
    zero = torch.zeros(E, device="cuda")
    steps = torch.randint(0, 2, (E,), generator=g, device="cuda").float() * 0.25
    for bias in (None, zero, steps):
        for kw in (dict(), dict(n_group=8, topk_group=3), dict(n_group=8, topk_group=3, group_top=1)):
            check_route(x, bias, cfg_of(E, 8, fn=fn, **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("shift", [-30.0, 25.0])
def test_keys_closer_than_fp32_resolves(fn, shift):
    """Saturated scores (sigmoid near 0 or 1) whose fp32 values collide, and
    biases that offset score differences: the selection is fp64's."""
    g = torch.Generator(device="cuda").manual_seed(11)
    T, E = 400, 64
    x = torch.randn(T, E, generator=g, device="cuda") + (shift if fn == "sigmoid" else 0.0)
    b = torch.rand(E, generator=g, device="cuda") * 1e-7 if shift > 0 else torch.zeros(E, device="cuda")
    for kw in (dict(), dict(n_group=8, topk_group=4)):
        check_route(x, b, cfg_of(E, 6, fn=fn, **kw))
    # every row: x_1 = x_0 up to an ulp, the bias making up for the difference in fp32
    x[:, 1] = torch.nextafter(x[:, 0], x[:, 0] + 1)
    x[:, :2] += 2.0
    check_route(x, torch.zeros(E, device="cuda"), cfg_of(E, 1, fn=fn))


@pytest.mark.gpu
def test_very_low_sigmoid_scores_keep_their_weights():
    x = torch.tensor([[-200.0, -201.0, -202.0, -300.0], [-90.0, -95.0, 3.0, -90.0]], device="cuda")
    b = torch.tensor([0.0, 0.0, -2.0, -1.0], device="cuda")
    plan, idx, w, _, _ = run_route(x, b, cfg_of(4, 2))
    assert idx.tolist() == [[0, 1], [0, 1]]
    for r, d in ((0, 1.0), (1, 5.0)):
        want = np.array([1.0, np.exp(-d)]) / (1.0 + np.exp(-d))
        assert np.abs(w[r].double().cpu().numpy() - want).max() <= 16 * U32


@pytest.mark.gpu
def test_nan_and_infinite_logits():
    nan, inf = float("nan"), float("inf")
    x = torch.tensor([[nan, 1.0, 2.0, 3.0], [inf, 1.0, 2.0, 3.0], [0.0, 1.0, 2.0, 3.0]], device="cuda")
    plan, idx, w, _, _ = run_route(x, None, cfg_of(4, 2, fn="softmax"))
    assert idx.tolist() == [[2, 3], [0, 3], [2, 3]]
    assert bool(torch.isnan(w[0]).all()) and w[1].tolist() == [1.0, 0.0] and bool(torch.isfinite(w[2]).all())
    plan, idx, w, _, _ = run_route(x, None, cfg_of(4, 2, fn="sigmoid", renorm=False))
    assert idx.tolist() == [[2, 3], [0, 3], [2, 3]] and bool(torch.isfinite(w).all()) and float(w[1, 0]) == 1.0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("pad", [1, 8, 13])
def test_row_strides_and_offset_bases(dtype, pad):
    g = torch.Generator(device="cuda").manual_seed(3)
    T, E = 90, 64
    big = torch.randn(T, E + pad, generator=g, device="cuda").to(DTYPES[dtype])
    check_route(big, None, cfg_of(E, 4, dtype=dtype), stride=E + pad)
    check_route(big[:, 1:], None, cfg_of(E - 1, 4, dtype=dtype), stride=E + pad)  # a base that is not 16-byte aligned
    # the gradient with strides on both sides writes its rows' E elements only
    plan, idx, w, _, _ = run_route(big, None, cfg_of(E, 4, dtype=dtype), stride=E + pad)
    d = torch.full((T, E + pad), 7.0, device="cuda").to(DTYPES[dtype])
    dw = torch.randn(T, 4, generator=g, device="cuda")
    rg.moe_route_bwd(plan, T, big, idx, dw, d, logits_stride=E + pad, dlogits_stride=E + pad)
    d0 = torch.empty(T, E, device="cuda", dtype=DTYPES[dtype])
    rg.moe_route_bwd(plan, T, big[:, :E].contiguous(), idx, dw, d0)
    assert bool((d[:, E:] == 7).all()) and torch.equal(d[:, :E], d0)


@pytest.mark.gpu
def test_another_stream_and_no_tokens():
    T, E = 1000, 64
    x = torch.randn(T, E, device="cuda")
    ref = run_route(x, None, cfg_of(E, 4))
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = run_route(x, None, cfg_of(E, 4), stream=st)
    torch.cuda.synchronize()
    for a, b in zip(ref[1:], got[1:]):
        assert torch.equal(a, b)
    _, idx, w, cnt, ps = run_route(x[:0], None, cfg_of(E, 4))
    assert int(cnt.abs().sum()) == 0 and float(ps.abs().sum()) == 0.0


def jacobian_bwd(x, idx, dw, dps, fn, renorm, scale):
    """dL/dx in fp64 by torch's autograd over the definition; and, per element,
    the sum of the absolute values of the terms that make it up."""
    x = torch.tensor(x, dtype=torch.float64, requires_grad=True)
    live = x > -float("inf")
    xs = torch.where(live, x, torch.zeros_like(x))
    if fn == "sigmoid":
        s = torch.where(live, torch.sigmoid(xs), torch.zeros_like(x))
    else:
        m = torch.where(live, x, torch.full_like(x, -1e300)).max(1, keepdim=True).values.detach()
        e = torch.where(live, torch.exp(torch.where(live, x - m, torch.zeros_like(x))), torch.zeros_like(x))
        s = e / e.sum(1, keepdim=True).clamp_min(1e-300)
    on = torch.tensor(idx >= 0)
    at = torch.tensor(np.where(idx >= 0, idx, 0)).long()
    q = torch.where(on, torch.gather(s, 1, at), torch.zeros_like(dw))
    w = q / q.sum(1, keepdim=True).clamp_min(1e-300) if renorm else q
    loss = (w * dw).sum() * scale
    if dps is not None:
        loss = loss + ((s / s.sum(1, keepdim=True).clamp_min(1e-300)).sum(0) * dps).sum()
    loss.backward()
    return x.grad.numpy()


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("sums", [True, False])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,E,k", [(1, 256, 8), (37, 60, 4), (9, 1, 1), (130, 33, 16), (2100, 384, 8), (70, 512, 10)])
def test_gradient_matches_fp64_autograd(T, E, k, fn, renorm, sums, dtype):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    k = min(k, E)
    x = torch.randn(T, E, generator=g, device="cuda") * 1.5
    x[torch.rand(T, E, generator=g, device="cuda") < 0.1] = -float("inf")
    if T > 8:
        x[3] = -float("inf")
    x = x.to(DTYPES[dtype])
    plan, idx, w, _, _ = run_route(x, None, cfg_of(E, k, fn=fn, dtype=dtype, renorm=renorm, scale=2.5))
    dw = torch.randn(T, k, generator=g, device="cuda")
    dps = torch.randn(E, generator=g, device="cuda") if sums else None
    d = torch.full((T, E), float("nan"), device="cuda").to(DTYPES[dtype])
    rg.moe_route_bwd(plan, T, x, idx, dw, d, dprob_sum=dps)
    ref = jacobian_bwd(x.double().cpu().numpy(), idx.cpu().numpy(), dw.double().cpu(),
                       None if dps is None else dps.double().cpu(), fn, renorm, 2.5)
    got = d.double().cpu().numpy()
    # terms up to (2.5 |dw| + |d|) times a score of at most 1, each with fp32 errors as the weights'; fp16's
    # smallest step is 2^-24
    size = 2.5 * dw.abs().max(1, keepdim=True).values.double().cpu().numpy() + (0 if dps is None else float(dps.abs().max()))
    err32 = 4 * 48 * U32 * size
    tol = HALF_ULP[dtype] * np.abs(ref) + err32 + (2.0 ** -25 if dtype == "fp16" else 0.0)
    assert np.all(np.abs(got - ref) <= tol)
    assert np.all(got[np.isneginf(x.double().cpu().numpy())] == 0)


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gradient_matches_differences(fn, renorm):
    """Central differences of the fp64 definition with the selection held: step
    h leaves h^2 / 6 times the third derivative (below 8 for these scores)."""
    g = torch.Generator(device="cuda").manual_seed(2)
    T, E, k, h = 5, 24, 3, 1e-3
    x = torch.randn(T, E, generator=g, device="cuda")
    plan, idx, w, _, _ = run_route(x, None, cfg_of(E, k, fn=fn, renorm=renorm))
    dw = torch.randn(T, k, generator=g, device="cuda")
    dps = torch.randn(E, generator=g, device="cuda")
    d = torch.empty(T, E, device="cuda")
    rg.moe_route_bwd(plan, T, x, idx, dw, d, dprob_sum=dps)
    xn, i, a, b = x.double().cpu().numpy(), idx.cpu().numpy(), dw.double().cpu().numpy(), dps.double().cpu().numpy()

    def loss(v):
        s = scores(v, fn)
        q = np.take_along_axis(s, i.astype(np.int64), 1)
        q = q / q.sum(1, keepdims=True) if renorm else q
        return (q * a).sum(1) + ((s / s.sum(1, keepdims=True)) * b).sum(1)

    num = np.zeros((T, E))
    for e in range(E):
        up, dn = xn.copy(), xn.copy()
        up[:, e] += h
        dn[:, e] -= h
        num[:, e] = (loss(up) - loss(dn)) / (2 * h)
    size = np.abs(a).max() + np.abs(b).max()
    assert np.abs(d.double().cpu().numpy() - num).max() <= size * (8 * h * h / 6 + 4 * 48 * U32)


@pytest.mark.gpu
def test_gradient_skips_slots_outside_the_range():
    T, E, k = 4, 16, 3
    x = torch.randn(T, E, device="cuda")
    plan = rg.moe_route_plan_create(E, k)
    idx = torch.tensor([[-1, -1, -1], [2, 5, 99], [2, 5, -1], [1 << 30, -(1 << 30), 3]], dtype=torch.int32, device="cuda")
    dw = torch.randn(T, k, device="cuda")
    dw[2, :2] = dw[1, :2]
    x[2] = x[1]
    d = torch.full((T, E), float("nan"), device="cuda")
    rg.moe_route_bwd(plan, T, x, idx, dw, d)
    assert bool((d[0] == 0).all()) and torch.equal(d[1], d[2]) and bool(torch.isfinite(d).all())


@pytest.mark.gpu
def test_repeated_calls_and_a_graph_give_the_same_bits():
    T, E = 3000, 256
    x = torch.randn(T, E, device="cuda")
    bias = torch.rand(E, device="cuda") * 0.1
    cfg = cfg_of(E, 8, n_group=8, topk_group=4)
    plan, idx, w, cnt, ps = run_route(x, bias, cfg)
    ws = torch.empty(rg.moe_route_workspace_bytes(plan, T), dtype=torch.uint8, device="cuda")
    idx2, w2, cnt2, ps2 = (torch.zeros_like(t) for t in (idx, w, cnt, ps))
    d, d2 = torch.empty_like(x), torch.zeros_like(x)
    dw = torch.randn(T, 8, device="cuda")
    rg.moe_route_bwd(plan, T, x, idx, dw, d, dprob_sum=bias)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rg.moe_route(plan, T, x, bias, idx2, w2, cnt2, ps2, ws)
        rg.moe_route_bwd(plan, T, x, idx2, dw, d2, dprob_sum=bias)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for a, b in ((idx, idx2), (w, w2), (cnt, cnt2), (ps, ps2), (d, d2)):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- refusals (no GPU needed)
@pytest.fixture(scope="module")
def L():
    from routing_grouped_expert_gemm_gb300 import build as rgbuild
    rgbuild.build()
    return rg.lib()


@pytest.mark.parametrize("kw,code", [
    (dict(E=0), rg.MOE_ERR_UNSUPPORTED_SHAPE), (dict(E=513), rg.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(k=0), rg.MOE_ERR_UNSUPPORTED_SHAPE), (dict(k=17), rg.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(n_group=0), rg.MOE_ERR_UNSUPPORTED_SHAPE), (dict(n_group=7), rg.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(n_group=64, topk_group=64), rg.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(n_group=8, topk_group=9), rg.MOE_ERR_UNSUPPORTED_SHAPE), (dict(topk_group=0), rg.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(n_group=32, topk_group=1), rg.MOE_ERR_UNSUPPORTED_SHAPE),  # 8 of 2 experts
    (dict(score_fn=2), rg.MOE_ERR_INVALID_ARG), (dict(logits_dtype=3), rg.MOE_ERR_INVALID_ARG),
    (dict(logits_dtype=-1), rg.MOE_ERR_INVALID_ARG), (dict(group_top=3), rg.MOE_ERR_INVALID_ARG),
    (dict(group_top=0), rg.MOE_ERR_INVALID_ARG), (dict(scale=float("nan")), rg.MOE_ERR_INVALID_ARG),
    (dict(scale=float("inf")), rg.MOE_ERR_INVALID_ARG), (dict(renormalize=2), rg.MOE_ERR_INVALID_ARG),
])
def test_plan_refusals(L, kw, code):
    with pytest.raises(rg.MoEError) as ei:
        rg.moe_route_plan_create(**{**dict(E=64, k=8), **kw})
    assert ei.value.code == code


def test_null_plan_refusals(L):
    assert L.moe_route_plan_create(None, None) == rg.MOE_ERR_INVALID_ARG
    assert L.moe_route_workspace_bytes(None, 4) == 0
    assert L.moe_route(None, 1, None, 0, None, None, None, None, None, None, 0, None) == rg.MOE_ERR_INVALID_ARG
    assert L.moe_route_bwd(None, 1, None, 0, None, None, None, None, 0, None) == rg.MOE_ERR_INVALID_ARG
    assert L.moe_route_plan_destroy(None) == 0


@pytest.mark.gpu
def test_call_refusals():
    T, E, k = 100, 64, 8
    plan = rg.moe_route_plan_create(E, k)
    x = torch.randn(T, E, device="cuda")
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, device="cuda")
    cnt = torch.empty(E, dtype=torch.int32, device="cuda")

    def code(f, *a, **kw):
        with pytest.raises(rg.MoEError) as ei:
            f(*a, **kw)
        return ei.value.code

    bad = rg.MOE_ERR_INVALID_ARG
    assert code(rg.moe_route, plan, -1, x, None, idx, w) == bad
    assert code(rg.moe_route, plan, T, None, None, idx, w) == bad
    assert code(rg.moe_route, plan, T, x, None, None, w) == bad
    assert code(rg.moe_route, plan, T, x, None, idx, None) == bad
    assert code(rg.moe_route, plan, T, x, None, idx, w, logits_stride=E - 1) == bad
    assert code(rg.moe_route, plan, T, x.data_ptr() + 2, None, idx, w) == bad
    assert code(rg.moe_route, plan, T, x, None, idx, w, expert_counts=cnt) == bad  # sums want a workspace
    ws = torch.empty(16, dtype=torch.uint8, device="cuda")
    assert code(rg.moe_route, plan, T, x, None, idx, w, expert_counts=cnt, workspace=ws) == rg.MOE_ERR_WORKSPACE_TOO_SMALL
    assert code(rg.moe_route_bwd, plan, T, x, idx, None, x.clone()) == bad
    assert code(rg.moe_route_bwd, plan, T, x, idx, w, None) == bad
    assert code(rg.moe_route_bwd, plan, T, x, idx, w, x.clone(), dlogits_stride=E - 1) == bad


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_many_equal_or_crowded_keys(fn, with_bias):
    """More equal (or nearly equal) keys than one lane each can hold: all logits
    the same; the large ones all in a few neighbouring experts; logits so close
    that a whole row is within fp32's error."""
    g = torch.Generator(device="cuda").manual_seed(21)
    T, E = 64, 512
    flat = torch.full((T, E), 0.25, device="cuda")
    crowd = torch.randn(T, E, generator=g, device="cuda") - 20.0
    crowd[:, 32:80] += 20.0
    near = 0.5 + torch.randint(0, 3, (T, E), generator=g, device="cuda") * 2.0 ** -23
    for x in (flat, crowd, near):
        for bias in ((torch.zeros(E, device="cuda"), torch.randint(0, 3, (E,), generator=g, device="cuda") * 2.0 ** -25)
                     if with_bias else (None,)):
            for kw in (dict(), dict(n_group=16, topk_group=2), dict(n_group=2, topk_group=1, group_top=1)):
                check_route(x, bias, cfg_of(E, 16, fn=fn, **kw))


def plain_route_rows(x, bias, k, fn, n_group, topk_group, group_top, renorm, scale):
    """plain_route for many rows at once (sorted keys, stable: ties to the lower id)."""
    T, E = x.shape
    s, ls = scores(x, fn), log_scores(x, fn)
    live = x > -np.inf
    key = np.where(live, x if bias is None else s + bias, -np.inf)
    if n_group > 1:
        val = np.where(live, s if bias is None else s + bias, -np.inf).reshape(T, n_group, -1)
        top = -np.sort(-val, axis=2)[:, :, :group_top]
        none = np.isneginf(top[:, :, 0])
        gs = np.where(none, -np.inf, np.where(np.isneginf(top), 0.0, top).sum(2))
        place = np.argsort(np.argsort(-gs, axis=1, kind="stable"), axis=1, kind="stable")
        key = np.where(np.repeat((place < topk_group) & ~none, E // n_group, axis=1), key, -np.inf)
    first = np.argsort(-key, axis=1, kind="stable")[:, :k]
    ok = ~np.isneginf(np.take_along_axis(key, first, 1))
    idx = np.sort(np.where(ok, first, E), axis=1)
    got = idx < E
    at = np.where(got, idx, 0)
    if renorm:
        l = np.where(got, np.take_along_axis(ls, at, 1), -np.inf)
        u = np.exp(l - np.where(got.any(1, keepdims=True), l.max(1, keepdims=True), 0.0))
        w = scale * u / np.maximum(u.sum(1, keepdims=True), 1e-300)
    else:
        w = np.where(got, scale * np.take_along_axis(s, at, 1), 0.0)
    lm = ls.max(1, keepdims=True)
    l = np.exp(ls - np.where(np.isneginf(lm), 0.0, lm))
    tot = l.sum(1, keepdims=True)
    return (np.where(got, idx, -1).astype(np.int32), w, np.bincount(idx[got], minlength=E),
            (l / np.where(tot == 0, 1.0, tot)).sum(0))


def check_rows(x, bias, cfg):
    plan, idx, w, cnt, ps = run_route(x, bias, cfg)
    b = None if bias is None else bias.double().cpu().numpy()
    args = (x.double().cpu().numpy(), b, cfg["k"], cfg["score_fn"], cfg["n_group"], cfg["topk_group"], cfg["group_top"],
            cfg["renormalize"], cfg["scale"])
    ri, rw, rc, rp = plain_route_rows(*args)
    assert np.array_equal(idx.cpu().numpy(), ri)
    assert np.array_equal(cnt.cpu().numpy(), rc)
    tol = (16 + 32 * (cfg["score_fn"] == "softmax")) * U32
    assert np.abs(w.double().cpu().numpy() - rw).max() <= tol * cfg["scale"]
    assert np.all(np.abs(ps.double().cpu().numpy() - rp) <= (tol + 2e-6) * np.maximum(rp, 1e-3))
    _, i2, w2, _, _ = run_route(x, bias, cfg, sums=False)  # (a kernel of its own)
    assert torch.equal(i2, idx) and torch.equal(w2, w)


def test_the_two_plain_forms_agree():
    r = np.random.default_rng(0)
    x = r.standard_normal((40, 24))
    x[r.random((40, 24)) < 0.3] = -np.inf
    x[3] = -np.inf
    x = np.round(x * 2) / 2
    for fn in ("sigmoid", "softmax"):
        for b in (None, np.round(r.standard_normal(24) * 4) / 8):
            for a in ((5, fn, 1, 1, 2, True, 1.0), (5, fn, 4, 2, 2, False, 2.5), (4, fn, 6, 2, 1, True, 1.0)):
                u, v = plain_route(x, b, *a), plain_route_rows(x, b, *a)
                assert np.array_equal(u[0], v[0]) and np.array_equal(u[2], v[2])
                assert np.allclose(u[1], v[1], rtol=1e-12) and np.allclose(u[3], v[3], rtol=1e-12)


MANY = [(9728, 256, 8, dict(n_group=8, topk_group=4, scale=2.5)), (9731, 256, 8, {}), (9800, 200, 16, dict(renorm=False)),
        (9733, 64, 6, {}), (9730, 60, 4, dict(n_group=4, topk_group=2)), (9999, 128, 8, dict(n_group=4, topk_group=2)),
        (9729, 128, 3, dict(n_group=8, topk_group=1, group_top=1)), (10001, 33, 1, {}), (9728, 16, 4, dict(n_group=2)),
        (4864, 384, 8, dict(scale=2.5)), (4865, 384, 6, dict(n_group=8, topk_group=3)), (5001, 300, 10, {}),
        (4867, 512, 16, dict(n_group=16, topk_group=5)), (5003, 512, 10, dict(renorm=False)), (20003, 256, 5, {})]


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,k,kw", MANY)
def test_many_rows_match_fp64(T, E, k, kw, with_bias, fn):
    """Row counts from which several rows share a warp, and odd ones."""
    g = torch.Generator(device="cuda").manual_seed(T + E)
    dtype = ("fp32", "bf16", "fp16")[(T + E + with_bias) % 3]
    x = torch.randn(T, E, generator=g, device="cuda") * 1.5
    if T % 2:
        x[torch.rand(T, E, generator=g, device="cuda") < 0.2] = -float("inf")
        x[::97] = -float("inf")
    bias = (torch.rand(E, generator=g, device="cuda") - 0.5) * 0.2 if with_bias else None
    check_rows(x.to(DTYPES[dtype]), bias, cfg_of(E, k, fn=fn, dtype=dtype, **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_many_rows_with_ties_and_crowds(fn, with_bias):
    """Rows that several to a warp cannot hold, beside ones that they can."""
    g = torch.Generator(device="cuda").manual_seed(4)
    T, E = 9728, 256
    x = torch.randn(T, E, generator=g, device="cuda") * 1.5
    few = torch.randint(-2, 3, (T, E), generator=g, device="cuda").float()
    x[::3] = few[::3]                       # ties everywhere
    x[1::7] = x[1::7] - 20.0
    x[1::7, 40:64] += 20.0                  # the large ones side by side
    x[2::11] = 0.25                         # one value
    x[5::13] -= 60.0                        # sigmoid scores of 1e-26
    x[6::17] = 0.5 + torch.randint(0, 3, (len(x[6::17]), E), generator=g, device="cuda") * 2.0 ** -23
    bias = torch.zeros(E, device="cuda") if with_bias else None
    for kw in (dict(n_group=8, topk_group=4), dict(), dict(n_group=8, topk_group=2, group_top=1, renorm=False)):
        check_rows(x, bias, cfg_of(E, 8, fn=fn, **kw))
        if with_bias:
            check_rows(x, torch.randint(0, 3, (E,), generator=g, device="cuda") * 2.0 ** -25, cfg_of(E, 8, fn=fn, **kw))


@pytest.mark.gpu
def test_many_rows_with_nan():
    T, E = 9728, 256
    g = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(T, E, generator=g, device="cuda")
    _, i0, w0, _, _ = run_route(x, None, cfg_of(E, 8, fn="softmax"))
    y = x.clone()
    y[5, 17] = float("nan")
    y[6, 0] = float("inf")
    _, i1, w1, _, ps = run_route(y, None, cfg_of(E, 8, fn="softmax"))
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[5:7] = False
    assert torch.equal(i0[keep], i1[keep]) and torch.equal(w0[keep], w1[keep])
    assert bool(torch.isnan(w1[5]).all()) and 17 not in i1[5].tolist() and bool(torch.isnan(ps).all())
    assert i1[6, 0] == 0 and float(w1[6, 0]) == 1.0 and float(w1[6, 1:].abs().sum()) == 0.0


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """More than 2^32 bytes of logits: the last rows are those of a call of their own."""
    T, E, k = (1 << 22) + 37, 264, 8
    x = torch.empty(T, E, device="cuda")
    x.uniform_(-3.0, 3.0)
    bias = torch.rand(E, device="cuda") * 0.1
    plan, idx, w, cnt, ps = run_route(x, bias, cfg_of(E, k, n_group=8, topk_group=4))
    tail = slice(T - 100, T)
    _, i2, w2, _, _ = run_route(x[tail].contiguous(), bias, cfg_of(E, k, n_group=8, topk_group=4))
    assert torch.equal(idx[tail], i2) and torch.equal(w[tail], w2) and int(cnt.long().sum()) == T * k
    dw = torch.randn(T, k, device="cuda")
    d = torch.empty_like(x)
    rg.moe_route_bwd(plan, T, x, idx, dw, d, dprob_sum=bias)
    d2 = torch.empty(100, E, device="cuda")
    rg.moe_route_bwd(plan, 100, x[tail].contiguous(), i2, dw[tail].contiguous(), d2, dprob_sum=bias)
    assert torch.equal(d[tail], d2)


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
def test_one_renormalised_expert_has_a_constant_weight(fn):
    """k = 1, or one expert left: the weight is scale itself and its gradient 0."""
    T, E = 300, 48
    x = torch.randn(T, E, device="cuda") * 3
    for k, keep in ((1, E), (3, 1)):
        y = x.clone()
        y[:, keep:] = -float("inf")
        plan, idx, w, _, _ = run_route(y, None, cfg_of(E, k, fn=fn, scale=2.5))
        assert bool((w[:, 0] == 2.5).all()) and bool((w[:, 1:] == 0).all())
        d = torch.full_like(y, float("nan"))
        rg.moe_route_bwd(plan, T, y, idx, torch.randn(T, k, device="cuda"), d)
        assert bool((d == 0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("n_inf", [1, 3, 4, 9, 40])
def test_a_bias_of_plus_infinity_forces_its_experts(fn, n_inf):
    """Fewer of them than slots, as many, more; equal keys, so the lowest ids win."""
    T, E = 70, 128
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, E, generator=g, device="cuda")
    bias = torch.rand(E, generator=g, device="cuda") * 0.1
    bias[torch.randperm(E, generator=g, device="cuda")[:n_inf]] = float("inf")
    for kw in (dict(), dict(n_group=8, topk_group=3), dict(n_group=8, topk_group=3, group_top=1, renorm=False)):
        check_route(x, bias, cfg_of(E, 4, fn=fn, **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [-5000.0, 300.0, 5000.0, 1e30])
def test_softmax_of_large_logits(shift):
    """The row's maximum is subtracted, not its rounded product with log2 e."""
    T, E = 300, 64
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(T, E, generator=g, device="cuda") + shift
    bias = torch.rand(E, generator=g, device="cuda") * 0.1
    for b in (None, bias):
        for kw in (dict(), dict(n_group=8, topk_group=3), dict(renorm=False)):
            check_route(x, b, cfg_of(E, 6, fn="softmax", **kw))


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("spread", [0.5, 3.0, 20.0])
def test_many_near_borders(fn, spread):
    """Biases that cancel the scores but for a few units of fp32's rounding: each row's border is close."""
    T, E = 500, 96
    g = torch.Generator(device="cuda").manual_seed(6)
    base = torch.randn(E, generator=g, device="cuda") * spread
    x = base[None, :] + (torch.randint(-2, 3, (T, E), generator=g, device="cuda") * 2.0 ** -22) * base.abs()[None, :]
    s = torch.sigmoid(base.double()) if fn == "sigmoid" else torch.softmax(base.double(), 0)
    bias = (0.5 - s).float()
    for kw in (dict(), dict(n_group=8, topk_group=4), dict(n_group=12, topk_group=5, group_top=1)):
        check_route(x, bias, cfg_of(E, 8, fn=fn, **kw))


FMAX = float(torch.finfo(torch.float32).max)


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("out", [-1e4, -1e9, 1e9, -FMAX, float("inf")])
@pytest.mark.parametrize("kw", [dict(), dict(n_group=8, topk_group=4)])
def test_a_few_far_biases_do_not_slow_every_row(fn, out, kw):
    """Experts held out or forced by a bias: the rows' borders are as far from
    fp32's error as before, so a call takes as long (within half of it)."""
    T, E = 16384, 256
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(T, E, generator=g, device="cuda") * 1.5
    bias = (torch.rand(E, generator=g, device="cuda") - 0.5) * 0.1
    far = bias.clone()
    far[[3, 77, 130, 131]] = out
    plan = rg.moe_route_plan_create(**cfg_of(E, 8, fn=fn, **kw))
    idx = torch.empty(T, 8, dtype=torch.int32, device="cuda")
    w = torch.empty(T, 8, device="cuda")

    def ms(b):
        best = float("inf")
        for _ in range(5):
            a, z = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(20):
                rg.moe_route(plan, T, x, b, idx, w)
            z.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(z) / 20)
        return best

    ms(bias)
    assert ms(far) <= 1.5 * ms(bias)


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size", [3.0, 1e4, 1e9, FMAX])
@pytest.mark.parametrize("sign", [-1, 1, 0])
def test_biases_far_outside_the_scores_range(fn, size, sign):
    """Experts held out (or forced) by a large finite bias, or some of both (sign
    0): few of them, and so many that held-out ones must be selected too."""
    T, E = 120, 96
    g = torch.Generator(device="cuda").manual_seed(31)
    x = torch.randn(T, E, generator=g, device="cuda") * 1.5
    x[::5] = torch.randint(-2, 3, (len(x[::5]), E), generator=g, device="cuda").float()
    for n_out in (2, 40, 92):
        bias = (torch.rand(E, generator=g, device="cuda") - 0.5) * 0.1
        out = torch.randperm(E, generator=g, device="cuda")[:n_out]
        how = torch.full((n_out,), float(sign or 1), device="cuda")
        if sign == 0:
            how[::2] = -1.0
        bias[out] = size * how
        for kw in (dict(), dict(n_group=8, topk_group=3), dict(n_group=8, topk_group=3, group_top=1),
                   dict(n_group=12, topk_group=5)):
            check_route(x, bias, cfg_of(E, 6, fn=fn, **kw))


@pytest.mark.gpu
def test_saturated_scores_tie_as_in_fp64():
    """The keys are those of fp64: 1 / (1 + e^-40) and 1 / (1 + e^-41) are both 1
    there, so with a bias the lower id wins; without one the logits decide."""
    x = torch.tensor([[40.0, 41.0, 0.0], [41.0, 40.0, 0.0], [-800.0, -790.0, -900.0]], device="cuda")
    for bias, want in ((torch.zeros(3, device="cuda"), [[0], [0], [0]]), (None, [[1], [0], [1]])):
        _, idx, _, _, _ = run_route(x, bias, cfg_of(3, 1))
        assert idx.tolist() == want


def rare_experts(T, E, seed):
    """Logits whose experts' popularity falls by up to e^-20."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, E, generator=g, device="cuda") * 1.5
    return x - torch.linspace(0.0, 20.0, E, device="cuda")[torch.randperm(E, generator=g, device="cuda")]


def score_error(xn, fn):
    """Relative error of a score or its share of the row: the exponential's
    2.22 d + 3 units of 2^-24 (d its argument), the row's sum and reciprocal 40."""
    d = (xn.max(1, keepdims=True) - xn).max() if fn == "softmax" else np.abs(xn).max()
    return (2.22 * d + 43) * U32


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E", [(600, 160), (5000, 96)])
def test_sums_and_weights_of_rare_experts(fn, T, E):
    """Element by element, relative to the element: all terms are positive.  The
    sums over the tokens add 64 units at most (runs of a few rows, 8 warps, up to
    15 partials in each of 32 warps); a weight adds exp's 2, |x - m| and 4."""
    x = rare_experts(T, E, 17)
    xn = x.double().cpu().numpy()
    plan, idx, w, _, ps = run_route(x, None, cfg_of(E, 9, fn=fn, renorm=False, scale=2.5))
    _, rw, _, rp = plain_route_rows(xn, None, 9, fn, 1, 1, 2, False, 2.5)
    err = score_error(xn, fn)
    assert np.all(np.abs(ps.double().cpu().numpy() - rp) <= (err + 64 * U32) * rp)
    assert np.all(np.abs(w.double().cpu().numpy() - rw) <= (err + 16 * U32) * rw)


@pytest.mark.gpu
@pytest.mark.parametrize("fn", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("sums", [True, False])
def test_gradients_of_rare_experts(fn, renorm, sums):
    """Element by element, relative to the terms that make the element up (which
    cancel): a score times (the gradient of it, and the row's mean of those); both
    scores' errors, 64 units for the mean's sum and the products."""
    T, E, k, scale = 600, 160, 9, 2.5
    x = rare_experts(T, E, 18)
    g = torch.Generator(device="cuda").manual_seed(19)
    plan, idx, w, _, _ = run_route(x, None, cfg_of(E, k, fn=fn, renorm=renorm, scale=scale))
    dw = torch.randn(T, k, generator=g, device="cuda")
    dps = torch.randn(E, generator=g, device="cuda") if sums else None
    d = torch.full((T, E), float("nan"), device="cuda")
    rg.moe_route_bwd(plan, T, x, idx, dw, d, dprob_sum=dps)
    xn, i, a = x.double().cpu().numpy(), idx.cpu().numpy().astype(np.int64), dw.double().cpu().numpy()
    s = scores(xn, fn)
    share = s / s.sum(1, keepdims=True)
    q = np.take_along_axis(s, i, 1)
    if renorm:
        q = q / q.sum(1, keepdims=True)
    # the formula itself (the other tests hold it against autograd and differences, whose own rounding is far above
    # these elements), and beside it its terms' sizes
    part = scale * q * (a - ((q * a).sum(1, keepdims=True) if renorm else 0.0))
    most = scale * q * (np.abs(a) + ((q * np.abs(a)).sum(1, keepdims=True) if renorm else 0.0))
    ref, size = np.zeros((T, E)), np.zeros((T, E))
    np.put_along_axis(ref, i, part, 1)
    np.put_along_axis(size, i, most, 1)
    if fn == "softmax" and not renorm:
        ref -= s * part.sum(1, keepdims=True)
        size += s * most.sum(1, keepdims=True)
    if sums:
        b = dps.double().cpu().numpy()
        ref += share * (b - (share * b).sum(1, keepdims=True))
        size += share * (np.abs(b) + (share * np.abs(b)).sum(1, keepdims=True))
    if fn == "sigmoid":
        ref /= 1.0 + np.exp(xn)
        size /= 1.0 + np.exp(xn)
    tol = (2 * score_error(xn, fn) + 64 * U32) * size
    assert np.all(np.abs(d.double().cpu().numpy() - ref) <= tol)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40, 3000])
def test_logits_written_just_before_the_call(T):
    """The launch is set up while the kernels before it run: it must see what they
    write, call after call into the same buffers."""
    E, k = 256, 8
    cfg = cfg_of(E, k, n_group=8, topk_group=4)
    g = torch.Generator(device="cuda").manual_seed(7)
    xs = torch.randn(8, T, E, generator=g, device="cuda")
    bias = torch.rand(E, generator=g, device="cuda") * 0.1
    dw = torch.randn(T, k, generator=g, device="cuda")
    plan = rg.moe_route_plan_create(**cfg)
    ws = torch.empty(rg.moe_route_workspace_bytes(plan, T), dtype=torch.uint8, device="cuda")

    def call(x, idx, w, cnt, ps, d):
        rg.moe_route(plan, T, x, bias, idx, w, cnt, ps, ws)
        rg.moe_route_bwd(plan, T, x, idx, dw, d, dprob_sum=bias)

    def outputs():
        return (torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda"),
                torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E, device="cuda"), torch.empty(T, E, device="cuda"))

    want = []
    for i in range(8):
        torch.cuda.synchronize()
        want.append(outputs())
        call(xs[i], *want[-1])
    torch.cuda.synchronize()
    x, out = torch.empty_like(xs[0]), outputs()
    for rep in range(40):
        i = rep % 8
        x.copy_(xs[i])
        call(x, *out)
        x.mul_(2.0)  # (after them: reads of this call must not see it)
        same = [torch.equal(a, b) for a, b in zip(out, want[i])] if rep >= 32 else None
        assert same is None or all(same), same
