"""moe_decode and moe_decode_routed against the layer's definition in 64 bits.

Tolerance of out: h is rounded to bf16 (half a step, 2^-9 relative ... eps / 2 =
2^-8 at most) before the down projection and out once at the end (2^-8 at most);
sums of up to 8 K products are fp32.  An output element is a sum over I products
of h whose roundings are independent, so its error is at most 2^-8 of the sum of
magnitudes and about 2^-8 / sqrt(3) of the 2-norm; with the output's own rounding
the relative 2-norm stays below sqrt(2) 2^-8 / sqrt(3) = 3.2e-3, and MXFP8 plans,
whose oracle rounds x and h as the plan does, differ besides only where an fp32
sum lands on the other side of a code's border: 1e-4 of the elements, each by 2^-3
at most, 1.3e-3 more.  5e-3 covers both.  Weights g: logits of D products of fp32
sums, sqrt(D) 2^-24 of unit logits: 5e-5 relative, as for moe_fwd.
"""
import numpy as np
import pytest
import torch

import routing_grouped_expert_gemm_gb300 as rg

pytestmark = pytest.mark.gpu


def mx_round(v):
    """OCP MX: blocks of 32, scale 2^(floor(log2 max) - 8), E4M3 to nearest even."""
    b = v.unflatten(-1, (-1, 32))
    m = b.abs().amax(-1, keepdim=True)
    e = torch.where(m > 0, torch.frexp(m).exponent - 9, 0)
    q = torch.ldexp(b, -e).clamp(-448, 448).float().to(torch.float8_e4m3fn).to(v.dtype)
    return torch.where(m > 0, torch.ldexp(q, e), 0.0).flatten(-2)


class Layer:
    def __init__(self, T, D=256, I=128, E=16, k=4, I_s=128, score="sigmoid", precision="bf16", bias=False, seed=0, T_max=None, **kw):
        self.__dict__.update({n: v for n, v in locals().items() if n != "self"})
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.gen = g
        self.plan = rg.moe_plan_create(T_max or T, D, I, E, k, I_s, score_fn=score, precision=precision, **kw)
        rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g, device="cuda") * std).bfloat16()  # noqa: E731
        self.x = rnd(T, D)
        self.w = {"W_router": rnd(E, D, std=D**-0.5)}
        if bias:
            self.w["b_router"] = torch.randn(E, generator=g, device="cuda") * 0.3
        self.val = {}
        for n, r, c in (("W_up", I, D), ("W_gate", I, D), ("W_down", D, I)):
            w = rnd(E, r, c, std=c**-0.5)
            self.val[n] = w.double()
            if precision == "mxfp8":
                q = torch.empty(E * r, c, dtype=torch.uint8, device="cuda")
                s = torch.empty(rg.moe_mxfp8_scale_bytes(E * r, c), dtype=torch.uint8, device="cuda")
                rg.moe_quantize_mxfp8(self.plan, w, E * r, c, q, s)
                self.w[n], self.w[n + "_scale"] = q, s
                self.val[n] = mx_round(w.double())
            else:
                self.w[n] = w
        if I_s:
            for n, r, c in (("Ws_up", I_s, D), ("Ws_gate", I_s, D), ("Ws_down", D, I_s)):
                self.w[n] = rnd(r, c, std=c**-0.5)
        self.ws = torch.full((rg.moe_decode_workspace_bytes(self.plan, T),), 0xFF, dtype=torch.uint8, device="cuda")

    def logits(self):
        v = self.x.double() @ self.w["W_router"].double().T
        return v + self.w["b_router"].double() if self.bias else v

    def route(self):
        v = self.logits()
        idx = torch.sort(v, dim=1, descending=True, stable=True).indices[:, : self.k].sort(1).values
        got = torch.gather(v, 1, idx)
        s = torch.sigmoid(got) if self.score == "sigmoid" else torch.exp(got - got.amax(1, keepdim=True))
        return idx, s / s.sum(1, keepdim=True)

    def oracle(self, idx, w):
        rnd = mx_round if self.precision == "mxfp8" else (lambda v: v)
        x = self.x.double()
        xr = rnd(x)
        out = torch.zeros_like(x)
        for e in range(self.E):
            t, j = (idx == e).nonzero(as_tuple=True)
            if len(t):
                a = xr[t] @ self.val["W_gate"][e].T
                y = rnd(a * torch.sigmoid(a) * (xr[t] @ self.val["W_up"][e].T)) @ self.val["W_down"][e].T
                out.index_add_(0, t, y * w[t, j].double()[:, None])
        if self.I_s:
            a = x @ self.w["Ws_gate"].double().T
            out += (a * torch.sigmoid(a) * (x @ self.w["Ws_up"].double().T)) @ self.w["Ws_down"].double().T
        return out

    def run(self, T=None, **kw):
        T = self.T if T is None else T
        out = torch.full((T, self.D), float("nan"), dtype=torch.bfloat16, device="cuda")
        idx = torch.full((T, self.k), -7, dtype=torch.int32, device="cuda")
        w = torch.full((T, self.k), float("nan"), device="cuda")
        rg.moe_decode(self.plan, T, self.x, self.w, out, self.ws, topk_idx=idx, topk_w=w, **kw)
        return out, idx, w

    def run_routed(self, idx, w):
        out = torch.full((self.T, self.D), float("nan"), dtype=torch.bfloat16, device="cuda")
        rg.moe_decode_routed(self.plan, self.T, self.x, self.w, idx, w, out, self.ws)
        return out

    def status(self):
        return rg.moe_get_status(self.plan, self.ws)


def close(got, ref, tol=5e-3):
    assert torch.isfinite(got).all()
    d = got.double() - ref
    rel = float(d.norm() / ref.norm())
    assert rel <= tol, rel
    # no row or column stands out: an element's error is a sum of many small ones
    worst = float((d.abs() / (ref.abs() + ref.square().mean().sqrt())).max())
    assert worst <= 8 * tol, worst


def check(c):
    out, idx, w = c.run()
    assert c.status() == rg.MOE_STATUS_OK
    ri, rw = c.route()
    assert torch.equal(idx.long(), ri)
    assert ((w.double() - rw).abs() <= 5e-5 * rw).all()
    close(out, c.oracle(ri, rw))


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
@pytest.mark.parametrize("T", [1, 2, 3, 5, 8, 15, 16, 17, 31, 33, 47, 48, 63, 64])
def test_tokens(T, precision):
    check(Layer(T, D=512, I=256, E=24, k=4, I_s=256, precision=precision, seed=T))


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
@pytest.mark.parametrize("T,D,I,E,k,I_s,score,bias", [
    (1, 256, 128, 1, 1, 0, "sigmoid", False), (7, 256, 128, 4, 4, 128, "softmax", True), (64, 256, 128, 16, 16, 0, "sigmoid", True),
    (13, 2816, 1408, 60, 4, 0, "softmax", True), (1, 7168, 384, 32, 8, 640, "sigmoid", False), (64, 768, 640, 512, 10, 128, "softmax", False),
    (9, 1024, 128, 257, 3, 1152, "sigmoid", True), (33, 8448, 256, 8, 2, 128, "softmax", False), (64, 512, 256, 2, 1, 0, "sigmoid", False),
    (5, 16384, 128, 6, 2, 0, "sigmoid", True)])
def test_shapes(T, D, I, E, k, I_s, score, bias, precision):
    check(Layer(T, D=D, I=I, E=E, k=k, I_s=I_s, score=score, precision=precision, bias=bias, seed=T + E))


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
@pytest.mark.parametrize("T,empty", [(1, 0.5), (40, 0.3), (64, 0.9), (6, 1.0)])
@pytest.mark.parametrize("I_s", [0, 256])
def test_given_routing(T, empty, I_s, precision):
    c = Layer(T, D=512, I=256, E=32, k=6, I_s=I_s, precision=precision, seed=T)
    idx = torch.rand(T, 32, generator=c.gen, device="cuda").argsort(1)[:, :6]
    w = torch.randn(T, 6, generator=c.gen, device="cuda")
    gone = torch.rand(T, 6, generator=c.gen, device="cuda") < empty
    idx = torch.where(gone, -1, idx).to(torch.int32)
    w = torch.where(gone, float("nan"), w)  # the weight of an empty slot is not looked at
    out = c.run_routed(idx, w)
    assert c.status() == rg.MOE_STATUS_OK
    ref = c.oracle(idx.long(), torch.where(gone, 0.0, w))
    if float(ref.norm()) == 0.0:
        assert (out == 0).all()
    else:
        close(out, ref)


def test_given_routing_of_the_own_router():
    """On the routing that the built-in router made: the same bits."""
    for precision in ("bf16", "mxfp8"):
        c = Layer(21, D=512, I=256, E=32, k=6, I_s=256, precision=precision, seed=3)
        out, idx, w = c.run()
        assert torch.equal(c.run_routed(idx, w), out)


def test_bad_routing_is_reported():
    c = Layer(4, E=8, k=3, seed=1)
    good = torch.tensor([[0, 1, 2], [3, -1, 5], [7, 6, 5], [2, 4, 0]], dtype=torch.int32, device="cuda")
    w = torch.rand(4, 3, generator=c.gen, device="cuda")
    for at, bad in (((0, 1), 8), ((1, 0), -2), ((2, 2), 1 << 30), ((3, 2), 2), ((0, 0), 1)):
        idx = good.clone()
        idx[at] = bad
        out = c.run_routed(idx, w)
        assert c.status() == rg.MOE_STATUS_SCHEDULE_INVALID
        ref = idx.clone()
        ref[at] = -1
        if at == (0, 0):  # the later of two slots is the one left out
            ref[0] = torch.tensor([1, -1, 2])
        close(out, c.oracle(ref.long(), w))
    c.run_routed(good, w)
    assert c.status() == rg.MOE_STATUS_OK


def test_against_the_layer():
    for precision in ("bf16", "mxfp8"):
        c = Layer(50, D=1024, I=512, E=64, k=8, I_s=512, precision=precision, seed=5)
        out, idx, w = c.run()
        ref, ri = torch.empty_like(out), torch.empty_like(idx)
        ws = torch.empty(rg.moe_workspace_bytes(c.plan, 50), dtype=torch.uint8, device="cuda")
        rg.moe_fwd(c.plan, 50, c.x, c.w, ref, ws, topk_idx=ri)
        assert torch.equal(idx, ri)
        close(out, ref.double(), 8e-3)


def test_repeats_are_the_same_bits():
    for T, precision in ((1, "bf16"), (64, "bf16"), (30, "mxfp8")):
        c = Layer(T, D=2048, I=512, E=64, k=8, I_s=512, precision=precision, seed=T)
        want = c.run()
        for _ in range(20):
            c.ws.fill_(0xFF)
            got = c.run()
            assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_router_ties_and_near_ties():
    """Equal experts: the lower id.  Logits closer than fp32 resolves: by their exact values."""
    c = Layer(16, D=512, E=32, k=4, seed=2)
    W = c.w["W_router"]
    W[20] = W[3]
    W[7] = W[9]
    check(c)
    W[:] = W[:1]  # all the same
    out, idx, w = c.run()
    assert torch.equal(idx, torch.arange(4, dtype=torch.int32, device="cuda").expand(16, 4))
    c.x.zero_()
    out, idx, w = c.run()
    assert torch.equal(idx, torch.arange(4, dtype=torch.int32, device="cuda").expand(16, 4)) and (w == 0.25).all()
    # large parts that cancel: logits of about 40 beside magnitudes of 2e6, where fp32 sums are off by up to 5
    c = Layer(8, D=1024, E=16, k=3, seed=4)
    c.x[:, ::2] = (torch.randn(8, 512, generator=c.gen, device="cuda") * 300).bfloat16()
    c.x[:, 1::2] = -c.x[:, ::2]
    base = (torch.randn(16, 512, generator=c.gen, device="cuda") * 16).bfloat16()
    c.w["W_router"][:, ::2] = base
    c.w["W_router"][:, 1::2] = base
    c.w["W_router"][:, 1] += (torch.randn(16, generator=c.gen, device="cuda") * 2.0**-3).bfloat16()
    assert torch.equal(c.run()[1].long(), c.route()[0])


def test_router_bias_that_holds_out_or_forces():
    c = Layer(12, D=512, E=32, k=4, bias=True, seed=6)
    c.w["b_router"][5] = float("-inf")
    c.w["b_router"][6] = -1e9
    c.w["b_router"][11] = 1e9
    out, idx, w = c.run()
    assert (idx == 11).any(1).all() and not ((idx == 5) | (idx == 6)).any()
    ri, _ = c.route()
    assert torch.equal(idx.long(), ri)


def test_bad_tokens_stay_alone():
    """A token of NaN or infinities spoils its own row only."""
    c = Layer(20, D=512, I=256, E=8, k=3, I_s=256, seed=7)
    want, idx, _ = c.run()
    c.x[4, 17] = float("nan")
    c.x[9] = float("inf")
    out, idx2, _ = c.run()
    assert torch.isnan(out[4]).all() and torch.isnan(out[9]).all()
    assert (idx2 >= 0).all() and (idx2 < 8).all() and (idx2[:, 1:] > idx2[:, :-1]).all()
    keep = [t for t in range(20) if t not in (4, 9)]
    assert torch.equal(idx2[keep], idx[keep])
    close(out[keep], want[keep].double())


def test_rows_behind_the_batch_and_guards():
    c = Layer(40, D=512, I=256, seed=8, T_max=100)
    full, _, _ = c.run()
    for T in (39, 17, 1):
        ws = torch.full((rg.moe_decode_workspace_bytes(c.plan, T) + 256,), 0x5A, dtype=torch.uint8, device="cuda")
        out = torch.full((40, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        rg.moe_decode(c.plan, T, c.x, c.w, out, ws[:-256])
        assert (out[T:] == 7).all() and (ws[-256:] == 0x5A).all()
        close(out[:T], full[:T].double())
    rg.moe_decode(c.plan, 0, c.x, c.w, full, c.ws)
    assert rg.moe_decode_workspace_bytes(c.plan, 65) == 0 and rg.moe_decode_workspace_bytes(c.plan, 64) > 0


def test_without_the_shared_expert_in_the_call():
    c = Layer(9, D=512, I=256, I_s=256, seed=9)
    c.w = {n: v for n, v in c.w.items() if not n.startswith("Ws")}
    c.I_s = 0
    check(c)


def test_streams_graphs_and_two_at_once():
    a, b = Layer(3, D=1024, I=512, E=32, seed=10), Layer(50, D=512, I=256, E=64, seed=11)
    want = [a.run()[0], b.run()[0]]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty_like(o) for o in want]
    torch.cuda.synchronize()
    for _ in range(30):  # two streams, calls in turn
        for c, o, s in zip((a, b), outs, streams):
            with torch.cuda.stream(s):
                rg.moe_decode(c.plan, c.T, c.x, c.w, o, c.ws)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(outs, want))
    assert a.status() == b.status() == rg.MOE_STATUS_OK
    graphs = []
    for c, o in zip((a, b), outs):  # two graphs, one workspace each; a third on the first's workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            rg.moe_decode(c.plan, c.T, c.x, c.w, o, c.ws)
        graphs.append(g)
    g = torch.cuda.CUDAGraph()
    again = torch.empty_like(outs[0])
    with torch.cuda.graph(g):
        rg.moe_decode(a.plan, a.T, a.x, a.w, again, a.ws)
    for o in (*outs, again):
        o.zero_()
    for _ in range(5):
        for r in (*graphs, g):
            r.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and torch.equal(again, want[0])
    a.x.copy_(a.x.flip(1).clone())
    graphs[0].replay()
    new = outs[0].clone()
    assert torch.equal(new, a.run()[0]) and not torch.equal(new, want[0])


def test_refusals():
    c = Layer(4, T_max=80)
    out = torch.empty(4, 256, dtype=torch.bfloat16, device="cuda")
    idx, w = torch.zeros(4, 4, dtype=torch.int32, device="cuda"), torch.zeros(4, 4, device="cuda")

    def refused(code, f, *a, **k):
        with pytest.raises(rg.MoEError) as e:
            f(*a, **k)
        assert e.value.code == code

    bad = rg.MOE_ERR_INVALID_ARG
    for T in (-1, 65, 81):
        refused(bad, rg.moe_decode, c.plan, T, c.x, c.w, out, c.ws)
        refused(bad, rg.moe_decode_routed, c.plan, T, c.x, c.w, idx, w, out, c.ws)
    for n in ("W_router", "W_up", "W_gate", "W_down", "Ws_up"):
        refused(bad, rg.moe_decode, c.plan, 4, c.x, {k: v for k, v in c.w.items() if k != n}, out, c.ws)
    for args in ((None, out), (c.x, None), (c.x.data_ptr() + 2, out), (c.x, out.data_ptr() + 8)):
        refused(bad, rg.moe_decode, c.plan, 4, args[0], c.w, args[1], c.ws)
    refused(bad, rg.moe_decode, c.plan, 4, c.x, c.w, out, c.ws.data_ptr() + 16, workspace_bytes=1 << 30)
    refused(bad, rg.moe_decode, c.plan, 4, c.x, c.w, out, c.ws, topk_w=w.data_ptr() + 1)
    refused(rg.MOE_ERR_WORKSPACE_TOO_SMALL, rg.moe_decode, c.plan, 4, c.x, c.w, out, c.ws, workspace_bytes=c.ws.numel() - 1)
    refused(bad, rg.moe_decode_routed, c.plan, 4, c.x, c.w, None, w, out, c.ws)
    refused(bad, rg.moe_decode_routed, c.plan, 4, c.x, c.w, idx, None, out, c.ws)
    refused(bad, rg.moe_decode_routed, c.plan, 4, c.x, c.w, idx, w.data_ptr() + 2, out, c.ws)
    m = Layer(4, precision="mxfp8")
    refused(bad, rg.moe_decode, m.plan, 4, m.x, {k: v for k, v in m.w.items() if k != "W_up_scale"}, out, m.ws)


SIZES = [dict(D=4096, I=1536, E=128, k=8, I_s=0), dict(D=1024, I=1024, E=17, k=1, I_s=1024), dict(D=768, I=640, E=20, k=6, I_s=256),
         dict(D=7168, I=2048, E=256, k=8, I_s=2048)]


@pytest.mark.parametrize("precision", ["bf16", "mxfp8"])
@pytest.mark.parametrize("shape", range(len(SIZES)))
def test_workspace_sizes_never_fall(shape, precision):
    plan = rg.moe_plan_create(64, precision=precision, **SIZES[shape])
    sizes = [rg.moe_decode_workspace_bytes(plan, T) for T in range(1, 65)]
    assert sizes == sorted(sizes) and sizes[0] > 0


@pytest.mark.parametrize("most", [48, 64])
@pytest.mark.parametrize("shape,precision", [(0, "bf16"), (1, "bf16"), (2, "bf16"), (2, "mxfp8")])
def test_one_workspace_for_every_batch(shape, precision, most):
    """A server's workspace, made once for its largest batch."""
    c = Layer(most, precision=precision, seed=shape, **SIZES[shape])
    idx, w = c.route()
    ref = c.oracle(idx, w)
    c.ws = torch.cat([c.ws, torch.full((256,), 0x5A, dtype=torch.uint8, device="cuda")])
    for T in range(1, most + 1):
        out, got, _ = c.run(T, workspace_bytes=c.ws.numel() - 256)
        assert torch.equal(got.long(), idx[:T])
        close(out, ref[:T])
    assert (c.ws[-256:] == 0x5A).all()


def cancelling(seed, T=64, D=2048, E=16, k=4, **kw):
    """Logits of about 1 that are what is left of parts of up to 10^5: columns in pairs of opposite
    tokens and equal weights, at random places, so that a pair cancels neither in a product nor in a
    chunk; one pair has weights that differ.  Every product is exact and so, nearly, are fp64 sums."""
    c = Layer(T, D=D, E=E, k=k, seed=seed, **kw)
    at = torch.randperm(D, generator=c.gen, device="cuda")
    a = (torch.randn(T, D // 2, generator=c.gen, device="cuda") * 300).bfloat16()
    base = (torch.randn(E, D // 2, generator=c.gen, device="cuda") * 16).bfloat16()
    base[:, 0] = (torch.randn(E, generator=c.gen, device="cuda") * 2.0**-8).bfloat16()
    c.x[:, at[0::2]], c.x[:, at[1::2]] = a, -a
    c.w["W_router"][:, at[0::2]] = c.w["W_router"][:, at[1::2]] = base
    c.w["W_router"][:, at[0]] = (torch.randn(E, generator=c.gen, device="cuda") * 2.0**-8).bfloat16()
    return c


@pytest.mark.parametrize("T", [3, 64])
@pytest.mark.parametrize("of_x,of_w", [(0, 0), (-60, -60), (-80, 0), (-90, 0), (0, -95), (-90, -30), (-75, -75)])
def test_selection_of_any_magnitude(T, of_x, of_w):
    """Powers of two in front of the tokens or the router change no order: not where squares of the
    elements, or even their products (the last two cases), are below what fp32 holds."""
    c = cancelling(T, T=T)
    want = c.route()[0]
    c.x *= 2.0**of_x
    c.w["W_router"] *= 2.0**of_w
    ri, _ = c.route()
    assert torch.equal(ri, want)  # (the scaling is exact)
    assert torch.equal(c.run()[1].long(), ri)


def test_tokens_of_zeros_among_small_ones():
    """A token of zeros: a tie of all experts.  One element that is not zero decides."""
    c = Layer(8, D=512, E=40, k=3, seed=12)
    c.x[1], c.x[3], c.x[6] = 0.0, -0.0, 0.0
    c.x[6, 400] = 2.0**-120
    c.x[5] *= 2.0**-110
    c.w["W_router"][7] = 0.0
    out, idx, w = c.run()
    assert torch.equal(idx.long(), c.route()[0])
    assert torch.equal(idx[[1, 3]], torch.arange(3, dtype=torch.int32, device="cuda").expand(2, 3))


@pytest.mark.parametrize("T", [3, 64])
@pytest.mark.parametrize("score,bias", [("softmax", False), ("sigmoid", False), ("softmax", True)])
def test_weights_where_parts_cancel(T, score, bias):
    """The logits that decide are the weights', too: fp64 sums rounded once, off by 2^-24 of at most 10."""
    c = cancelling(T + 1, T=T, score=score, bias=bias)
    if bias:  # held out and forced by a large bias, as any others are
        c.w["b_router"][2], c.w["b_router"][9] = -1e9, 3.0
    check(c)


def test_weights_of_few_experts_all_in():
    """Nothing to select: weights alone."""
    c = cancelling(5, T=6, E=4, k=4, score="softmax")
    check(c)
