"""moe_norm and moe_norm_bwd against their definition in 64 bits.

Tolerances are counted in roundings.  A stored value is off by at most half a
step of its type (eps / 2 relative; for fp16 also half a subnormal step, 2^-25).
In fp32 a value passes through some 12 roundings of 2^-24, the row's sums
through NV 8 = 32 serial additions, 5 + 5 of the tree and 32 of the warps', whose
error is relative to the sum of the terms' magnitudes: 80 x 2^-24 of the
magnitudes that enter an element bounds them together.  Sums over the rows add
at most T / 152 + 1 rows per CTA serially, then 19 + 8 partial sums of at most
1216 / 8 each: (T / 152 + 240) x 2^-24 of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

import routing_grouped_expert_gemm_gb300 as rg

pytestmark = pytest.mark.gpu

U = 2.0**-24
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HALF = {k: torch.finfo(t).eps / 2 for k, t in DT.items()}
TINY = {"fp32": 2.0**-149, "bf16": 2.0**-133, "fp16": 2.0**-25}


def rows(gen, T, D, dtype, pad=0, scale=1.0, shift=0.0):
    """[T, D] of a tensor whose rows are D + pad apart, NaN in between."""
    t = torch.full((T, D + pad), float("nan"), dtype=DT[dtype], device="cuda")
    t[:, :D] = torch.randn(T, D, generator=gen, device="cuda") * scale + shift
    return t[:, :D]


class Case:
    def __init__(self, T, D, kind="rms", stream="bf16", branch="bf16", param="fp32", post=True, pre=True, gate=None,
                 bias=False, x=True, o=True, pad=0, offset=0.0, x_scale=1.0, o_scale=1.0, shift=0.0, seed=0, weights=True):
        self.__dict__.update({k: v for k, v in locals().items() if k != "self"})
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.gen = g
        self.vx = rows(g, T, D, stream, pad, 2.0, shift) if x else None
        self.vo = rows(g, T, D, branch, pad, 1.0, shift) if o else None
        par = lambda m, s: (m + s * torch.randn(D, generator=g, device="cuda")).to(DT[param])  # noqa: E731
        self.params = {}
        for n, on in (("post", post), ("pre", pre)):
            if on and weights:
                self.params[n + "_weight"] = par(1.0 - offset, 0.2)
            if on and bias:
                self.params[n + "_bias"] = par(0.0, 0.2)
        if gate == "vector":
            self.params["gate"] = par(0.5, 0.5)
        elif gate == "rows":
            self.params["gate"] = rows(g, T, D, branch, pad, 0.7)
        self.plan = rg.moe_norm_plan_create(D, kind=kind, post=post, pre=pre, stream_dtype=stream, branch_dtype=branch,
                                            param_dtype=param, eps=1e-5, weight_offset=offset, x_scale=x_scale, o_scale=o_scale)

    def p64(self, name, d=None):
        v = self.params.get(name)
        if v is None:
            return torch.ones(self.D, dtype=torch.float64, device="cuda") if name.endswith("weight") or name == "gate" else 0.0
        return v.double() + (self.offset if name.endswith("weight") else 0.0)

    def norm(self, v, name, grad=False):
        m = v.mean(1, keepdim=True) if self.kind == "layer" else torch.zeros_like(v[:, :1])
        r = ((v - m).square().mean(1, keepdim=True) + float(np.float32(1e-5))) ** -0.5
        w, b = self.p64(name + "_weight"), self.p64(name + "_bias")
        # magnitudes that enter an element: (v - m) r w and, through m and r, the row's
        mag = ((v - m).abs() + (v.abs().mean(1, keepdim=True) if self.kind == "layer" else 0.0)) * r * w.abs() + (
            b.abs() if torch.is_tensor(b) else 0.0)
        return (v - m) * r * w + b, mag, m, r


def near(got, ref, mag, dtype, units=80.0, what=""):
    tol = HALF[dtype] * (ref.abs() + units * U * mag) + units * U * mag + TINY[dtype]
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float(((got.double() - ref).abs() / tol).max()):.2f}"


def guarded(T, D, dtype, pad):
    return torch.full((T, D + pad), 7.0, dtype=DT[dtype], device="cuda")


def forward(c, stats=True, y=True):
    out = {"y": guarded(c.T, c.D, c.stream, c.pad) if y else None, "h": guarded(c.T, c.D, c.branch, c.pad) if c.pre else None,
           "stats": torch.full((c.T, 4), float("nan"), device="cuda") if stats else None}
    v = {k: t[:, : c.D] if k != "stats" and t is not None else t for k, t in out.items()}
    rg.moe_norm(c.plan, c.T, c.params, x=c.vx, o=c.vo, **v)
    for k in ("y", "h"):
        if out[k] is not None:
            assert (out[k][:, c.D :] == 7.0).all(), k  # nothing written between the rows
    return v


SHAPES = [(1, 1), (1, 7168), (3, 8), (2, 31), (5, 33), (300, 64), (7, 256), (1000, 255), (613, 1001), (40, 2048), (33, 2056),
          (400, 4096), (9, 8192), (5, 8200), (3, 16384), (2, 16383), (700, 7168)]
VARIANTS = [
    dict(),
    dict(kind="layer", bias=True, gate="rows", stream="fp16", branch="fp16", param="fp16", pad=3, shift=0.5),
    dict(kind="layer", bias=True, gate="vector", stream="fp32", branch="fp32", x_scale=0.75, o_scale=-0.5, shift=3.0),
    dict(stream="fp32", branch="bf16", gate="vector", param="bf16", offset=1.0, pad=8),
    dict(stream="fp32", branch="fp16", gate="rows", param="bf16", o_scale=0.25, pad=16),
    dict(kind="layer", offset=1.0, shift=1.0),
]


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("v", range(len(VARIANTS)))
def test_forward(T, D, v):
    c = Case(T, D, seed=T + D, **VARIANTS[v])
    out = forward(c)
    z, mag, m1, r1 = c.norm(c.vo.double(), "post")
    b = c.o_scale * c.p64("gate") * z
    y = c.x_scale * c.vx.double() + b
    near(out["y"], y, (c.x_scale * c.vx.double()).abs() + (c.o_scale * c.p64("gate")).abs() * mag, c.stream, what="y")
    h, mag, m2, r2 = c.norm(out["y"].double(), "pre")
    near(out["h"], h, mag, c.branch, what="h")
    st = out["stats"].double()
    for i, (m, r) in ((0, (m1, r1)), (2, (m2, r2))):
        v64 = (c.vo if i == 0 else out["y"]).double()
        assert ((st[:, i : i + 1] - m).abs() <= 80 * U * v64.abs().mean(1, keepdim=True)).all()
        dev = 1 + v64.abs().mean(1, keepdim=True) * m.abs() * r * r  # what an error of m adds, relative
        assert ((st[:, i + 1 : i + 2] / r - 1).abs() <= 80 * U * dev).all()


@pytest.mark.parametrize("kw", [
    dict(post=False), dict(pre=False), dict(post=False, pre=False), dict(x=False), dict(post=False, o=False), dict(weights=False),
    dict(x=False, pre=False, gate="vector"), dict(post=False, gate="rows", pre=False, x_scale=0.5)])
@pytest.mark.parametrize("T,D", [(5, 1024), (3, 77)])
def test_forward_parts(T, D, kw):
    c = Case(T, D, seed=9, **kw)
    out = forward(c)
    y, mag = torch.zeros(T, D, dtype=torch.float64, device="cuda"), 0.0
    if c.vo is not None:
        z, zm = (c.norm(c.vo.double(), "post")[:2] if c.post else (c.vo.double(), c.vo.double().abs()))
        g = c.p64("gate")
        y, mag = y + c.o_scale * g * z, mag + g.abs() * zm
    if c.vx is not None:
        y, mag = y + c.x_scale * c.vx.double(), mag + c.vx.double().abs()
    near(out["y"], y, mag, c.stream, what="y")
    if c.pre:
        h, mag = c.norm(out["y"].double(), "pre")[:2]
        near(out["h"], h, mag, c.branch, what="h")
    else:
        assert (out["stats"][:, 2:] == 0).all()
    if not c.post:
        assert (out["stats"][:, :2] == 0).all()


@pytest.mark.parametrize("D", [2048, 1001])
def test_forward_fused_is_separate_in_place_and_without_y(D):
    """One call gives the bits of a post norm alone followed by a pre norm alone,
    of a call in place and of one that does not write y."""
    T = 300
    c = Case(T, D, gate="vector", seed=4)
    want = forward(c)
    a = rg.moe_norm_plan_create(D, post=True, pre=False, eps=1e-5)
    b = rg.moe_norm_plan_create(D, post=False, pre=True, eps=1e-5)
    y, h = torch.empty_like(want["y"]), torch.empty_like(want["h"])
    rg.moe_norm(a, T, {k: c.params[k] for k in ("post_weight", "gate")}, x=c.vx, o=c.vo, y=y)
    rg.moe_norm(b, T, {"pre_weight": c.params["pre_weight"]}, x=y, h=h)
    assert torch.equal(y, want["y"]) and torch.equal(h, want["h"])
    assert torch.equal(forward(c, y=False)["h"], want["h"])
    x, o = c.vx.clone(), c.vo.clone()
    rg.moe_norm(c.plan, T, c.params, x=x, o=o, y=x, h=o)
    assert torch.equal(x, want["y"]) and torch.equal(o, want["h"])
    for i in (0, 17, T - 1):  # a row by itself
        y1, h1 = torch.empty(1, D, dtype=torch.bfloat16, device="cuda"), torch.empty(1, D, dtype=torch.bfloat16, device="cuda")
        rg.moe_norm(c.plan, 1, c.params, x=c.vx[i : i + 1], o=c.vo[i : i + 1], y=y1, h=h1)
        assert torch.equal(y1[0], want["y"][i]) and torch.equal(h1[0], want["h"][i])


def test_forward_odd_rows():
    """Rows of zeros, of one value, large and tiny ones; an infinity or a NaN stays in its row."""
    D = 512
    c = Case(6, D, kind="layer", stream="fp32", branch="fp32", seed=1)
    for i, v in enumerate((0.0, 5.0, 1e15, 1e-30)):
        c.vx[i] = v * (1 + 0.25 * torch.randn(D, device="cuda") * (i > 1))
        c.vo[i] = c.vx[i]
    clean = forward(c)
    assert torch.isfinite(clean["h"]).all() and torch.isfinite(clean["y"]).all()
    z, mag = c.norm(c.vo.double(), "post")[:2]
    near(clean["y"], c.vx.double() + z, c.vx.double().abs() + mag, "fp32", what="y")
    c.vo[4, 3], c.vx[5, 500] = float("inf"), float("nan")
    got = forward(c)
    assert torch.equal(got["h"][:4], clean["h"][:4]) and torch.equal(got["y"][:4], clean["y"][:4])
    assert torch.isnan(got["h"][4:]).all() and torch.isnan(got["y"][4]).all() and int(torch.isnan(got["y"][5]).sum()) == 1


# ------------------------------------------------------------------ backward
def backward(c, want=None, dy=True, inplace=False):
    f = forward(c)
    g = c.gen
    v = {"y": f["y"] if c.pre else None, "o": c.vo, "dy": rows(g, c.T, c.D, c.stream, c.pad) if dy else None,
         "dh": rows(g, c.T, c.D, c.branch, c.pad) if c.pre else None}
    saved = {k: None if t is None else t.clone() for k, t in v.items()}
    buf = {"dx": guarded(c.T, c.D, c.stream, c.pad), "do": guarded(c.T, c.D, c.branch, c.pad)}
    out = {k: t[:, : c.D] for k, t in buf.items()}
    if inplace:
        out = {"dx": v["dy"], "do": v["dh"]}
    grads = {}
    for n, p in c.params.items():
        grads[n] = torch.full((c.D,), float("nan"), device="cuda")
        if n == "gate" and c.gate == "rows":
            grads[n] = guarded(c.T, c.D, c.branch, c.pad)[:, : c.D]
    ws = torch.full((rg.moe_norm_workspace_bytes(c.plan, c.T),), 0xFF, dtype=torch.uint8, device="cuda")
    rg.moe_norm_bwd(c.plan, c.T, c.params, f["stats"], grads, **v, **out, workspace=ws)
    if not inplace:
        assert (buf["dx"][:, c.D :] == 7.0).all() and (buf["do"][:, c.D :] == 7.0).all()
    return {**out, "grads": grads, "in": saved, "stats": f["stats"]}


def oracle_backward(c, v):
    """The formula in 64 bits, with the magnitudes that enter every output."""
    def back(d, dmag, x, name):
        w = c.p64(name + "_weight")
        m = x.mean(1, keepdim=True) if c.kind == "layer" else torch.zeros_like(x[:, :1])
        r = ((x - m).square().mean(1, keepdim=True) + float(np.float32(1e-5))) ** -0.5
        n = (x - m) * r
        nm = n.abs() + (x.abs().mean(1, keepdim=True) * r if c.kind == "layer" else 0.0)
        u, um = d * w, dmag * w.abs()
        cc, cm = (u * n).mean(1, keepdim=True), (um * nm).mean(1, keepdim=True)
        o, om = u - n * cc, um + nm * cm
        if c.kind == "layer":
            o, om = o - u.mean(1, keepdim=True), om + um.mean(1, keepdim=True)
        sums[name + "_weight"] = ((d * n).sum(0), (dmag * nm).sum(0))
        sums[name + "_bias"] = (d.sum(0), dmag.sum(0))
        return r * o, r * om, n * w + c.p64(name + "_bias"), nm * w.abs() + (c.p64(name + "_bias").abs() if name + "_bias" in c.params else 0.0)

    sums = {}
    d = torch.zeros(c.T, c.D, dtype=torch.float64, device="cuda") if v["dy"] is None else v["dy"].double()
    dm = d.abs()
    if c.pre:
        a, am, _, _ = back(v["dh"].double(), v["dh"].double().abs(), v["y"].double(), "pre")
        d, dm = d + a, dm + am
    ref = {"dx": (c.x_scale * d, abs(c.x_scale) * dm)}
    d, dm = c.o_scale * d, abs(c.o_scale) * dm
    g = c.p64("gate")
    dz, dzm = d * g, dm * g.abs()
    if c.post:
        do, dom, z, zm = back(dz, dzm, v["o"].double(), "post")
    else:
        do, dom, z, zm = dz, dzm, v["o"].double(), v["o"].double().abs()
    ref["do"] = (do, dom)
    sums["gate"] = (d * z, dm * zm) if c.gate == "rows" else ((d * z).sum(0), (dm * zm).sum(0))
    return ref, sums


BWD_SHAPES = [(1, 1), (1, 7168), (3, 8), (5, 33), (300, 64), (1000, 255), (613, 1001), (33, 2056), (400, 4096), (9, 8192),
              (5, 8200), (3, 16384), (2, 16383), (700, 7168), (4099, 128)]


@pytest.mark.parametrize("T,D", BWD_SHAPES)
@pytest.mark.parametrize("v", range(len(VARIANTS)))
def test_backward(T, D, v):
    c = Case(T, D, seed=3 * T + D, **VARIANTS[v])
    check_backward(c, backward(c))


@pytest.mark.parametrize("kw", [
    dict(post=False), dict(pre=False), dict(post=False, pre=False), dict(post=False, pre=False, gate="vector"), dict(weights=False),
    dict(kind="layer", bias=True, weights=False), dict(pre=False, gate="rows", kind="layer", bias=True)])
@pytest.mark.parametrize("T,D", [(5, 1024), (3, 77)])
def test_backward_parts(T, D, kw):
    c = Case(T, D, seed=5, **kw)
    check_backward(c, backward(c))


@pytest.mark.parametrize("T,D,kw", [(1001, 4104, dict()), (1000, 8192, dict(gate="vector")), (777, 6144, dict(stream="fp32", gate="vector")),
                                    (2001, 7168, dict(stream="fp16", branch="fp16", param="fp16", pad=8, x_scale=0.5)),
                                    (913, 7168, dict(kind="layer", bias=True, gate="vector")), (1500, 4096, dict(stream="fp32", branch="fp32"))])
def test_many_rows(T, D, kw):
    c = Case(T, D, seed=T, **kw)
    check_backward(c, backward(c))


# several rows a CTA: vectors that do not fill the threads, one at a time and in pairs; elements one by one
# with the parameters beside the ring, without them, and with a ring of one row
@pytest.mark.parametrize("T,D", [(1300, 2056), (1300, 5952), (5000, 40), (5000, 42), (700, 3001), (400, 5951), (400, 8191)])
@pytest.mark.parametrize("v", [0, 1, 2, 4])
def test_many_rows_of_each_form(T, D, v):
    test_forward(T, D, v)
    test_backward(T, D, v)


@pytest.mark.parametrize("T,D", [(400, 8191), (400, 5951), (3, 8193)])
def test_wide_rows_of_every_tensor(T, D):
    kw = dict(kind="layer", bias=True, gate="rows", stream="fp32", branch="fp32", x_scale=0.5)
    check_backward(c := Case(T, D, seed=5, **kw), backward(c))


def test_backward_without_dy():
    c = Case(70, 512, seed=6)
    check_backward(c, backward(c, dy=False))


def check_backward(c, out):
    ref, sums = oracle_backward(c, out["in"])
    near(out["dx"], *ref["dx"], c.stream, units=160, what="dx")
    near(out["do"], *ref["do"], c.branch, units=240, what="do")  # two norms deep
    for n, got in out["grads"].items():
        per_row = n == "gate" and c.gate == "rows"
        near(got, *sums[n], c.branch if per_row else "fp32", units=240 if per_row else 480 + c.T / 152, what=n)


@pytest.mark.parametrize("D", [1024, 1003])
def test_backward_in_place_and_twice(D):
    c = Case(333, D, gate="vector", seed=8)
    state = c.gen.get_state()
    a = backward(c)
    c.gen.set_state(state)
    b = backward(c, inplace=True)
    for n in ("dx", "do"):
        assert torch.equal(a[n], b[n])
    for n in a["grads"]:
        assert torch.equal(a["grads"][n], b["grads"][n])


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_gradients_are_the_differences(kind):
    """<grad, direction> against a central difference of the kernel's own forward in fp32.

    The loss L = <a, y> + <b, h> has values of about sqrt(2 T D) = 45 with errors of
    some 8 x 2^-24 per element, sqrt(2 T D) 8 2^-24 = 2e-5 in L; over 2 e = 2^-5 that is
    7e-4, and the third derivative adds e^2 = 2.4e-4 of derivatives of about 45: 1e-2.
    Directional derivatives are about 45 themselves: 0.1 absolute holds both with room
    and is a 400th of them."""
    T, D = 4, 256
    c = Case(T, D, kind=kind, stream="fp32", branch="fp32", gate="vector", bias=kind == "layer", seed=2)
    out = backward(c)
    a, b = out["in"]["dy"].double(), out["in"]["dh"].double()
    e = 2.0**-6
    leaves = {"x": (c.vx, out["dx"]), "o": (c.vo, out["do"]), **{n: (c.params[n], out["grads"][n]) for n in c.params}}
    for n, (t, grad) in leaves.items():
        d = torch.randn(t.shape, generator=c.gen, device="cuda")
        at = t.clone()
        L = []
        for s in (e, -e):
            t.copy_(at + s * d)
            f = forward(c)
            L.append(float((a * f["y"].double()).sum() + (b * f["h"].double()).sum()))
        t.copy_(at)
        assert abs((L[0] - L[1]) / (2 * e) - float((grad.double() * d.double()).sum())) <= 0.1, n


# ------------------------------------------------------------------ calls
def test_empty_batch():
    c = Case(3, 64, gate="vector")
    rg.moe_norm(c.plan, 0, c.params, x=c.vx, o=c.vo, y=c.vx, h=c.vo)
    grads = {n: torch.full((64,), float("nan"), device="cuda") for n in c.params}
    rg.moe_norm_bwd(c.plan, 0, c.params, None, grads)
    assert all((g == 0).all() for g in grads.values())


def test_rows_behind_the_batch_stay():
    c = Case(40, 128, seed=1)
    y, h = guarded(50, 128, "bf16", 0), guarded(50, 128, "bf16", 0)
    rg.moe_norm(c.plan, 40, c.params, x=c.vx, o=c.vo, y=y, h=h)
    assert (y[40:] == 7).all() and (h[40:] == 7).all() and not (y[:40] == 7).all(1).any()


def test_other_stream_and_graph():
    """On a stream of its own, captured and replayed on new inputs, beside another graph of the same plan."""
    c = Case(200, 1024, gate="vector", seed=3)
    want = backward(c)
    f = forward(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y, h, st = torch.empty_like(f["y"]), torch.empty_like(f["h"]), torch.empty_like(f["stats"])
    dx, do = torch.empty_like(want["dx"]), torch.empty_like(want["do"])
    grads = {n: torch.empty(1024, device="cuda") for n in c.params}
    dy, dh = want["in"]["dy"].clone(), want["in"]["dh"].clone()
    ws = torch.empty(rg.moe_norm_workspace_bytes(c.plan, c.T), dtype=torch.uint8, device="cuda")

    def both():
        rg.moe_norm(c.plan, c.T, c.params, x=c.vx, o=c.vo, y=y, h=h, stats=st)
        rg.moe_norm_bwd(c.plan, c.T, c.params, st, grads, o=c.vo, y=y, dy=dy, dh=dh, dx=dx, do=do, workspace=ws)

    with torch.cuda.stream(s):
        both()
    s.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g in graphs:
        with torch.cuda.graph(g, stream=s):
            both()
    x, o = c.vx.clone(), c.vo.clone()
    for g, scale in ((graphs[0], 0.5), (graphs[1], 1.0), (graphs[0], 1.0)):
        c.vx.copy_(x * scale)
        c.vo.copy_(o)
        for t in (y, h, dx, do, *grads.values()):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        ref = forward(c)
        assert torch.equal(y, ref["y"]) and torch.equal(h, ref["h"])
        if scale == 1.0:
            assert torch.equal(dx, want["dx"]) and torch.equal(do, want["do"])
            assert all(torch.equal(grads[n], want["grads"][n]) for n in grads)


def test_long_offsets():
    """Rows past 2^31 bytes and elements."""
    T, D, ld = 3, 64, 1 << 30
    big = torch.empty((T - 1) * ld + D, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(big, (T, D), (ld, 1))
    x.copy_(torch.randn(T, D, device="cuda"))
    plan = rg.moe_norm_plan_create(D, post=False)
    h, h2 = torch.empty(T, D, dtype=torch.bfloat16, device="cuda"), torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    rg.moe_norm(plan, T, {}, x=x, h=h)
    rg.moe_norm(plan, T, {}, x=x.clone(), h=h2)
    assert torch.equal(h, h2)


def test_refusals():
    c = Case(4, 64, gate="vector")
    y, h = torch.empty_like(c.vx), torch.empty_like(c.vo)
    st = torch.empty(4, 4, device="cuda")
    ws = torch.empty(rg.moe_norm_workspace_bytes(c.plan, 4), dtype=torch.uint8, device="cuda")
    w = c.params
    ok = dict(x=c.vx, o=c.vo, y=y, h=h)
    g = {"pre_weight": torch.empty(64, device="cuda")}
    bk = dict(o=c.vo, y=y, dy=y, dh=h, dx=torch.empty_like(y), do=torch.empty_like(h), workspace=ws)
    one = lambda t: t.data_ptr() + 1  # noqa: E731

    def refused(code, f, *a, **k):
        with pytest.raises(rg.MoEError) as e:
            f(*a, **k)
        assert e.value.code == code

    bad = rg.MOE_ERR_INVALID_ARG
    for k in (dict(h=None), dict(o=None), dict(x=None, o=None), dict(x=one(c.vx)), dict(stats=st.data_ptr() + 2), dict(y=one(y))):
        refused(bad, rg.moe_norm, c.plan, 4, w, **{**ok, **k})
    refused(bad, rg.moe_norm, c.plan, -1, w, **ok)
    refused(bad, rg.moe_norm, c.plan, 4, {**w, "pre_bias": w["pre_weight"]}, **ok)  # no biases with rms
    refused(bad, rg.moe_norm, c.plan, 4, {**w, "pre_weight": one(w["pre_weight"])}, **ok)
    refused(bad, rg.moe_norm, c.plan, 4, w, **{**ok, "x": torch.zeros(64, device="cuda", dtype=torch.bfloat16).expand(4, 64)})
    refused(bad, rg.moe_norm, c.plan, 4, w, **{**ok, "x": torch.zeros(4, 128, device="cuda", dtype=torch.bfloat16)[:, ::2]})
    post = rg.moe_norm_plan_create(64, pre=False)
    refused(bad, rg.moe_norm, post, 4, {}, x=c.vx, o=c.vo, y=y, h=h)  # no h without a pre norm
    refused(bad, rg.moe_norm, post, 4, {}, x=c.vx, o=c.vo)
    for k in (dict(y=None), dict(dh=None), dict(o=None), dict(dx=one(y)), dict(workspace=None), dict(workspace=one(ws), workspace_bytes=1 << 20)):
        refused(bad, rg.moe_norm_bwd, c.plan, 4, w, st, g, **{**bk, **k})
    refused(bad, rg.moe_norm_bwd, c.plan, 4, w, None, g, **bk)
    refused(bad, rg.moe_norm_bwd, c.plan, 4, w, st, {"pre_bias": st}, **bk)
    refused(bad, rg.moe_norm_bwd, c.plan, 4, {}, st, {"gate": st}, **bk)
    refused(rg.MOE_ERR_WORKSPACE_TOO_SMALL, rg.moe_norm_bwd, c.plan, 4, w, st, g, **bk, workspace_bytes=ws.numel() - 1)


# rows enough for the forms that keep two of them a CTA ahead and the weights in shared memory:
# whole vectors in all threads, not in all, elements with the parameters beside the rows and without
LARGE = [(700, 7168), (1300, 5952), (1000, 8192), (2500, 2048), (1300, 2053), (400, 5951), (400, 8191), (700, 8200)]


@pytest.mark.parametrize("T,D", LARGE)
@pytest.mark.parametrize("kw", [dict(), dict(stream="fp32", branch="bf16", x_scale=0.75), dict(kind="layer", bias=True, stream="fp16", branch="fp16"),
                                dict(gate="vector", o_scale=0.5), dict(kind="layer", bias=True, gate="rows")])
def test_forward_of_large_batches_is_that_of_rows(T, D, kw):
    """A batch's bits are those of its rows alone, of two calls, of a call in place and of one that does not write y."""
    c = Case(T, D, seed=T, **kw)
    want = forward(c)
    assert torch.equal(forward(c, y=False)["h"], want["h"])
    x, o = c.vx.clone(), c.vo.clone()
    rg.moe_norm(c.plan, T, c.params, x=x, o=o, y=x, h=o)
    assert torch.equal(x, want["y"]) and torch.equal(o, want["h"])
    some = torch.tensor([0, 1, T // 2, T - 2, T - 1], device="cuda")
    few = {n: torch.empty(5, *t.shape[1:], dtype=t.dtype, device="cuda") for n, t in want.items()}
    p = {**c.params, "gate": c.params["gate"][some].contiguous()} if c.gate == "rows" else c.params
    rg.moe_norm(c.plan, 5, p, x=c.vx[some].contiguous(), o=c.vo[some].contiguous(), **few)
    for n in want:
        assert torch.equal(few[n], want[n][some]), n
    same = dict(kind=c.kind, stream_dtype=c.stream, branch_dtype=c.branch, eps=1e-5)
    a = rg.moe_norm_plan_create(D, post=True, pre=False, x_scale=c.x_scale, o_scale=c.o_scale, **same)
    b = rg.moe_norm_plan_create(D, post=False, pre=True, **same)
    y, h = torch.empty_like(want["y"]), torch.empty_like(want["h"])
    rg.moe_norm(a, T, {n: v for n, v in c.params.items() if not n.startswith("pre")}, x=c.vx, o=c.vo, y=y)
    rg.moe_norm(b, T, {n: v for n, v in c.params.items() if n.startswith("pre")}, x=y, h=h)
    assert torch.equal(y, want["y"]) and torch.equal(h, want["h"])


@pytest.mark.parametrize("T,D", LARGE)
@pytest.mark.parametrize("kw", [dict(), dict(gate="vector", stream="fp32", branch="bf16"), dict(kind="layer", bias=True)])
def test_backward_of_large_batches_in_place(T, D, kw):
    c = Case(T, D, seed=T, **kw)
    state = c.gen.get_state()
    a = backward(c)
    c.gen.set_state(state)
    b = backward(c, inplace=True)
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["do"], b["do"])
    for n in a["grads"]:
        assert torch.equal(a["grads"][n], b["grads"][n]), n
