"""Workloads of the operators of a block around the expert layer: inputs, the
operators' plain form in elementary torch operations, the framework's calls, and
the operators' definition in 64 bits.

decode     the whole expert layer for a few tokens: router, top-k, the selected
           experts and the shared expert, the weighted sum; or on a given
           routing; bf16 or MXFP8 (E4M3 codes, one power-of-two scale per 32)
           routed experts
norm       a block's output norm, gate and scaled residual and the next block's
           input norm:  z = N(o), y = a x + b g z, h = N(y)
norm_bwd   its gradients: of the stream, the block's output, the norms' weights
           and biases and the gate
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


def _decode(name, T, D, I, E, k, I_s, score, precision, bias=False, empty=0.0, given=False):
    c = dict(op="decode", T=T, D=D, I=I, E=E, k=k, I_s=I_s, score=score, precision=precision, bias=bias, empty=empty,
             given=given)
    return dict(name=name, **c) if name else c


def _norm(op, name, T, D, kind, stream, branch, param, post=True, pre=True, gate="none", biases=False, x_scale=1.0,
          o_scale=1.0, offset=0.0, pad=0):
    c = dict(op=op, T=T, D=D, kind=kind, stream=stream, branch=branch, param=param, post=post, pre=pre, gate=gate,
             biases=biases, x_scale=x_scale, o_scale=o_scale, offset=offset, pad=pad)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one token through a small layer: latency alone counts
        _decode("decode_small_1", 1, 512, 256, 16, 4, 256, "sigmoid", "bf16"),
        # one token of a decode step through the 256-expert layer
        _decode("decode_1", 1, 7168, 2048, 256, 8, 2048, "sigmoid", "bf16"),
        # a few sequences, odd sizes, softmax router with a bias, no shared expert
        _decode("decode_odd_13", 13, 2816, 1408, 60, 4, 0, "softmax", "bf16", bias=True),
        # a batch of decode steps whose routing another router made, some slots empty
        _decode("decode_given_32", 32, 4096, 1536, 128, 8, 0, "softmax", "bf16", empty=0.1, given=True),
        # a few sequences on MXFP8 experts
        _decode("decode_mxfp8_8", 8, 7168, 2048, 256, 8, 2048, "sigmoid", "mxfp8"),
        # the largest decode batch: most of the 256 experts' weights are read
        _decode("decode_64", 64, 7168, 2048, 256, 8, 2048, "sigmoid", "bf16"),
        # between two blocks of a decode step, one token
        _norm("norm", "norm_1", 1, 7168, "rms", "bf16", "bf16", "bf16"),
        # between two blocks of a training step
        _norm("norm", "norm_16384", 16384, 7168, "rms", "bf16", "bf16", "fp32", o_scale=0.5),
        # layer norms with biases, a gate per token, odd sizes, padded rows
        _norm("norm", "norm_odd", 1003, 2053, "layer", "fp16", "fp16", "fp16", gate="rows", biases=True, pad=3),
        # gradients of the training step's
        _norm("norm_bwd", "norm_bwd_16384", 16384, 7168, "rms", "bf16", "bf16", "fp32", o_scale=0.5),
        # a stream in fp32 beside a branch in bf16, a learned gate per channel
        _norm("norm_bwd", "norm_bwd_mixed", 2048, 4096, "rms", "fp32", "bf16", "fp32", gate="vector", offset=1.0),
        # layer norms, odd sizes, fp32
        _norm("norm_bwd", "norm_bwd_odd", 777, 1001, "layer", "fp32", "fp32", "fp32", gate="vector", biases=True, x_scale=0.75),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "norm", "norm_bwd"])
    if op == "decode":
        T = _log_int(rng, 1, 64)
        D = 256 * _log_int(rng, 1, 28)
        I = 128 * _log_int(rng, 1, 16)
        E = _log_int(rng, 4, max(4, min(256, int(3.7e9 / (D * I)))))
        k = rng.randint(1, min(10, E))
        I_s = rng.choice([0, I, 128 * _log_int(rng, 1, 16)])
        given = rng.random() < 0.3
        return _decode(None, T, D, I, E, k, I_s, rng.choice(["sigmoid", "softmax"]), rng.choice(["bf16", "bf16", "mxfp8"]),
                       rng.random() < 0.4, rng.choice([0.0, 0.2]) if given else 0.0, given)
    stream = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    branch = rng.choice(["bf16", "fp16", "fp32"]) if stream == "fp32" else stream
    kind = rng.choice(["rms", "rms", "layer"])
    D = rng.choice([8 * _log_int(rng, 4, 1024), _log_int(rng, 32, 8192)])
    T = _log_int(rng, 1, max(1, min(32768, int(5.0e7 / D))))
    post, pre = rng.choice([(True, True), (True, True), (False, True), (True, False)])
    return _norm(op, None, T, D, kind, stream, branch, rng.choice(["fp32", branch]), post, pre,
                 rng.choice(["none", "none", "vector", "rows"]), kind == "layer" and rng.random() < 0.7,
                 rng.choice([1.0, 0.75]), rng.choice([1.0, 0.25]), rng.choice([0.0, 1.0]), rng.choice([0, 0, 5, 8]))


def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _decode_inputs(c, seed, device="cuda"):
    """Weights of unit gain, tokens of unit size; MXFP8 weights as codes and
    exponents (a row-major E8M0 byte per 32 codes)."""
    g = _gen(seed, device)
    T, D, I, E, k, I_s = c["T"], c["D"], c["I"], c["E"], c["k"], c["I_s"]

    def normal(*shape, std):
        return torch.randn(*shape, generator=g, device=device, dtype=torch.bfloat16).mul_(std)

    s = {"x": normal(T, D, std=1.0), "W_router": None, "b_router": None}
    for name, rows, cols in (("W_up", I, D), ("W_gate", I, D), ("W_down", D, I)):
        if c["precision"] == "bf16":
            s[name] = normal(E, rows, cols, std=cols**-0.5)
        else:
            s[name] = normal(E, rows, cols, std=96.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
            e = torch.randint(-1, 2, (E, rows, cols // 32), generator=g, device=device, dtype=torch.int32)
            s[name + "_e8m0"] = (e + (127 - 7 - round(0.5 * math.log2(cols)))).to(torch.uint8)
    for name, rows, cols in (("Ws_up", I_s, D), ("Ws_gate", I_s, D), ("Ws_down", D, I_s)):
        s[name] = normal(rows, cols, std=cols**-0.5) if I_s else None
    if c["given"]:
        order = torch.rand(T, E, generator=g, device=device).argsort(1)[:, :k].sort(1).values
        w = torch.rand(T, k, generator=g, device=device) + 0.1
        gone = torch.rand(T, k, generator=g, device=device) < c["empty"]
        s["topk_idx"] = torch.where(gone, -1, order).to(torch.int32)
        s["topk_w"] = torch.where(gone, 0.0, w / w.sum(1, keepdim=True))
    else:
        s["W_router"] = normal(E, D, std=D**-0.5)
        if c["bias"]:
            s["b_router"] = torch.randn(E, generator=g, device=device) * 0.3
    return s


def _norm_inputs(c, seed, device="cuda"):
    """A residual stream whose channels differ in size, a block's output, norm
    weights near one; rows `pad` elements further apart than D."""
    g = _gen(seed, device)
    T, D, pad = c["T"], c["D"], c["pad"]
    loud = torch.exp(0.5 * torch.randn(D, generator=g, device=device))

    def rows(dtype, by=1.0):
        v = torch.randn(T, D, generator=g, device=device)
        t = torch.zeros(T, D + pad, dtype=DTYPES[dtype], device=device)
        t[:, :D] = v.mul_(by)
        return t[:, :D]

    def param(mean, std):
        return (mean + std * torch.randn(D, generator=g, device=device)).to(DTYPES[c["param"]])

    s = {"o": rows(c["branch"], loud.flip(0)), "gate": None}
    for n, on in (("post", c["post"]), ("pre", c["pre"])):
        s[n + "_weight"] = param(1.0 - c["offset"], 0.1) if on else None
        s[n + "_bias"] = param(0.0, 0.1) if on and c["biases"] else None
    if c["gate"] == "vector":
        s["gate"] = param(0.5, 0.2)
    elif c["gate"] == "rows":
        s["gate"] = rows(c["branch"], 0.5)
    if c["op"] == "norm":
        s["x"] = rows(c["stream"], loud * 2.0)
    else:
        s["y"] = rows(c["stream"], loud * 2.0) if c["pre"] else None
        s["dy"] = rows(c["stream"])
        s["dh"] = rows(c["branch"]) if c["pre"] else None
        # what a forward saved per row: mean and reciprocal deviation of o and of y
        st = torch.zeros(T, 4, device=device, dtype=torch.float64)
        for at, v in ((0, s["o"] if c["post"] else None), (2, s["y"])):
            if v is not None:
                v = v.double()
                m = v.mean(1, keepdim=True) if c["kind"] == "layer" else torch.zeros_like(v[:, :1])
                st[:, at : at + 1] = m
                st[:, at + 1 : at + 2] = (((v - m) ** 2).mean(1, keepdim=True) + EPS) ** -0.5
        s["stats"] = st.float()
    return s


def prepare(case, seed):
    c = case
    s = _decode_inputs(c, seed) if c["op"] == "decode" else _norm_inputs(c, seed)
    s["case"] = c
    if own:  # the handle, outputs and workspace that a program keeps
        import routing_grouped_expert_gemm_gb300 as rg
        s["rg"] = rg
        dev = dict(device="cuda")
        T, D = c["T"], c["D"]
        if c["op"] == "decode":
            k = c["k"]
            s["plan"] = rg.moe_plan_create(T, D, c["I"], c["E"], k, c["I_s"], score_fn=c["score"], precision=c["precision"])
            names = ("W_router", "b_router", "W_up", "W_gate", "W_down", "Ws_up", "Ws_gate", "Ws_down")
            s["weights"] = {n: s[n] for n in names if s[n] is not None}
            if c["precision"] == "mxfp8":  # scales in the library's 512-byte blocks of 128 rows x 4 scales
                for n in ("W_up", "W_gate", "W_down"):
                    E, rows, cols = s[n].shape
                    b = s[n + "_e8m0"].view(E * rows // 128, 4, 32, cols // 128, 4)
                    s["weights"][n + "_scale"] = b.permute(0, 3, 2, 1, 4).contiguous()
            s["out"] = torch.empty(T, D, dtype=torch.bfloat16, **dev)
            if not c["given"]:
                s["topk_idx"] = torch.empty(T, k, dtype=torch.int32, **dev)
                s["topk_w"] = torch.empty(T, k, dtype=torch.float32, **dev)
            s["ws"] = torch.empty(rg.moe_decode_workspace_bytes(s["plan"], T), dtype=torch.uint8, **dev)
        else:
            s["plan"] = rg.moe_norm_plan_create(D, kind=c["kind"], post=c["post"], pre=c["pre"], stream_dtype=c["stream"],
                                                branch_dtype=c["branch"], param_dtype=c["param"], eps=EPS,
                                                weight_offset=c["offset"], x_scale=c["x_scale"], o_scale=c["o_scale"])
            names = ("post_weight", "post_bias", "pre_weight", "pre_bias", "gate")
            s["params"] = {n: s[n] for n in names if s[n] is not None}
            stream, branch = DTYPES[c["stream"]], DTYPES[c["branch"]]
            if c["op"] == "norm":
                s["y"] = torch.empty(T, D, dtype=stream, **dev)
                s["h"] = torch.empty(T, D, dtype=branch, **dev) if c["pre"] else None
                s["stats"] = torch.empty(T, 4, dtype=torch.float32, **dev)
            else:
                s["dx"] = torch.empty(T, D, dtype=stream, **dev)
                s["do"] = torch.empty(T, D, dtype=branch, **dev)
                s["grads"] = {n: torch.empty(D, dtype=torch.float32, **dev) for n in s["params"]}
                if c["gate"] == "rows":
                    s["grads"]["gate"] = torch.empty(T, D, dtype=branch, **dev)
                s["ws"] = torch.empty(rg.moe_norm_workspace_bytes(s["plan"], T), dtype=torch.uint8, **dev)
    return s


def run(state):
    s, c = state, state["case"]
    if c["op"] == "decode":
        return _decode_own(s, c) if own else _decode_plain(s, c)
    if c["op"] == "norm":
        return _norm_own(s, c) if own else _norm_plain(s, c)
    return _norm_bwd_own(s, c) if own else _norm_bwd_plain(s, c)


# ---------------------------------------------------------------- the framework's calls
def _decode_own(s, c):
    if c["given"]:
        s["rg"].moe_decode_routed(s["plan"], c["T"], s["x"], s["weights"], s["topk_idx"], s["topk_w"], s["out"], s["ws"])
        return {"out": s["out"]}
    s["rg"].moe_decode(s["plan"], c["T"], s["x"], s["weights"], s["out"], s["ws"], topk_idx=s["topk_idx"], topk_w=s["topk_w"])
    return {"out": s["out"], "topk_idx": s["topk_idx"], "topk_w": s["topk_w"]}


def _norm_own(s, c):
    s["rg"].moe_norm(s["plan"], c["T"], s["params"], x=s["x"], o=s["o"], y=s["y"], h=s["h"], stats=s["stats"])
    return {"y": s["y"], "h": s["h"]}


def _norm_bwd_own(s, c):
    s["rg"].moe_norm_bwd(s["plan"], c["T"], s["params"], s["stats"], s["grads"], o=s["o"], y=s["y"], dy=s["dy"], dh=s["dh"],
                         dx=s["dx"], do=s["do"], workspace=s["ws"])
    return {"dx": s["dx"], "do": s["do"], **s["grads"]}


# ---------------------------------------------------------------- plain forms
def _mx_round(v):
    """The values that MXFP8 holds for v (blocks of 32 along the last axis): the
    scale 2^(floor(log2 max) - 8), elements to the nearest E4M3."""
    b = v.unflatten(-1, (-1, 32))
    m = b.abs().amax(-1, keepdim=True)
    e = torch.where(m > 0, torch.frexp(m).exponent - 1 - 8, -127).clamp(-127, 127)
    q = torch.ldexp(b, -e).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).to(v.dtype)
    return torch.where(m > 0, torch.ldexp(q, e), 0.0).flatten(-2)


def _values(s, name, pick):
    """A stack of routed weights in 32 bits: those of the experts in `pick`, or all."""
    w = s[name] if pick is None else s[name].view(torch.uint8 if s[name].element_size() == 1 else s[name].dtype)[pick].view(s[name].dtype)
    w = w.float()
    if name + "_e8m0" in s:
        e = s[name + "_e8m0"] if pick is None else s[name + "_e8m0"][pick]
        w.unflatten(-1, (-1, 32)).mul_(torch.exp2(e.float() - 127).unsqueeze(-1))
    return w


def _silu_times(gate, up):
    return gate / (1 + torch.exp(-gate)) * up


def _route_plain(s, c):
    """The selection compares logits next to each other: in 64 bits."""
    x = s["x"].double() @ s["W_router"].double().T
    if s["b_router"] is not None:
        x = x + s["b_router"].double()
    idx = torch.sort(x, dim=1, descending=True, stable=True).indices[:, : c["k"]].sort(1).values
    got = torch.gather(x, 1, idx)
    w = 1 / (1 + torch.exp(-got)) if c["score"] == "sigmoid" else torch.exp(got - got.amax(1, keepdim=True))
    return idx, (w / w.sum(1, keepdim=True)).float()


def _decode_plain(s, c):
    T, E, k = c["T"], c["E"], c["k"]
    if c["given"]:
        idx, w = s["topk_idx"].long(), s["topk_w"]
        idx, w = torch.where(idx >= 0, idx, 0), torch.where(idx >= 0, w, 0.0)
    else:
        idx, w = _route_plain(s, c)
    x = s["x"].float()
    mx = c["precision"] == "mxfp8"
    xr = _mx_round(x) if mx else x
    if T * k <= E:  # the selected experts' weights, a route each
        pick = idx.flatten()
        xp = xr.repeat_interleave(k, 0).unsqueeze(2)
        h = _silu_times(torch.matmul(_values(s, "W_gate", pick), xp), torch.matmul(_values(s, "W_up", pick), xp))
        if mx:
            h = _mx_round(h.squeeze(2)).unsqueeze(2)
        y = torch.matmul(_values(s, "W_down", pick), h).view(T, k, -1)
        out = (y * w.unsqueeze(2)).sum(1)
    else:  # every expert on every token, weighted
        h = _silu_times(torch.matmul(xr, _values(s, "W_gate", None).transpose(1, 2)),
                        torch.matmul(xr, _values(s, "W_up", None).transpose(1, 2)))
        if mx:
            h = _mx_round(h)
        full = torch.zeros(T, E, device=x.device).scatter_add_(1, idx, w)
        out = (torch.matmul(h, _values(s, "W_down", None).transpose(1, 2)) * full.T.unsqueeze(2)).sum(0)
    if c["I_s"]:
        h = _silu_times(torch.matmul(x, s["Ws_gate"].float().T), torch.matmul(x, s["Ws_up"].float().T))
        out = out + torch.matmul(h, s["Ws_down"].float().T)
    out = out.to(torch.bfloat16)
    return {"out": out} if c["given"] else {"out": out, "topk_idx": idx.to(torch.int32), "topk_w": w}


def _weight(s, c, name):
    return s[name + "_weight"].float() + c["offset"]


def _normed(v, s, c, name):
    if c["kind"] == "layer":
        v = v - v.mean(1, keepdim=True)
    v = v * (v.square().mean(1, keepdim=True) + EPS).rsqrt() * _weight(s, c, name)
    return v if s[name + "_bias"] is None else v + s[name + "_bias"].float()


def _norm_plain(s, c):
    z = s["o"].float()
    if c["post"]:
        z = _normed(z, s, c, "post")
    if s["gate"] is not None:
        z = z * s["gate"].float()
    y = c["x_scale"] * s["x"].float() + c["o_scale"] * z
    h = _normed(y, s, c, "pre") if c["pre"] else None
    return {"y": y.to(s["x"].dtype), "h": None if h is None else h.to(s["o"].dtype)}


def _norm_bwd_plain(s, c):
    grads = {}
    st = s["stats"]

    def back(d, v, name, at):
        """Through one norm: the gradient of its input; its parameters' into grads."""
        r = st[:, at + 1 : at + 2]
        n = (v.float() - st[:, at : at + 1]) * r
        grads[name + "_weight"] = (d * n).sum(0, dtype=torch.float64).float()
        if s[name + "_bias"] is not None:
            grads[name + "_bias"] = d.sum(0, dtype=torch.float64).float()
        u = d * _weight(s, c, name)
        t = u - n * (u * n).mean(1, keepdim=True)
        return r * (t - u.mean(1, keepdim=True) if c["kind"] == "layer" else t)

    dy = s["dy"].float()
    if c["pre"]:
        dy = dy + back(s["dh"].float(), s["y"], "pre", 2)
    dz = c["o_scale"] * dy
    if s["gate"] is not None:
        z = s["o"].float()
        if c["post"]:
            z = (z - st[:, 0:1]) * st[:, 1:2] * _weight(s, c, "post")
            z = z if s["post_bias"] is None else z + s["post_bias"].float()
        dg = dz * z
        grads["gate"] = dg.to(s["o"].dtype) if c["gate"] == "rows" else dg.sum(0, dtype=torch.float64).float()
        dz = dz * s["gate"].float()
    do = back(dz, s["o"], "post", 0) if c["post"] else dz
    order = ("post_weight", "post_bias", "pre_weight", "pre_bias", "gate")
    return {"dx": (c["x_scale"] * dy).to(s["dy"].dtype), "do": do.to(s["o"].dtype), **{n: grads[n] for n in order if n in grads}}


# ---------------------------------------------------------------- work
def work(case):
    c = case
    T, D = c["T"], c["D"]
    size = {"fp32": 4, "bf16": 2, "fp16": 2}
    if c["op"] == "decode":
        E, k, I, I_s = c["E"], c["k"], c["I"], c["I_s"]
        used = E * (1 - (1 - k * (1 - c["empty"]) / E) ** T)  # experts with a token, where every expert is as likely
        per = 2.0 if c["precision"] == "bf16" else 1.0 + 1.0 / 32
        b = 3 * D * (used * I * per + I_s * 2) + 4 * T * D + 8 * T * k
        f = 6 * T * D * (k * (1 - c["empty"]) * I + I_s)
        if not c["given"]:
            b, f = b + 2 * E * D, f + 2 * T * E * D
        return {"bytes": int(b), "flops": int(f)}
    st, br, pa = size[c["stream"]], size[c["branch"]], size[c["param"]]
    n_par = (c["post"] + c["pre"]) * (2 if c["biases"] else 1) + (c["gate"] == "vector")
    rows = T * D * br if c["gate"] == "rows" else 0
    if c["op"] == "norm":
        return {"bytes": T * D * (2 * st + br * (2 if c["pre"] else 1)) + rows + n_par * D * pa, "flops": 12 * T * D}
    # o is needed for its norm and for the gate's gradient alone
    read = st + (st + br if c["pre"] else 0) + (br if c["post"] or c["gate"] != "none" else 0)
    return {"bytes": T * D * (read + st + br) + 2 * rows + 16 * T + n_par * D * (pa + 4), "flops": 30 * T * D}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    c = case
    if c["op"] == "decode":
        return _decode_exact(c, _decode_inputs(c, seed))
    s = _norm_inputs(c, seed)
    return _norm_exact(c, s) if c["op"] == "norm" else _norm_bwd_exact(c, s)


def _f8(v):
    """To the nearest E4M3 value (ties to even), from the format: 3 bits after
    the leading one, exponents from -6, largest 448."""
    a = v.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, 1.0)))
    e = torch.where(torch.pow(2.0, e) > a, e - 1, e).clamp(min=-6)
    step = torch.pow(2.0, e - 3)
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=448.0)


def _mx_exact(v):
    out = torch.zeros_like(v)
    for b in range(0, v.shape[-1], 32):
        m = v[..., b : b + 32].abs().amax(-1, keepdim=True)
        e = torch.floor(torch.log2(torch.where(m > 0, m, 1.0)))
        e = torch.where(torch.pow(2.0, e) > m, e - 1, torch.where(torch.pow(2.0, e + 1) <= m, e + 1, e)) - 8
        out[..., b : b + 32] = torch.where(m > 0, _f8(v[..., b : b + 32] * torch.pow(2.0, -e)) * torch.pow(2.0, e), 0.0)
    return out


def _expert(s, name, e):
    w = s[name][e].to(torch.float64)
    if name + "_e8m0" in s:
        p = torch.pow(2.0, s[name + "_e8m0"][e].to(torch.float64) - 127)
        w = (w.reshape(w.shape[0], -1, 32) * p[:, :, None]).reshape(w.shape)
    return w


def _ffn64(x, up, gate, down, rnd):
    a = x @ gate.T
    return rnd(a * torch.sigmoid(a) * (x @ up.T)) @ down.T


def _decode_exact(c, s):
    T, E, k = c["T"], c["E"], c["k"]
    x = s["x"].to(torch.float64)
    out = torch.zeros_like(x)
    res = {"out": out}
    if c["given"]:
        idx, w = s["topk_idx"].cpu().numpy(), s["topk_w"].double().cpu().numpy()
    else:
        l = (x @ s["W_router"].to(torch.float64).T).cpu().numpy()
        if s["b_router"] is not None:
            l = l + s["b_router"].double().cpu().numpy()
        idx = np.sort(np.argsort(-l, axis=1, kind="stable")[:, :k], axis=1)
        sel = np.take_along_axis(l, idx, axis=1)
        v = np.exp(-np.logaddexp(0.0, -sel)) if c["score"] == "sigmoid" else np.exp(sel - l.max(axis=1, keepdims=True))
        w = v / v.sum(axis=1, keepdims=True)
        res.update(topk_idx=idx.astype(np.int32), topk_w=w)
    mx = c["precision"] == "mxfp8"
    rnd = _mx_exact if mx else (lambda v: v)
    xr = rnd(x)
    for e in range(E):
        t, j = np.nonzero(idx == e)
        if len(t):
            at = torch.from_numpy(t).to(x.device)
            y = _ffn64(xr[at], _expert(s, "W_up", e), _expert(s, "W_gate", e), _expert(s, "W_down", e), rnd)
            out.index_add_(0, at, y * torch.from_numpy(w[t, j]).to(x.device)[:, None])
    if c["I_s"]:
        out += _ffn64(x, *(s[n].to(torch.float64) for n in ("Ws_up", "Ws_gate", "Ws_down")), lambda v: v)
    return res


def _mean_dev(v, c):
    m = v.mean(1, keepdim=True) if c["kind"] == "layer" else torch.zeros_like(v[:, :1])
    return m, torch.sqrt((v - m).pow(2).mean(1, keepdim=True) + EPS)


def _norm_exact(c, s):
    def norm(v, name):
        m, d = _mean_dev(v, c)
        v = (v - m) / d * (s[name + "_weight"].to(torch.float64) + c["offset"])
        return v if s[name + "_bias"] is None else v + s[name + "_bias"].to(torch.float64)

    z = s["o"].to(torch.float64)
    z = norm(z, "post") if c["post"] else z
    g = 1.0 if s["gate"] is None else s["gate"].to(torch.float64)
    y = c["x_scale"] * s["x"].to(torch.float64) + c["o_scale"] * g * z
    return {"y": y, "h": norm(y, "pre") if c["pre"] else None}


def _norm_bwd_exact(c, s):
    """By automatic differentiation of the forward in 64 bits, the stream taken at y."""
    if c["T"] * c["D"] > 5e8:
        return None
    names = ("post_weight", "post_bias", "pre_weight", "pre_bias", "gate")
    p = {n: s[n].to(torch.float64).requires_grad_() for n in names if s[n] is not None}
    o = s["o"].to(torch.float64).requires_grad_()

    def norm(v, name):
        m, d = _mean_dev(v, c)
        v = (v - m) / d * (p[name + "_weight"] + c["offset"])
        return v + p[name + "_bias"] if name + "_bias" in p else v

    z = norm(o, "post") if c["post"] else o
    b = c["o_scale"] * (z * p["gate"] if "gate" in p else z)
    dy = s["dy"].to(torch.float64)
    if c["pre"]:
        y = s["y"].to(torch.float64).requires_grad_()
        q = [p[n] for n in ("pre_weight", "pre_bias") if n in p]
        got = torch.autograd.grad(norm(y, "pre"), [y, *q], s["dh"].to(torch.float64))
        dy = dy + got[0]
        rest = dict(zip([n for n in ("pre_weight", "pre_bias") if n in p], got[1:]))
    else:
        rest = {}
    q = [n for n in ("post_weight", "post_bias", "gate") if n in p]
    got = torch.autograd.grad(b, [o, *(p[n] for n in q)], dy)
    rest.update(zip(q, got[1:]))
    return {"dx": c["x_scale"] * dy, "do": got[0], **{n: rest[n] for n in names if n in rest}}
