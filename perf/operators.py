"""Workloads of the routing and optimiser operators: inputs, the operators'
plain form in elementary torch operations, the framework's calls, and the
operators' definition in 64 bits.

route       scores of the router's logits (sigmoid or softmax), a balance bias
            that takes part in the selection only, expert groups, top-k,
            renormalised weights; optionally the routes per expert and the
            normalised scores summed over the tokens (for a balance loss)
route_bwd   the gradient of the logits from the gradients of the weights and of
            those score sums
muon        momentum and the orthogonalisation of the update of a stack of
            weight matrices by Newton-Schulz products
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
COEFS = (3.4445, -4.7750, 2.0315)


def _route(name, T, E, k, score, dtype, bias, n_group=1, topk_group=1, group_top=2, renorm=True, scale=1.0, sums=False,
           masked=0.0, op="route"):
    c = dict(op=op, T=T, E=E, k=k, score=score, dtype=dtype, bias=bias, n_group=n_group, topk_group=topk_group,
             group_top=group_top, renorm=renorm, scale=scale, sums=sums, masked=masked)
    return dict(name=name, **c) if name else c


def _muon(name, count, rows, cols, dtype, momentum):
    c = dict(op="muon", count=count, rows=rows, cols=cols, dtype=dtype, momentum=momentum)
    return dict(name=name, **c) if name else c


def listed():
    return [
        # one token of a decode step: 256 experts in 8 groups of which 4 are kept, balance bias
        _route("route_decode_1", 1, 256, 8, "sigmoid", "fp32", True, 8, 4, 2, True, 2.5),
        # odd sizes, fp16, some experts masked per token and some tokens wholly masked
        _route("route_odd_masked", 1003, 100, 6, "softmax", "fp16", True, 5, 3, 1, True, 1.0, True, 0.2),
        # a training batch of the grouped sigmoid router, with the balance loss's sums
        _route("route_train_256", 16384, 256, 8, "sigmoid", "fp32", True, 8, 4, 2, True, 2.5, True),
        # a large batch over 384 experts, bf16 logits, no groups
        _route("route_384", 32768, 384, 8, "sigmoid", "bf16", True, 1, 1, 2, True, 2.5),
        # gradients: the grouped sigmoid router with its balance loss (every logit gets a gradient)
        _route("route_bwd_train_256", 16384, 256, 8, "sigmoid", "fp32", True, 8, 4, 2, True, 2.5, True, op="route_bwd"),
        # softmax weights without renormalisation, bf16: dense gradient through the softmax
        _route("route_bwd_softmax_128", 8192, 128, 8, "softmax", "bf16", False, 1, 1, 1, False, 1.0, op="route_bwd"),
        # few tokens, odd expert count: renormalised, so only the selected logits get a gradient
        _route("route_bwd_small", 37, 60, 4, "softmax", "fp32", True, 1, 1, 1, True, 1.0, op="route_bwd"),
        # the up projections of a small layer: 16 experts of 128 x 256
        _muon("muon_tiny", 16, 128, 256, "bf16", True),
        # odd sizes, fp32 gradient, orthogonalisation alone
        _muon("muon_odd", 3, 777, 1001, "fp32", False),
        # a few experts' up projections, 1024 x 4096
        _muon("muon_1024x4096", 8, 1024, 4096, "bf16", True),
        # up projections (wide) and down projections (tall) of the 2048 x 7168 layer
        _muon("muon_wide", 16, 2048, 7168, "bf16", True),
        _muon("muon_tall", 8, 7168, 2048, "bf16", True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route", "route_bwd", "route_bwd", "muon", "muon"])
    if op != "muon":
        n_group = rng.choice([1, 1, 2, 4, 5, 8])
        gs = _log_int(rng, 8 if n_group == 1 else 4, 384 // n_group)
        E = n_group * gs
        topk_group = rng.randint(1, n_group)
        k = rng.randint(1, min(16, topk_group * gs))
        T = _log_int(rng, 1, 16384)
        return _route(None, T, E, k, rng.choice(["sigmoid", "softmax"]), rng.choice(["fp32", "bf16", "fp16"]),
                      rng.random() < 0.6, n_group, topk_group, rng.choice([1, 2]), rng.random() < 0.7,
                      rng.choice([1.0, 2.5]), rng.random() < 0.5, rng.choice([0.0, 0.0, 0.2]), op=op)
    rows, cols = _log_int(rng, 16, 4096), _log_int(rng, 16, 4096)
    most = 4.0e11 / (5 * _muon_flops(1, rows, cols))
    return _muon(None, max(1, _log_int(rng, 1, max(1.0, min(32.0, most)))), rows, cols,
                 rng.choice(["fp32", "bf16", "bf16", "fp16"]), rng.random() < 0.7)


def _gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _route_inputs(c, seed, device="cuda"):
    """Router logits whose experts differ in popularity, tokens in sharpness."""
    g = _gen(seed, device)
    T, E, k = c["T"], c["E"], c["k"]
    pop = torch.randn(E, generator=g, device=device) * 0.5
    sharp = 0.5 + torch.rand(T, 1, generator=g, device=device)
    x = torch.randn(T, E, generator=g, device=device) * sharp + pop - 1.0
    if c["masked"]:
        x.masked_fill_(torch.rand(T, E, generator=g, device=device) < c["masked"], -math.inf)
        x.masked_fill_(torch.rand(T, 1, generator=g, device=device) < c["masked"] / 4, -math.inf)
    s = {"logits": x.to(DTYPES[c["dtype"]]), "bias": None}
    if c["bias"]:
        s["bias"] = (torch.rand(E, generator=g, device=device) - 0.5) * 0.1
    if c["op"] == "route_bwd":
        # the experts a forward selected (here the largest logits), in ascending order; -1 for an empty slot
        v, i = torch.topk(s["logits"].float(), k, dim=1)
        i = torch.where(v > -math.inf, i, E).sort(dim=1).values
        s["topk_idx"] = torch.where(i < E, i, -1).to(torch.int32)
        s["dtopk_w"] = torch.randn(T, k, generator=g, device=device)
        s["dprob_sum"] = torch.randn(E, generator=g, device=device) * 0.1 if c["sums"] else None
    return s


def _muon_inputs(c, seed, device="cuda"):
    """Gradients of a stack of expert matrices: a decaying spectrum of shared
    directions above noise; the momentum of earlier steps likewise."""
    g = _gen(seed, device)
    B, R, C = c["count"], c["rows"], c["cols"]
    r = max(1, min(R, C) // 8)

    def one(n):
        u = torch.randn(B, R, r, generator=g, device=device)
        v = torch.randn(B, r, C, generator=g, device=device)
        d = torch.arange(1, r + 1, device=device, dtype=torch.float32) ** -0.5
        return torch.matmul(u * d, v) + n * torch.randn(B, R, C, generator=g, device=device)

    s = {"grad": (one(1.0) * 1e-4).to(DTYPES[c["dtype"]]), "momentum": None}
    if c["momentum"]:
        s["momentum"] = one(0.5) * 1e-3
    return s


def prepare(case, seed):
    c = case
    if c["op"] == "muon":
        s = _muon_inputs(c, seed)
    else:
        s = _route_inputs(c, seed)
    s["case"] = c
    if own:  # the handle, outputs and workspace that a program keeps
        import routing_grouped_expert_gemm_gb300 as rg
        s["rg"] = rg
        dev = dict(device="cuda")
        if c["op"] == "muon":
            s["plan"] = rg.moe_muon_plan_create(c["count"], c["rows"], c["cols"], grad_dtype=c["dtype"])
            s["update"] = torch.empty(c["count"], c["rows"], c["cols"], dtype=torch.bfloat16, **dev)
            s["ws"] = torch.empty(rg.moe_muon_workspace_bytes(s["plan"]), dtype=torch.uint8, **dev)
        else:
            T, E, k = c["T"], c["E"], c["k"]
            s["plan"] = rg.moe_route_plan_create(E, k, score_fn=c["score"], logits_dtype=c["dtype"], n_group=c["n_group"],
                                                 topk_group=c["topk_group"], group_top=c["group_top"],
                                                 renormalize=c["renorm"], scale=c["scale"])
            if c["op"] == "route":
                s["topk_idx"] = torch.empty(T, k, dtype=torch.int32, **dev)
                s["topk_w"] = torch.empty(T, k, dtype=torch.float32, **dev)
                s["counts"] = torch.empty(E, dtype=torch.int32, **dev) if c["sums"] else None
                s["prob_sum"] = torch.empty(E, dtype=torch.float32, **dev) if c["sums"] else None
                s["ws"] = torch.empty(rg.moe_route_workspace_bytes(s["plan"], T), dtype=torch.uint8, **dev)
            else:
                s["dlogits"] = torch.empty(T, E, dtype=DTYPES[c["dtype"]], **dev)
    return s


def run(state):
    s, c = state, state["case"]
    if c["op"] == "route":
        return _route_own(s, c) if own else _route_plain(s, c)
    if c["op"] == "route_bwd":
        return _route_bwd_own(s, c) if own else _route_bwd_plain(s, c)
    return _muon_own(s, c) if own else _muon_plain(s, c)


# ---------------------------------------------------------------- the framework's calls
def _route_own(s, c):
    s["rg"].moe_route(s["plan"], c["T"], s["logits"], s["bias"], s["topk_idx"], s["topk_w"], expert_counts=s["counts"],
                      prob_sum=s["prob_sum"], workspace=s["ws"])
    return {"topk_idx": s["topk_idx"], "topk_w": s["topk_w"], "counts": s["counts"], "prob_sum": s["prob_sum"]}


def _route_bwd_own(s, c):
    s["rg"].moe_route_bwd(s["plan"], c["T"], s["logits"], s["topk_idx"], s["dtopk_w"], s["dlogits"],
                          dprob_sum=s["dprob_sum"])
    return {"dlogits": s["dlogits"]}


def _muon_own(s, c):
    s["rg"].moe_muon_update(s["plan"], s["grad"], s["momentum"], s["update"], s["ws"], mu=0.95, nesterov=True, scale=0.2)
    return {"update": s["update"], "momentum": s["momentum"]}


# ---------------------------------------------------------------- plain forms
def _scores(x, score):
    """Scores of every expert and their sum over the row; a row without an expert scores 0."""
    if score == "sigmoid":
        s = torch.where(x > -math.inf, 1 / (1 + torch.exp(-x)), 0.0)
        return s, s.sum(1, keepdim=True)
    m = x.amax(1, keepdim=True)
    e = torch.where(x > -math.inf, torch.exp(x - torch.where(m > -math.inf, m, 0.0)), 0.0)
    z = e.sum(1, keepdim=True)
    s = torch.where(z > 0, e / z, 0.0)
    return s, torch.where(z > 0, 1.0, 0.0).to(s.dtype)


def _route_plain(s, c):
    E, k, G = c["E"], c["k"], c["n_group"]
    x = s["logits"].double()  # the selection compares values next to each other: in 64 bits
    live = x > -math.inf
    key = _scores(x, c["score"])[0] if (c["bias"] or G > 1) else x
    if s["bias"] is not None:
        key = key + s["bias"].double()
    key = torch.where(live, key, -math.inf)
    if G > 1:
        top = torch.sort(key.view(-1, G, E // G), dim=2, descending=True).values[:, :, : c["group_top"]]
        empty = top[:, :, 0] == -math.inf
        gscore = torch.where(top > -math.inf, top, 0.0).sum(2)
        gscore = torch.where(empty, -math.inf, gscore)
        order = torch.sort(gscore, dim=1, descending=True, stable=True).indices[:, : c["topk_group"]]
        keep = torch.zeros_like(gscore, dtype=torch.bool).scatter_(1, order, True)
        live = live & keep.repeat_interleave(E // G, dim=1)
        if s["bias"] is None:
            key = x
        key = torch.where(live, key, -math.inf)
    idx = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    got = torch.gather(live, 1, idx)
    idx = torch.where(got, idx, E).sort(dim=1).values
    got = idx < E
    at = torch.where(got, idx, 0)
    p, total = _scores(s["logits"].float(), c["score"])
    w = torch.where(got, torch.gather(p, 1, at), 0.0)
    if c["renorm"]:
        t = w.sum(1, keepdim=True)
        w = torch.where(t > 0, w / t, 0.0)
    out = {"topk_idx": torch.where(got, idx, -1).to(torch.int32), "topk_w": w * c["scale"], "counts": None, "prob_sum": None}
    if c["sums"]:
        hit = torch.zeros(idx.shape[0], E + 1, dtype=torch.int32, device=x.device).scatter_(1, idx, 1)
        out["counts"] = hit[:, :E].sum(0).to(torch.int32)
        out["prob_sum"] = torch.where(total > 0, p / total, 0.0).sum(0)
    return out


def _route_bwd_plain(s, c):
    x = s["logits"].float()
    p, total = _scores(x, c["score"])
    idx = s["topk_idx"].long()
    got = idx >= 0
    at = torch.where(got, idx, 0)
    dw = torch.where(got, s["dtopk_w"], 0.0) * c["scale"]
    q = torch.where(got, torch.gather(p, 1, at), 0.0)
    if c["renorm"]:
        t = q.sum(1, keepdim=True)
        q = torch.where(t > 0, q / t, 0.0)
        part = q * (dw - (q * dw).sum(1, keepdim=True))
    else:
        part = q * dw
    d = torch.zeros_like(p).scatter_add_(1, at, part)  # ds times s, at the selected experts
    if c["score"] == "softmax" and not c["renorm"]:
        d = d - p * part.sum(1, keepdim=True)
    if s["dprob_sum"] is not None:
        n = torch.where(total > 0, p / total, 0.0)
        d = d + n * (s["dprob_sum"] - (n * s["dprob_sum"]).sum(1, keepdim=True))
    if c["score"] == "sigmoid":
        d = d * (1 - p)
    return {"dlogits": d.to(s["logits"].dtype)}


def _muon_plain(s, c):
    u = s["grad"].float()
    if s["momentum"] is not None:
        m = s["momentum"].mul_(0.95).add_(u)
        u = u + 0.95 * m
    a, b, k = COEFS
    x = u / u.square().sum((1, 2), keepdim=True, dtype=torch.float64).sqrt().float()
    tall = c["rows"] > c["cols"]
    if tall:
        x = x.transpose(1, 2)
    for _ in range(5):
        y = torch.matmul(x, x.transpose(1, 2))
        x = a * x + torch.matmul(b * y + k * torch.matmul(y, y), x)
    if tall:
        x = x.transpose(1, 2)
    return {"update": (0.2 * x).to(torch.bfloat16).contiguous(), "momentum": s["momentum"]}


# ---------------------------------------------------------------- work
def _muon_flops(count, rows, cols):
    """One step's products: the two symmetric ones need half of their entries."""
    m, n = min(rows, cols), max(rows, cols)
    return count * (m * m * n + m * m * m + 2 * m * m * n)


def work(case):
    c = case
    size = 4 if c["dtype"] == "fp32" else 2
    if c["op"] == "muon":
        n = c["count"] * c["rows"] * c["cols"]
        return {"bytes": n * (size + 2 + (8 if c["momentum"] else 0)), "flops": 5 * _muon_flops(c["count"], c["rows"], c["cols"])}
    T, E, k = c["T"], c["E"], c["k"]
    if c["op"] == "route":
        return {"bytes": T * E * size + T * k * 8 + (4 * E if c["bias"] else 0) + (8 * E if c["sums"] else 0), "flops": 4 * T * E}
    dense = c["sums"] or (c["score"] == "softmax" and not c["renorm"])
    read = T * E * size if dense else T * k * size
    return {"bytes": read + T * k * 8 + T * E * size + (4 * E if c["sums"] else 0), "flops": (6 * T * E if dense else 8 * T * k)}


# ---------------------------------------------------------------- the definition in 64 bits
def _np(t):
    return None if t is None else t.to(torch.float64).cpu().numpy()


def exact(case, seed):
    c = case
    if c["op"] == "muon":
        return _muon_exact(c, seed)
    s = _route_inputs(c, seed)
    x = _np(s["logits"])
    return _route_exact(c, x, _np(s["bias"])) if c["op"] == "route" else _route_bwd_exact(c, x, s)


def _np_probs(c, x):
    """(score s, log of the score up to the row's shift) per row in 64 bits."""
    if c["score"] == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(np.isneginf(x), 0.0, np.exp(-np.logaddexp(0.0, -x)))
    m = np.max(x, axis=1, keepdims=True)
    e = np.exp(x - np.where(np.isneginf(m), 0.0, m))
    z = e.sum(axis=1, keepdims=True)
    return e / np.where(z == 0, 1.0, z)


def _np_share(v):
    """Each value over its row's sum; a row of zeros stays zero."""
    t = v.sum(axis=1, keepdims=True)
    return v / np.where(t == 0, 1.0, t)


def _route_exact(c, x, bias):
    T, E, k, G = c["T"], c["E"], c["k"], c["n_group"]
    p = _np_probs(c, x)
    rank = x if bias is None else np.where(np.isneginf(x), -np.inf, p + bias)
    if G > 1:
        value = np.where(np.isneginf(x), -np.inf, p + (0.0 if bias is None else bias)).reshape(T, G, E // G)
        best = -np.sort(-value, axis=2)[:, :, : c["group_top"]]
        score = np.where(np.isneginf(best[:, :, 0]), -np.inf, np.where(np.isneginf(best), 0.0, best).sum(axis=2))
        place = np.argsort(np.argsort(-score, axis=1, kind="stable"), axis=1, kind="stable")
        rank = np.where(np.repeat(place < c["topk_group"], E // G, axis=1), rank, -np.inf)
    first = np.argsort(-rank, axis=1, kind="stable")[:, :k]
    chosen = np.zeros((T, E), dtype=bool)
    np.put_along_axis(chosen, first, True, axis=1)
    chosen &= ~np.isneginf(rank)
    idx = np.sort(np.where(chosen, np.arange(E), E), axis=1)[:, :k]
    taken = np.where(chosen, p, 0.0)
    w = np.take_along_axis(np.concatenate([_np_share(taken) if c["renorm"] else taken, np.zeros((T, 1))], axis=1), idx, axis=1)
    out = {"topk_idx": np.where(idx < E, idx, -1).astype(np.int32), "topk_w": w * c["scale"], "counts": None, "prob_sum": None}
    if c["sums"]:
        out["counts"] = chosen.sum(axis=0).astype(np.int32)
        out["prob_sum"] = _np_share(p).sum(axis=0)
    return out


def _route_bwd_exact(c, x, s):
    """Through the Jacobian of each output with respect to the scores, then of the scores."""
    T, E = x.shape
    p = _np_probs(c, x)
    idx = s["topk_idx"].cpu().numpy().astype(np.int64)
    dw = np.zeros((T, E + 1))
    np.put_along_axis(dw, np.where(idx < 0, E, idx), _np(s["dtopk_w"]) * c["scale"], axis=1)
    chosen = np.zeros((T, E + 1), dtype=bool)
    np.put_along_axis(chosen, np.where(idx < 0, E, idx), True, axis=1)
    dw, chosen = dw[:, :E], chosen[:, :E]
    if c["renorm"]:
        t = np.where(chosen, p, 0.0).sum(axis=1, keepdims=True)
        t = np.where(t == 0, 1.0, t)
        ds = np.where(chosen, dw / t - (dw * np.where(chosen, p, 0.0)).sum(axis=1, keepdims=True) / t**2, 0.0)
    else:
        ds = np.where(chosen, dw, 0.0)
    if c["sums"]:
        d = _np(s["dprob_sum"])
        t = p.sum(axis=1, keepdims=True)
        t = np.where(t == 0, 1.0, t)
        ds = ds + d / t - (d * p).sum(axis=1, keepdims=True) / t**2
    if c["score"] == "sigmoid":
        return {"dlogits": ds * p * (1.0 - p)}
    return {"dlogits": p * ds - p * (p * ds).sum(axis=1, keepdims=True)}


def _muon_exact(c, seed):
    if 5 * _muon_flops(c["count"], c["rows"], c["cols"]) > 1.2e13:
        return None
    s = _muon_inputs(c, seed)
    a, b, k = COEFS
    update = torch.empty(s["grad"].shape, dtype=torch.float64, device="cuda")
    moved = None if s["momentum"] is None else torch.empty_like(update)
    for i in range(c["count"]):
        g = s["grad"][i].to(torch.float64)
        if moved is not None:
            moved[i] = 0.95 * s["momentum"][i].to(torch.float64) + g
            g = g + 0.95 * moved[i]
        x = g / torch.linalg.matrix_norm(g)
        for _ in range(5):  # p(X) = a X + b (X X') X + k (X X')^2 X, from the smaller side
            if c["rows"] <= c["cols"]:
                y = x @ x.T
                x = a * x + b * (y @ x) + k * (y @ (y @ x))
            else:
                y = x.T @ x
                x = a * x + b * (x @ y) + k * ((x @ y) @ y)
        update[i] = 0.2 * x
    return {"update": update, "momentum": moved}
