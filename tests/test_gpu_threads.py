"""Calls from host threads other than the one that made the plan."""
import threading

import pytest
import torch

import routing_grouped_expert_gemm_gb300 as rg

pytestmark = pytest.mark.gpu


def weights(gen, E, D, I):
    r = lambda *s: (torch.randn(*s, generator=gen, device="cuda") * s[-1] ** -0.5).bfloat16()  # noqa: E731
    return {"W_router": r(E, D), "W_up": r(E, I, D), "W_gate": r(E, I, D), "W_down": r(E, D, I)}


def bytes_of(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


def the_calls():
    """A call of each kind, with its outputs; every argument is made before."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    T, D, I, E, k = 16, 256, 256, 8, 2
    plan, w, s = rg.moe_plan_create(T, D, I, E, k), weights(gen, E, D, I), torch.cuda.current_stream()
    x = torch.randn(T, D, generator=gen, device="cuda").bfloat16()
    out, ws, dws = torch.empty_like(x), bytes_of(rg.moe_workspace_bytes(plan, T)), bytes_of(rg.moe_decode_workspace_bytes(plan, T))
    out_d, fws, bws = torch.empty_like(x), torch.empty_like(ws), bytes_of(rg.moe_bwd_workspace_bytes(plan, T))
    rg.moe_fwd(plan, T, x, w, out.clone(), fws)
    grads = {"dx": torch.empty_like(x), "dW_router": torch.empty(E, D, device="cuda"),
             **{"d" + n: torch.empty_like(w[n]) for n in ("W_up", "W_gate", "W_down")}}
    mplan = rg.moe_muon_plan_create(2, 300, 260, grad_dtype="fp32")
    g, mom, upd = torch.randn(2, 300, 260, generator=gen, device="cuda"), torch.zeros(2, 300, 260, device="cuda"), torch.empty(2, 300, 260, dtype=torch.bfloat16, device="cuda")
    mws = bytes_of(rg.moe_muon_workspace_bytes(mplan))
    i32 = lambda *n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    route = [i32(T, k), torch.empty(T, k, device="cuda"), i32(E), i32(E + 1), i32(T * k, 3), i32(T * k)]
    nplan, h = rg.moe_norm_plan_create(D, post=False), torch.empty_like(x)
    torch.cuda.synchronize()
    return {
        "moe_fwd": (lambda: rg.moe_fwd(plan, T, x, w, out, ws, stream=s), [out]),
        "moe_bwd": (lambda: rg.moe_bwd(plan, T, x, w, x, fws, grads, bws, stream=s), list(grads.values())),
        "moe_decode": (lambda: rg.moe_decode(plan, T, x, w, out_d, dws, stream=s), [out_d]),
        "moe_route_static": (lambda: rg.moe_route_static(plan, T, x, w["W_router"], None, *route, stream=s), route[:4]),
        "moe_muon_update": (lambda: rg.moe_muon_update(mplan, g, mom, upd, mws, mu=0.0, stream=s), [upd]),
        "moe_norm": (lambda: rg.moe_norm(nplan, T, {}, x=x, h=h, stream=s), [h]),
    }


@pytest.mark.parametrize("name", ["moe_fwd", "moe_bwd", "moe_decode", "moe_route_static", "moe_muon_update", "moe_norm"])
def test_first_call_of_a_thread(name):
    """Nothing of CUDA has run in the thread before."""
    f, outs = the_calls()[name]
    f()
    torch.cuda.synchronize()
    want, errors = [t.clone() for t in outs], []
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()

    def work():
        try:
            f()
        except rg.MoEError as e:
            errors.append(str(e))

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors
    assert all(torch.equal(a, b) for a, b in zip(want, outs))


def at_once(calls, outs, n):
    """n calls a thread, each thread on a stream and a workspace of its own: every call
    succeeds, and the outputs are those of a call alone.  The threads' calls go to the same
    kernels with different amounts of shared memory."""
    want = []
    for f, out in zip(calls, outs):
        f(torch.cuda.current_stream())
        torch.cuda.synchronize()
        want.append([t.clone() for t in out])
        for t in out:
            t.zero_()
    go, errors, streams = threading.Barrier(len(calls)), [], [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()

    def work(f, stream):
        go.wait()
        try:
            for _ in range(n):
                f(stream)
        except rg.MoEError as e:
            errors.append(str(e))

    threads = [threading.Thread(target=work, args=a) for a in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for w, out in zip(want, outs):
        assert all(torch.equal(a, b) for a, b in zip(w, out))


def test_batches_of_two_sizes_on_one_plan():
    gen = torch.Generator(device="cuda").manual_seed(1)
    D, I, E = 256, 128, 8
    plan, w = rg.moe_plan_create(64, D, I, E, 2), weights(gen, E, D, I)
    calls, outs = [], []
    for T in (1, 64, 1, 64):
        x = torch.randn(T, D, generator=gen, device="cuda").bfloat16()
        out = torch.empty_like(x)
        ws = torch.empty(rg.moe_decode_workspace_bytes(plan, T), dtype=torch.uint8, device="cuda")
        calls.append(lambda s, T=T, x=x, out=out, ws=ws: rg.moe_decode(plan, T, x, w, out, ws, stream=s))
        outs.append([out])
    at_once(calls, outs, 3000)


@pytest.mark.parametrize("widths", [(7168, 8192), (5001, 8001)])
def test_norms_of_two_widths(widths):
    gen = torch.Generator(device="cuda").manual_seed(2)
    calls, outs = [], []
    for D in 2 * widths:
        plan, T = rg.moe_norm_plan_create(D), 300
        x, o, dy, dh = (torch.randn(T, D, generator=gen, device="cuda").bfloat16() for _ in range(4))
        y, h, dx, do = (torch.empty_like(x) for _ in range(4))
        st, p = torch.empty(T, 4, device="cuda"), {n: torch.ones(D, device="cuda") for n in ("post_weight", "pre_weight")}
        g, ws = {n: torch.empty(D, device="cuda") for n in p}, torch.empty(rg.moe_norm_workspace_bytes(plan, T), dtype=torch.uint8, device="cuda")

        def call(s, plan=plan, T=T, p=p, x=x, o=o, y=y, h=h, st=st, g=g, dy=dy, dh=dh, dx=dx, do=do, ws=ws):
            rg.moe_norm(plan, T, p, x=x, o=o, y=y, h=h, stats=st, stream=s)
            rg.moe_norm_bwd(plan, T, p, st, g, o=o, y=y, dy=dy, dh=dh, dx=dx, do=do, workspace=ws, stream=s)

        calls.append(call)
        outs.append([y, h, dx, do, *g.values()])
    at_once(calls, outs, 3000)


def test_layers_of_two_plans():
    gen = torch.Generator(device="cuda").manual_seed(3)
    calls, outs = [], []
    for E in (8, 500, 8, 500):
        plan, T, D, I = rg.moe_plan_create(64, 256, 128, E, 2), 64, 256, 128
        w, x = weights(gen, E, D, I), torch.randn(T, D, generator=gen, device="cuda").bfloat16()
        out = torch.empty_like(x)
        ws = torch.empty(rg.moe_workspace_bytes(plan, T), dtype=torch.uint8, device="cuda")
        calls.append(lambda s, plan=plan, T=T, x=x, w=w, out=out, ws=ws: rg.moe_fwd(plan, T, x, w, out, ws, stream=s))
        outs.append([out])
    at_once(calls, outs, 1500)
