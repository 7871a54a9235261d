"""The norms' plans without a GPU: refused configurations, and null arguments."""
import pytest
import torch

import routing_grouped_expert_gemm_gb300 as rg
from routing_grouped_expert_gemm_gb300 import build as rgbuild


@pytest.fixture(scope="module")
def L():
    rgbuild.build()
    return rg.lib()


@pytest.mark.parametrize("kw,code", [
    (dict(D=0), rg.MOE_ERR_UNSUPPORTED_SHAPE), (dict(D=16385), rg.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(kind=2), rg.MOE_ERR_INVALID_ARG), (dict(post=2), rg.MOE_ERR_INVALID_ARG), (dict(pre=-1), rg.MOE_ERR_INVALID_ARG),
    (dict(stream_dtype=3), rg.MOE_ERR_INVALID_ARG), (dict(param_dtype=-1), rg.MOE_ERR_INVALID_ARG),
    (dict(stream_dtype="bf16", branch_dtype="fp16"), rg.MOE_ERR_INVALID_ARG),
    (dict(stream_dtype="bf16", branch_dtype="fp32"), rg.MOE_ERR_INVALID_ARG),
    (dict(eps=0.0), rg.MOE_ERR_INVALID_ARG), (dict(eps=float("nan")), rg.MOE_ERR_INVALID_ARG),
    (dict(eps=float("inf")), rg.MOE_ERR_INVALID_ARG), (dict(x_scale=float("inf")), rg.MOE_ERR_INVALID_ARG),
    (dict(o_scale=float("nan")), rg.MOE_ERR_INVALID_ARG), (dict(weight_offset=float("-inf")), rg.MOE_ERR_INVALID_ARG)])
def test_plan_refuses(L, kw, code):
    with pytest.raises(rg.MoEError) as e:
        rg.moe_norm_plan_create(**{**dict(D=64), **kw})
    assert e.value.code == code


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-GPU path")
@pytest.mark.parametrize("kw", [dict(), dict(D=1), dict(D=16384), dict(kind="layer", post=False, pre=False),
                                dict(stream_dtype="fp32", branch_dtype="fp16", param_dtype="bf16")])
def test_valid_plans_reach_the_device(L, kw):
    with pytest.raises(rg.MoEError) as e:
        rg.moe_norm_plan_create(**{**dict(D=64), **kw})
    assert e.value.code in (rg.MOE_ERR_CUDA, rg.MOE_ERR_UNSUPPORTED_DEVICE)


def test_null_arguments(L):
    assert L.moe_norm_plan_create(None, None) == rg.MOE_ERR_INVALID_ARG
    assert L.moe_norm_plan_destroy(None) == rg.MOE_OK
    assert L.moe_norm_workspace_bytes(None, 4) == 0
    assert L.moe_norm(None, 1, None, *[None, 0] * 4, None, None) == rg.MOE_ERR_INVALID_ARG
    assert L.moe_norm_bwd(None, 1, None, None, *[None, 0] * 6, None, None, 0, None) == rg.MOE_ERR_INVALID_ARG


class _Reached:
    """Stands in for the library: says yes, and what the binding called."""

    def __init__(self):
        self.calls = []

    def moe_error_string(self, code):
        return b"refused"

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name, a)) or rg.MOE_OK


T, D = 6, 8
ZERO = torch.zeros


def _calls(monkeypatch, gate, grad=None):
    """The calls that reach the library with this gate (and gradient), or the refusal's code."""
    stub = _Reached()
    monkeypatch.setattr(rg, "lib", lambda: stub)
    plan = rg.NormPlan(0, rg.moe_norm_config(D))
    row = ZERO(T, D, dtype=torch.bfloat16)
    try:
        if grad is None:
            rg.moe_norm(plan, T, {"gate": gate}, x=row, o=row, y=row, h=row, stream=0)
        else:
            rg.moe_norm_bwd(plan, T, {"gate": gate}, 0, {"gate": grad}, o=row, y=row, dy=row, dh=row, stream=0)
    except rg.MoEError as e:
        assert not stub.calls
        return e.code
    return stub.calls


# read as [T, D] or as [D], each of these would be read past its end or by the wrong rows
@pytest.mark.parametrize("gate", [
    ZERO(T, 1), ZERO(1, D), ZERO(T - 1, D), ZERO(1), ZERO(D - 1), ZERO(D + 1), ZERO(2 * D)[::2], ZERO(T, D + 1), ZERO(T, D - 1), ZERO(1, D).expand(T, D),
    ZERO(T, 1).expand(T, D), ZERO(2, T // 2, D - 1), ZERO(())], ids=lambda t: f"{tuple(t.shape)}_{tuple(t.stride())}")
def test_gates_of_other_shapes_are_refused(monkeypatch, gate):
    assert _calls(monkeypatch, gate) == rg.MOE_ERR_INVALID_ARG
    assert _calls(monkeypatch, gate, ZERO(D)) == rg.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("gate,stride", [(None, 0), (ZERO(D), 0), (ZERO(T, D), D), (ZERO(T + 3, D), D), (ZERO(2, T // 2, D), D),
                                         (ZERO(T, D + 5)[:, :D], D + 5), (4096, 0)])
def test_gates_that_are_taken(monkeypatch, gate, stride):
    (name, args), = _calls(monkeypatch, gate)
    assert name == "moe_norm" and args[2].gate_stride == stride


ROWS = torch.bfloat16


@pytest.mark.parametrize("gate,grad,ok", [
    (ZERO(D), ZERO(D), True), (ZERO(D), ZERO(1, D), True), (ZERO(D), ZERO(T, D), False), (ZERO(D), ZERO(1), False), (ZERO(D), ZERO(2 * D)[::2], False),
    (ZERO(T, D, dtype=ROWS), ZERO(T, D, dtype=ROWS), True), (ZERO(T, D, dtype=ROWS), ZERO(T, D + 2, dtype=ROWS)[:, :D], True),
    (ZERO(T, D, dtype=ROWS), ZERO(T * D, dtype=ROWS), True), (ZERO(T, D, dtype=ROWS), ZERO(D), False), (ZERO(T, D, dtype=ROWS), ZERO(1, D), False),
    (ZERO(T, D, dtype=ROWS), ZERO(T, D + 2, dtype=ROWS), False), (ZERO(T, D, dtype=ROWS), ZERO(T, 1), False), (None, None, True), (4096, 4096, True)])
def test_gradients_of_gates(monkeypatch, gate, grad, ok):
    if grad is None:
        grad = 0
    got = _calls(monkeypatch, gate, grad)
    if not ok:
        assert got == rg.MOE_ERR_INVALID_ARG
    else:
        (name, args), = got
        per_row = torch.is_tensor(gate) and gate.dim() > 1
        assert name == "moe_norm_bwd" and args[16].gate_stride == (0 if not per_row else grad.stride(0) if grad.dim() > 1 else D)
