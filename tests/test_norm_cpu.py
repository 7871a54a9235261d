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
