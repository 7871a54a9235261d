"""moe_decode without a GPU: null arguments."""
import pytest

import routing_grouped_expert_gemm_gb300 as rg
from routing_grouped_expert_gemm_gb300 import build as rgbuild


@pytest.fixture(scope="module")
def L():
    rgbuild.build()
    return rg.lib()


def test_null_arguments(L):
    assert L.moe_decode_workspace_bytes(None, 1) == 0
    assert L.moe_decode(None, 1, None, None, None, None, None, None, 0, None) == rg.MOE_ERR_INVALID_ARG
    assert L.moe_decode_routed(None, 1, None, None, None, None, None, None, 0, None) == rg.MOE_ERR_INVALID_ARG
    assert rg.MOE_DECODE_MAX_TOKENS == 64
