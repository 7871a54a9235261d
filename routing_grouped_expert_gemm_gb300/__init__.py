"""Python binding of the MoE-layer forward C ABI (``include/moe.h``).

Argument marshalling only: every step of the forward runs in the CUDA library
``_lib/libmoe_gb300.so`` (built by ``build.py``).  There is no fallback: if the
library is missing or cannot be loaded, every entry point raises.  PyTorch is
used only to hand over device pointers and streams.

Entry points keep the C names: ``moe_plan_create``, ``moe_plan_destroy``,
``moe_workspace_bytes``, ``moe_quantize_mxfp8``, ``moe_mxfp8_scale_bytes``,
``moe_fwd``, ``moe_bwd_workspace_bytes``, ``moe_bwd``, ``moe_get_status``,
``moe_get_phase_times``, ``moe_route_static``, ``moe_error_string``; the layer on a
given routing: ``moe_fwd_routed``, ``moe_bwd_routed``; routing from given logits: ``moe_route_plan_create``, ``moe_route_plan_destroy``,
``moe_route_workspace_bytes``, ``moe_route``, ``moe_route_bwd``; momentum and
orthogonalised updates: ``moe_muon_plan_create``, ``moe_muon_plan_destroy``,
``moe_muon_workspace_bytes``, ``moe_muon_update``, ``moe_muon_get_status``; the layer
for a few tokens: ``moe_decode_workspace_bytes``, ``moe_decode``, ``moe_decode_routed``; norms
around a block: ``moe_norm_plan_create``, ``moe_norm_plan_destroy``, ``moe_norm``,
``moe_norm_workspace_bytes``, ``moe_norm_bwd``.
"""
from __future__ import annotations

import ctypes
import os
import re

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libmoe_gb300.so")
if os.environ.get("MOE_TRACE_BUILD") == "1":  # profiling only: the MOE_TRACE variant of the same library
    LIB_PATH = os.path.join(_HERE, "_lib", "libmoe_gb300_trace.so")
elif os.environ.get("MOE_DEBUG_BUILD") == "1":  # debugging only: the MOE_DEBUG_LOG variant
    LIB_PATH = os.path.join(_HERE, "_lib", "libmoe_gb300_dbg.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "moe.h")
TESTING_HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "moe_testing.h")
# test hooks (one-tile probes of tensor-core encodings), a library of their own
TESTING_LIB_PATH = os.path.join(_HERE, "_lib", "libmoe_gb300_testing.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED_SHAPE = -2
MOE_ERR_WORKSPACE_TOO_SMALL = -3
MOE_ERR_CUDA = -4
MOE_ERR_UNSUPPORTED_DEVICE = -5
MOE_ERR_STATIC_SCRATCH_TOO_SMALL = -6
MOE_ROUTE_STATIC_MAX_TOKENS = 16384
MOE_DECODE_MAX_TOKENS = 64
MOE_STATUS_OK, MOE_STATUS_TIMEOUT, MOE_STATUS_SCHEDULE_INVALID, MOE_STATUS_STAGING_OVERFLOW = 0, 1, 2, 3
MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX = 0, 1
MOE_PREC_BF16, MOE_PREC_MXFP8 = 0, 1
MOE_DISPATCH_RING, MOE_DISPATCH_DIRECT, MOE_DISPATCH_SPREAD = 0, 1, 2
MOE_DTYPE_FP32, MOE_DTYPE_BF16, MOE_DTYPE_FP16 = 0, 1, 2
MOE_NORM_RMS, MOE_NORM_LAYER = 0, 1
_DTYPES = {"fp32": MOE_DTYPE_FP32, "bf16": MOE_DTYPE_BF16, "fp16": MOE_DTYPE_FP16}


class MoEError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {moe_error_string(code)} ({code})")


class moe_config(ctypes.Structure):
    _fields_ = [("T_max", ctypes.c_int64), ("D", ctypes.c_int64), ("I", ctypes.c_int64), ("E", ctypes.c_int64),
                ("k", ctypes.c_int64), ("I_s", ctypes.c_int64), ("score_fn", ctypes.c_int32),
                ("precision", ctypes.c_int32), ("minibatch", ctypes.c_int32), ("ring_slots", ctypes.c_int32),
                ("gather_ctas", ctypes.c_int32), ("gemm_ctas", ctypes.c_int32), ("lag", ctypes.c_int32),
                ("timeout_ms", ctypes.c_int32), ("dispatch", ctypes.c_int32), ("l2_prefetch", ctypes.c_int32),
                ("mma_pair", ctypes.c_int32), ("raster", ctypes.c_int32),
                ("test_unfilled_minibatch", ctypes.c_int32), ("clc", ctypes.c_int32),
                ("plain_launch", ctypes.c_int32), ("pad_odd_tiles", ctypes.c_int32)]


class moe_weights(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "W_router", "b_router", "W_up", "W_gate", "W_down", "W_up_scale", "W_gate_scale", "W_down_scale",
        "Ws_up", "Ws_gate", "Ws_down")]


class moe_grads(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "dx", "dW_router", "db_router", "dW_up", "dW_gate", "dW_down", "dWs_up", "dWs_gate", "dWs_down")]


class moe_outputs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "out", "topk_idx", "topk_w", "expert_counts", "expert_offsets", "sched", "route_row")]


class moe_route_config(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int64), ("k", ctypes.c_int64), ("n_group", ctypes.c_int64),
                ("topk_group", ctypes.c_int64), ("score_fn", ctypes.c_int32), ("logits_dtype", ctypes.c_int32),
                ("group_top", ctypes.c_int32), ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float)]


class moe_muon_config(ctypes.Structure):
    _fields_ = [("count", ctypes.c_int64), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("steps", ctypes.c_int32), ("grad_dtype", ctypes.c_int32), ("a", ctypes.c_float), ("b", ctypes.c_float),
                ("c", ctypes.c_float), ("timeout_ms", ctypes.c_int32)]


class moe_norm_config(ctypes.Structure):
    _fields_ = [("D", ctypes.c_int64), ("kind", ctypes.c_int32), ("post", ctypes.c_int32), ("pre", ctypes.c_int32),
                ("stream_dtype", ctypes.c_int32), ("branch_dtype", ctypes.c_int32), ("param_dtype", ctypes.c_int32),
                ("eps", ctypes.c_float), ("weight_offset", ctypes.c_float), ("x_scale", ctypes.c_float),
                ("o_scale", ctypes.c_float)]


class moe_norm_params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("post_weight", "post_bias", "pre_weight", "pre_bias", "gate")] + [
        ("gate_stride", ctypes.c_int64)]


moe_norm_grads = moe_norm_params  # the same fields: gradients of the parameters


_lib = None


def lib():
    """The loaded CUDA library (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"CUDA library not built: {LIB_PATH} is missing (run routing_grouped_expert_gemm_gb300/build.py)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, sz, i32p = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.POINTER(ctypes.c_int)
    L.moe_plan_create.argtypes = [ctypes.POINTER(moe_config), ctypes.POINTER(vp)]
    L.moe_plan_create.restype = ctypes.c_int
    L.moe_plan_destroy.argtypes = [vp]
    L.moe_plan_destroy.restype = ctypes.c_int
    L.moe_workspace_bytes.argtypes = [vp, i64]
    L.moe_workspace_bytes.restype = sz
    L.moe_quantize_mxfp8.argtypes = [vp, vp, i64, i64, vp, vp, vp]
    L.moe_quantize_mxfp8.restype = ctypes.c_int
    L.moe_mxfp8_scale_bytes.argtypes = [i64, i64]
    L.moe_mxfp8_scale_bytes.restype = sz
    L.moe_fwd.argtypes = [vp, i64, vp, ctypes.POINTER(moe_weights), ctypes.POINTER(moe_outputs), vp, sz, vp]
    L.moe_fwd.restype = ctypes.c_int
    L.moe_get_status.argtypes = [vp, vp, i32p, vp]
    L.moe_get_status.restype = ctypes.c_int
    L.moe_plan_set_timing_events.argtypes = [vp, ctypes.POINTER(vp)]
    L.moe_plan_set_timing_events.restype = ctypes.c_int
    L.moe_plan_set_bwd_timing_events.argtypes = [vp, ctypes.POINTER(vp)]
    L.moe_plan_set_bwd_timing_events.restype = ctypes.c_int
    L.moe_bwd_workspace_bytes.argtypes = [vp, i64]
    L.moe_bwd_workspace_bytes.restype = sz
    L.moe_bwd.argtypes = [vp, i64, vp, ctypes.POINTER(moe_weights), vp, vp, ctypes.POINTER(moe_grads), vp, sz, vp]
    L.moe_bwd.restype = ctypes.c_int
    L.moe_get_phase_times.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_double), vp]
    L.moe_get_phase_times.restype = ctypes.c_int
    L.moe_route_static.argtypes = [vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_route_static.restype = ctypes.c_int
    L.moe_route_static_scratch_bytes.argtypes = []
    L.moe_route_static_scratch_bytes.restype = sz
    L.moe_fwd_routed.argtypes = [vp, i64, vp, ctypes.POINTER(moe_weights), vp, vp, ctypes.POINTER(moe_outputs), vp, sz,
                                 vp]
    L.moe_fwd_routed.restype = ctypes.c_int
    L.moe_bwd_routed.argtypes = [vp, i64, vp, ctypes.POINTER(moe_weights), vp, vp, ctypes.POINTER(moe_grads), vp, vp, sz,
                                 vp]
    L.moe_bwd_routed.restype = ctypes.c_int
    L.moe_route_plan_create.argtypes = [ctypes.POINTER(moe_route_config), ctypes.POINTER(vp)]
    L.moe_route_plan_create.restype = ctypes.c_int
    L.moe_route_plan_destroy.argtypes = [vp]
    L.moe_route_plan_destroy.restype = ctypes.c_int
    L.moe_route_workspace_bytes.argtypes = [vp, i64]
    L.moe_route_workspace_bytes.restype = sz
    L.moe_route.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp, vp, vp, sz, vp]
    L.moe_route.restype = ctypes.c_int
    L.moe_route_bwd.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp, i64, vp]
    L.moe_route_bwd.restype = ctypes.c_int
    L.moe_muon_plan_create.argtypes = [ctypes.POINTER(moe_muon_config), ctypes.POINTER(vp)]
    L.moe_muon_plan_create.restype = ctypes.c_int
    L.moe_muon_plan_destroy.argtypes = [vp]
    L.moe_muon_plan_destroy.restype = ctypes.c_int
    L.moe_muon_workspace_bytes.argtypes = [vp]
    L.moe_muon_workspace_bytes.restype = sz
    L.moe_muon_update.argtypes = [vp, vp, i64, i64, vp, ctypes.c_float, ctypes.c_int32, ctypes.c_float, vp, vp, sz, vp]
    L.moe_muon_update.restype = ctypes.c_int
    L.moe_muon_get_status.argtypes = [vp, vp, i32p, vp]
    L.moe_muon_get_status.restype = ctypes.c_int
    L.moe_decode_workspace_bytes.argtypes = [vp, i64]
    L.moe_decode_workspace_bytes.restype = sz
    L.moe_decode.argtypes = [vp, i64, vp, ctypes.POINTER(moe_weights), vp, vp, vp, vp, sz, vp]
    L.moe_decode.restype = ctypes.c_int
    L.moe_decode_routed.argtypes = [vp, i64, vp, ctypes.POINTER(moe_weights), vp, vp, vp, vp, sz, vp]
    L.moe_decode_routed.restype = ctypes.c_int
    L.moe_norm_plan_create.argtypes = [ctypes.POINTER(moe_norm_config), ctypes.POINTER(vp)]
    L.moe_norm_plan_create.restype = ctypes.c_int
    L.moe_norm_plan_destroy.argtypes = [vp]
    L.moe_norm_plan_destroy.restype = ctypes.c_int
    L.moe_norm_workspace_bytes.argtypes = [vp, i64]
    L.moe_norm_workspace_bytes.restype = sz
    L.moe_norm.argtypes = [vp, i64, ctypes.POINTER(moe_norm_params)] + [vp, i64] * 4 + [vp, vp]
    L.moe_norm.restype = ctypes.c_int
    L.moe_norm_bwd.argtypes = [vp, i64, ctypes.POINTER(moe_norm_params), vp] + [vp, i64] * 6 + [
        ctypes.POINTER(moe_norm_grads), vp, sz, vp]
    L.moe_norm_bwd.restype = ctypes.c_int
    L.moe_error_string.argtypes = [ctypes.c_int]
    L.moe_error_string.restype = ctypes.c_char_p
    _lib = L
    return L


_testing_lib = None


def testing_lib():
    """The test-hook library (one-tile probes; raises if it was not built)."""
    global _testing_lib
    if _testing_lib is not None:
        return _testing_lib
    if not os.path.exists(TESTING_LIB_PATH):
        raise RuntimeError(f"test-hook library not built: {TESTING_LIB_PATH} is missing")
    L = ctypes.CDLL(TESTING_LIB_PATH)
    vp = ctypes.c_void_p
    L.moe_testing_mx_tile.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp]
    L.moe_testing_mx_tile.restype = ctypes.c_int
    L.moe_testing_pair_tile.argtypes = [vp, vp, vp, vp, ctypes.c_int, vp]
    L.moe_testing_pair_tile.restype = ctypes.c_int
    L.moe_testing_pair_mma_time.argtypes = [vp, vp, vp, vp, ctypes.c_int, ctypes.c_int, vp, vp]
    L.moe_testing_pair_mma_time.restype = ctypes.c_int
    L.moe_testing_pair_mx_tile.argtypes = [vp, vp, vp, vp, vp, ctypes.c_int, vp]
    L.moe_testing_pair_mx_tile.restype = ctypes.c_int
    L.moe_testing_mn_tile.argtypes = [vp, vp, vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                      ctypes.c_int, vp]
    L.moe_testing_mn_tile.restype = ctypes.c_int
    L.moe_testing_tma3d_load.argtypes = [vp, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, vp, vp, vp]
    L.moe_testing_tma3d_load.restype = ctypes.c_int
    _testing_lib = L
    return L


def declared_functions(header: str | None = None) -> list[str]:
    """Function names declared in one header (default: include/moe.h, the ABI)."""
    text = open(header or HEADER_PATH).read()
    return sorted(set(re.findall(r"^\s*(?:int|size_t|const char\*)\s+(moe_\w+)\s*\(", text, flags=re.M)))


def _ptr(v) -> int | None:
    if v is None or isinstance(v, int):
        return v
    return v.data_ptr()  # torch tensor


def _current_stream() -> int:
    """The current stream's handle without a Stream object (0.2 us a call instead of 3)."""
    global _current_stream
    import torch

    raw, device = torch._C._cuda_getCurrentRawStream, torch.cuda.current_device
    _current_stream = lambda: raw(device())  # noqa: E731  (without the import from now on)
    return _current_stream()


def _stream(stream) -> int | None:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def moe_error_string(code: int) -> str:
    return lib().moe_error_string(code).decode()


class Plan:
    """Owns a moe_plan*; released by moe_plan_destroy (or garbage collection)."""

    def __init__(self, handle: int, cfg: moe_config):
        self.handle = handle
        self.cfg = cfg

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.moe_plan_destroy(self.handle)
            self.handle = None


def moe_plan_create(T_max, D, I, E, k, I_s=0, score_fn=MOE_SCORE_SIGMOID, precision=MOE_PREC_BF16, minibatch=0,
                    ring_slots=0, gather_ctas=0, gemm_ctas=0, lag=1, timeout_ms=0, dispatch=MOE_DISPATCH_RING,
                    l2_prefetch=0, mma_pair=0, raster=0, test_unfilled_minibatch=0, clc=0, plain_launch=0,
                    pad_odd_tiles=0) -> Plan:
    if isinstance(score_fn, str):
        score_fn = {"sigmoid": MOE_SCORE_SIGMOID, "softmax": MOE_SCORE_SOFTMAX}[score_fn]
    if isinstance(precision, str):
        precision = {"bf16": MOE_PREC_BF16, "mxfp8": MOE_PREC_MXFP8}[precision]
    if isinstance(dispatch, str):
        dispatch = {"ring": MOE_DISPATCH_RING, "direct": MOE_DISPATCH_DIRECT, "spread": MOE_DISPATCH_SPREAD}[dispatch]
    cfg = moe_config(T_max, D, I, E, k, I_s, score_fn, precision, minibatch, ring_slots, gather_ctas, gemm_ctas,
                     lag, timeout_ms, dispatch, l2_prefetch, mma_pair, raster, test_unfilled_minibatch, clc, plain_launch,
                     pad_odd_tiles)
    h = ctypes.c_void_p()
    rc = lib().moe_plan_create(ctypes.byref(cfg), ctypes.byref(h))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_plan_create")
    return Plan(h.value, cfg)


def moe_plan_destroy(plan: Plan) -> None:
    if plan.handle:
        lib().moe_plan_destroy(plan.handle)
        plan.handle = None


def moe_workspace_bytes(plan: Plan, T: int) -> int:
    return int(lib().moe_workspace_bytes(plan.handle, T))


def moe_mxfp8_scale_bytes(rows: int, K: int) -> int:
    return int(lib().moe_mxfp8_scale_bytes(rows, K))


def moe_quantize_mxfp8(plan: Plan, W, rows: int, K: int, q, scales, stream=None) -> None:
    rc = lib().moe_quantize_mxfp8(plan.handle, _ptr(W), rows, K, _ptr(q), _ptr(scales), _stream(stream))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_quantize_mxfp8")


def moe_fwd(plan: Plan, T: int, x, weights: dict, out, workspace, workspace_bytes: int | None = None,
            topk_idx=None, topk_w=None, expert_counts=None, expert_offsets=None, sched=None, route_row=None,
            stream=None) -> None:
    """weights: dict with keys of moe_weights (W_router, b_router, W_up, ...)."""
    w = moe_weights(**{k: _ptr(v) for k, v in weights.items()})
    o = moe_outputs(_ptr(out), _ptr(topk_idx), _ptr(topk_w), _ptr(expert_counts), _ptr(expert_offsets),
                    _ptr(sched), _ptr(route_row))
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    rc = lib().moe_fwd(plan.handle, T, _ptr(x), ctypes.byref(w), ctypes.byref(o), _ptr(workspace),
                       workspace_bytes, _stream(stream))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_fwd")


def moe_bwd_workspace_bytes(plan: Plan, T: int) -> int:
    return int(lib().moe_bwd_workspace_bytes(plan.handle, T))


def moe_bwd(plan: Plan, T: int, x, weights: dict, dO, fwd_workspace, grads: dict, workspace,
            workspace_bytes: int | None = None, stream=None) -> None:
    """Backward pass: ``grads`` has keys of moe_grads (dx, dW_router, db_router,
    dW_up, dW_gate, dW_down, dWs_up, dWs_gate, dWs_down); ``fwd_workspace`` is
    the workspace of the moe_fwd call on the same x and weights."""
    w = moe_weights(**{k: _ptr(v) for k, v in weights.items()})
    g = moe_grads(**{k: _ptr(v) for k, v in grads.items()})
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    rc = lib().moe_bwd(plan.handle, T, _ptr(x), ctypes.byref(w), _ptr(dO), _ptr(fwd_workspace), ctypes.byref(g),
                       _ptr(workspace), workspace_bytes, _stream(stream))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_bwd")


def moe_fwd_routed(plan: Plan, T: int, x, weights: dict, topk_idx, topk_w, out, workspace,
                   workspace_bytes: int | None = None, expert_counts=None, expert_offsets=None, sched=None,
                   route_row=None, stream=None) -> None:
    """The forward with its routing given: ``topk_idx`` [T, k] int32 (-1: an
    empty slot) and ``topk_w`` [T, k] fp32, as ``moe_route`` writes them."""
    w = moe_weights(**{k: _ptr(v) for k, v in weights.items()})
    o = moe_outputs(_ptr(out), None, None, _ptr(expert_counts), _ptr(expert_offsets), _ptr(sched), _ptr(route_row))
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    rc = lib().moe_fwd_routed(plan.handle, T, _ptr(x), ctypes.byref(w), _ptr(topk_idx), _ptr(topk_w), ctypes.byref(o),
                              _ptr(workspace), workspace_bytes, _stream(stream))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_fwd_routed")


def moe_bwd_routed(plan: Plan, T: int, x, weights: dict, dO, fwd_workspace, grads: dict, dtopk_w, workspace,
                   workspace_bytes: int | None = None, stream=None) -> None:
    """Backward of ``moe_fwd_routed``: ``grads`` as for ``moe_bwd`` without the
    router's, and the gradient of ``topk_w`` in ``dtopk_w`` [T, k] fp32."""
    w = moe_weights(**{k: _ptr(v) for k, v in weights.items()})
    g = moe_grads(**{k: _ptr(v) for k, v in grads.items()})
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    rc = lib().moe_bwd_routed(plan.handle, T, _ptr(x), ctypes.byref(w), _ptr(dO), _ptr(fwd_workspace), ctypes.byref(g),
                              _ptr(dtopk_w), _ptr(workspace), workspace_bytes, _stream(stream))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_bwd_routed")


def moe_get_status(plan: Plan, workspace, stream=None) -> int:
    st = ctypes.c_int(-1)
    rc = lib().moe_get_status(plan.handle, _ptr(workspace), ctypes.byref(st), _stream(stream))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_get_status")
    return st.value


def moe_get_phase_times(plan: Plan, workspace, stream=None) -> dict:
    """Phase stamps of the last forward on ``workspace`` (ms after the persistent
    kernel's start; None where the phase did not happen)."""
    arr = (ctypes.c_double * 3)()
    rc = lib().moe_get_phase_times(plan.handle, _ptr(workspace), arr, _stream(stream))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_get_phase_times")
    keys = ("last_fill", "combine_start", "combine_end")
    return {k: (None if v < 0 else float(v)) for k, v in zip(keys, arr)}


def moe_plan_set_timing_events(plan: Plan, events) -> None:
    """events: four torch.cuda.Event (created with enable_timing) or None."""
    if events is None:
        rc = lib().moe_plan_set_timing_events(plan.handle, None)
    else:
        arr = (ctypes.c_void_p * 4)(*[int(e.cuda_event) for e in events])
        rc = lib().moe_plan_set_timing_events(plan.handle, arr)
    if rc != MOE_OK:
        raise MoEError(rc, "moe_plan_set_timing_events")


def moe_plan_set_bwd_timing_events(plan: Plan, events) -> None:
    """events: five torch.cuda.Event (created with enable_timing) or None."""
    if events is None:
        rc = lib().moe_plan_set_bwd_timing_events(plan.handle, None)
    else:
        arr = (ctypes.c_void_p * 5)(*[int(e.cuda_event) for e in events])
        rc = lib().moe_plan_set_bwd_timing_events(plan.handle, arr)
    if rc != MOE_OK:
        raise MoEError(rc, "moe_plan_set_bwd_timing_events")


def moe_route_static(plan: Plan, T: int, x, W_router, b_router, topk_idx, topk_w, expert_counts, expert_offsets,
                     sched, route_row, device_status=None, stream=None) -> None:
    """Routing stage (top-k, g, counts, offsets, schedule table) that allocates
    nothing: its scratch is a fixed array inside the library, for callers that
    cannot call cudaMalloc.  Calls that overlap on the GPU race on that array."""
    rc = lib().moe_route_static(plan.handle, T, _ptr(x), _ptr(W_router), _ptr(b_router), _ptr(topk_idx),
                                _ptr(topk_w), _ptr(expert_counts), _ptr(expert_offsets), _ptr(sched),
                                _ptr(route_row), _ptr(device_status), _stream(stream))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_route_static")


def moe_route_static_scratch_bytes() -> int:
    return int(lib().moe_route_static_scratch_bytes())


class RoutePlan:
    """Owns a moe_route_plan*; released by moe_route_plan_destroy (or garbage collection)."""

    def __init__(self, handle: int, cfg: moe_route_config):
        self.handle = handle
        self.cfg = cfg

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.moe_route_plan_destroy(self.handle)
            self.handle = None


def moe_route_plan_create(E, k, score_fn=MOE_SCORE_SIGMOID, logits_dtype=MOE_DTYPE_FP32, n_group=1, topk_group=1,
                          group_top=2, renormalize=True, scale=1.0) -> RoutePlan:
    """Plan of the general router (``moe_route``, ``moe_route_bwd``)."""
    if isinstance(score_fn, str):
        score_fn = {"sigmoid": MOE_SCORE_SIGMOID, "softmax": MOE_SCORE_SOFTMAX}[score_fn]
    if isinstance(logits_dtype, str):
        logits_dtype = _DTYPES[logits_dtype]
    cfg = moe_route_config(E, k, n_group, topk_group, score_fn, logits_dtype, group_top, int(renormalize), scale)
    h = ctypes.c_void_p()
    rc = lib().moe_route_plan_create(ctypes.byref(cfg), ctypes.byref(h))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_route_plan_create")
    return RoutePlan(h.value, cfg)


def moe_route_plan_destroy(plan: RoutePlan) -> None:
    if plan.handle:
        lib().moe_route_plan_destroy(plan.handle)
        plan.handle = None


def moe_route_workspace_bytes(plan: RoutePlan, T: int) -> int:
    return int(lib().moe_route_workspace_bytes(plan.handle, T))


def moe_route(plan: RoutePlan, T: int, logits, bias, topk_idx, topk_w, expert_counts=None, prob_sum=None,
              workspace=None, workspace_bytes: int | None = None, logits_stride: int = 0, stream=None) -> None:
    """Scores, selection (bias, groups, top-k) and weights of ``logits`` [T, E];
    ``expert_counts`` and ``prob_sum`` are the sums a balance bias or loss needs."""
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().moe_route(plan.handle, T, _ptr(logits), logits_stride, _ptr(bias), _ptr(topk_idx), _ptr(topk_w),
                         _ptr(expert_counts), _ptr(prob_sum), _ptr(workspace), workspace_bytes, _stream(stream))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_route")


def moe_route_bwd(plan: RoutePlan, T: int, logits, topk_idx, dtopk_w, dlogits, dprob_sum=None, logits_stride: int = 0,
                  dlogits_stride: int = 0, stream=None) -> None:
    """Gradient of the logits from those of ``topk_w`` and (optionally) ``prob_sum``."""
    rc = lib().moe_route_bwd(plan.handle, T, _ptr(logits), logits_stride, _ptr(topk_idx), _ptr(dtopk_w),
                             _ptr(dprob_sum), _ptr(dlogits), dlogits_stride, _stream(stream))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_route_bwd")


class MuonPlan:
    """Owns a moe_muon_plan*; released by moe_muon_plan_destroy (or garbage collection)."""

    def __init__(self, handle: int, cfg: moe_muon_config):
        self.handle = handle
        self.cfg = cfg

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.moe_muon_plan_destroy(self.handle)
            self.handle = None


def moe_muon_plan_create(count, rows, cols, steps=5, grad_dtype=MOE_DTYPE_BF16, coefficients=(3.4445, -4.7750, 2.0315),
                         timeout_ms=0) -> MuonPlan:
    """Plan of ``moe_muon_update`` for a stack of ``count`` matrices of rows x cols."""
    if isinstance(grad_dtype, str):
        grad_dtype = _DTYPES[grad_dtype]
    cfg = moe_muon_config(count, rows, cols, steps, grad_dtype, *coefficients, timeout_ms)
    h = ctypes.c_void_p()
    rc = lib().moe_muon_plan_create(ctypes.byref(cfg), ctypes.byref(h))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_muon_plan_create")
    return MuonPlan(h.value, cfg)


def moe_muon_plan_destroy(plan: MuonPlan) -> None:
    if plan.handle:
        lib().moe_muon_plan_destroy(plan.handle)
        plan.handle = None


def moe_muon_workspace_bytes(plan: MuonPlan) -> int:
    return int(lib().moe_muon_workspace_bytes(plan.handle))


def moe_muon_update(plan: MuonPlan, grad, momentum, update, workspace, workspace_bytes: int | None = None, mu=0.95,
                    nesterov=True, scale=1.0, grad_row_stride: int = 0, grad_stride: int = 0, stream=None) -> None:
    """Advance ``momentum`` (fp32, in place; None = no momentum) by ``grad`` and
    write the orthogonalised update of every matrix, times ``scale``, to ``update`` (bf16)."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    rc = lib().moe_muon_update(plan.handle, _ptr(grad), grad_row_stride, grad_stride, _ptr(momentum), mu, int(nesterov),
                               scale, _ptr(update), _ptr(workspace), workspace_bytes, _stream(stream))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_muon_update")


def moe_muon_get_status(plan: MuonPlan, workspace, stream=None) -> int:
    st = ctypes.c_int(-1)
    rc = lib().moe_muon_get_status(plan.handle, _ptr(workspace), ctypes.byref(st), _stream(stream))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_muon_get_status")
    return st.value


def moe_decode_workspace_bytes(plan: Plan, T: int) -> int:
    return int(lib().moe_decode_workspace_bytes(plan.handle, T))


def moe_decode(plan: Plan, T: int, x, weights: dict, out, workspace, workspace_bytes: int | None = None, topk_idx=None,
               topk_w=None, stream=None) -> None:
    """``moe_fwd``'s layer for at most MOE_DECODE_MAX_TOKENS tokens, in one launch bound by the experts' weights."""
    w = moe_weights(**{k: _ptr(v) for k, v in weights.items()})
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    rc = lib().moe_decode(plan.handle, T, _ptr(x), w, _ptr(out), _ptr(topk_idx), _ptr(topk_w), _ptr(workspace),
                          workspace_bytes, _stream(stream))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_decode")


def moe_decode_routed(plan: Plan, T: int, x, weights: dict, topk_idx, topk_w, out, workspace,
                      workspace_bytes: int | None = None, stream=None) -> None:
    """``moe_decode`` with its routing given: ``topk_idx`` [T, k] int32 (-1: an empty slot) and ``topk_w`` [T, k] fp32."""
    w = moe_weights(**{k: _ptr(v) for k, v in weights.items()})
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    rc = lib().moe_decode_routed(plan.handle, T, _ptr(x), w, _ptr(topk_idx), _ptr(topk_w), _ptr(out), _ptr(workspace),
                                 workspace_bytes, _stream(stream))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_decode_routed")


class NormPlan:
    """Owns a moe_norm_plan*; released by moe_norm_plan_destroy (or garbage collection)."""

    def __init__(self, handle: int, cfg: moe_norm_config):
        self.handle = handle
        self.cfg = cfg

    def __del__(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.moe_norm_plan_destroy(self.handle)
            self.handle = None


def moe_norm_plan_create(D, kind=MOE_NORM_RMS, post=True, pre=True, stream_dtype=MOE_DTYPE_BF16, branch_dtype=MOE_DTYPE_BF16,
                         param_dtype=MOE_DTYPE_FP32, eps=1e-6, weight_offset=0.0, x_scale=1.0, o_scale=1.0) -> NormPlan:
    """Plan of ``moe_norm`` and ``moe_norm_bwd`` for rows of D elements."""
    if isinstance(kind, str):
        kind = {"rms": MOE_NORM_RMS, "layer": MOE_NORM_LAYER}[kind]
    stream_dtype, branch_dtype, param_dtype = (_DTYPES[d] if isinstance(d, str) else d
                                               for d in (stream_dtype, branch_dtype, param_dtype))
    cfg = moe_norm_config(D, kind, int(post), int(pre), stream_dtype, branch_dtype, param_dtype, eps, weight_offset,
                          x_scale, o_scale)
    h = ctypes.c_void_p()
    rc = lib().moe_norm_plan_create(ctypes.byref(cfg), ctypes.byref(h))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_norm_plan_create")
    return NormPlan(h.value, cfg)


def moe_norm_plan_destroy(plan: NormPlan) -> None:
    if plan.handle:
        lib().moe_norm_plan_destroy(plan.handle)
        plan.handle = None


def moe_norm_workspace_bytes(plan: NormPlan, T: int) -> int:
    return int(lib().moe_norm_workspace_bytes(plan.handle, T))


def _row_stride(t) -> int:
    """Elements between the rows of a tensor [T, D]: 0 (rows of D) where it is
    contiguous or only a pointer, else its stride."""
    if t is None or isinstance(t, int) or t.is_contiguous():
        return 0
    if t.dim() != 2 or t.stride(1) != 1 or t.stride(0) <= 0:
        raise MoEError(MOE_ERR_INVALID_ARG, "rows of a tensor that is neither contiguous nor [T, D] with a row stride")
    return t.stride(0)


def _gate_stride(gate, D: int, T: int) -> int:
    """0: one gate per channel, [D]; else the stride of a gate per row, [T, D] (its
    rows may have further dimensions).  Any other shape is refused: read as
    either, it would be read past its end."""
    if gate is None or isinstance(gate, int):
        return 0
    if gate.dim() == 1 and gate.shape[0] == D and gate.is_contiguous():
        return 0
    if gate.dim() < 2 or gate.shape[-1] != D or gate.numel() < T * D:
        raise MoEError(MOE_ERR_INVALID_ARG, "a gate that is neither [D] nor [T, D]")
    return _row_stride(gate) or D


def _norm_args(plan: NormPlan, params: dict, gate_stride: int) -> moe_norm_params:
    get = params.get
    return moe_norm_params(_ptr(get("post_weight")), _ptr(get("post_bias")), _ptr(get("pre_weight")), _ptr(get("pre_bias")),
                           _ptr(get("gate")), get("gate_stride") or gate_stride)


def _gate_grad_stride(grad, D: int, T: int, per_row: bool) -> int:
    """The same of a gate's gradient: [T, D] for a gate per row, else [D]."""
    if grad is None or isinstance(grad, int):
        return 0
    if not per_row:
        if grad.numel() != D or not grad.is_contiguous():
            raise MoEError(MOE_ERR_INVALID_ARG, "the gradient of a gate [D] that is not [D]")
        return 0
    if grad.numel() < T * D or (grad.dim() > 1 and grad.shape[-1] != D):
        raise MoEError(MOE_ERR_INVALID_ARG, "the gradient of a gate [T, D] that is not [T, D]")
    return _row_stride(grad) or D


def moe_norm(plan: NormPlan, T: int, params: dict, x=None, o=None, y=None, h=None, stats=None, stream=None) -> None:
    """z = N(o), y = x_scale x + o_scale gate z, h = N(y).  ``params``: post_weight,
    post_bias, pre_weight, pre_bias and gate ([D], or [T, D] for a gate per row; no
    other shape), each optional.  Rows may be further apart than D (a view of a wider
    tensor); ``stats`` [T, 4] fp32 keeps what ``moe_norm_bwd`` needs."""
    q = _norm_args(plan, params, _gate_stride(params.get("gate"), plan.cfg.D, T))
    rc = lib().moe_norm(plan.handle, T, q, _ptr(x), _row_stride(x), _ptr(o), _row_stride(o), _ptr(y), _row_stride(y),
                        _ptr(h), _row_stride(h), _ptr(stats), _stream(stream))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_norm")


def moe_norm_bwd(plan: NormPlan, T: int, params: dict, stats, grads: dict, o=None, y=None, dy=None, dh=None, dx=None,
                 do=None, workspace=None, workspace_bytes: int | None = None, stream=None) -> None:
    """The gradients of ``moe_norm``: of the rows in ``dx`` and ``do``, of the parameters
    in ``grads`` (the keys of ``params``: fp32 [D]; a gate per row: [T, D] of the branch's type)."""
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    q = _norm_args(plan, params, _gate_stride(params.get("gate"), plan.cfg.D, T))
    g = _norm_args(plan, grads, _gate_grad_stride(grads.get("gate"), plan.cfg.D, T, q.gate_stride != 0))
    rc = lib().moe_norm_bwd(plan.handle, T, q, _ptr(stats), _ptr(o), _row_stride(o), _ptr(y), _row_stride(y), _ptr(dy),
                            _row_stride(dy), _ptr(dh), _row_stride(dh), _ptr(dx), _row_stride(dx), _ptr(do),
                            _row_stride(do), g, _ptr(workspace), workspace_bytes, _stream(stream))
    if rc != MOE_OK:
        raise MoEError(rc, "moe_norm_bwd")
