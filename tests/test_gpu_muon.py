"""moe_muon_update against a plain fp64 implementation.

Tolerances, relative to the Frobenius norm of the result.  Operands of a
product are rounded to fp16 (relative 2^-11 at most, 2^-11 / sqrt(3) in the
root mean square over a binade's worst end): X's hi in both products, A and B
once each, four roundings a step, each multiplied by what the step does to its
operand (|a| + |b| + |c| = 10.3 at worst, the terms cancelling to 1); errors of
one step pass the next ones with factors near 1.  Five steps of four roundings
add as independent errors: sqrt(20) * 2^-11 / sqrt(3) = 1.3e-3 at unit gain,
and twice that is allowed; then the result's own rounding to bf16 (2^-8 at
most per element, below 2^-9 in the root mean square)."""
import numpy as np
import pytest
import torch

import routing_grouped_expert_gemm_gb300 as rg

COEFS = (3.4445, -4.7750, 2.0315)
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
TOL = 2 * np.sqrt(20.0) * 2.0 ** -11 / np.sqrt(3.0) + 2.0 ** -9


def plain(grad, mom, mu=0.95, nesterov=True, steps=5, coefs=COEFS, scale=1.0):
    """fp64, matrix by matrix; returns (update, momentum)."""
    a, b, c = (float(np.float32(v)) for v in coefs)
    mu, scale = float(np.float32(mu)), float(np.float32(scale))
    g = grad.double()
    m = None
    if mom is not None:
        m = mu * mom.double() + g
        g = g + mu * m if nesterov else m
    out = torch.zeros_like(g)
    for i in range(g.shape[0]):
        n = torch.linalg.matrix_norm(g[i])
        if float(n) == 0.0:
            continue
        x = g[i] / n
        for _ in range(steps):
            y = x @ x.T if x.shape[0] <= x.shape[1] else x.T @ x
            p = b * y + c * (y @ y)
            x = a * x + (p @ x if x.shape[0] <= x.shape[1] else x @ p)
        out[i] = scale * x
    return out, m


def stack(count, rows, cols, kind, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if kind == "flat":
        return torch.randn(count, rows, cols, generator=g, device="cuda")
    r = max(1, min(rows, cols) // 4)
    u = torch.randn(count, rows, r, generator=g, device="cuda")
    v = torch.randn(count, r, cols, generator=g, device="cuda")
    if kind == "low rank":
        return u @ v
    d = torch.arange(1, r + 1, device="cuda", dtype=torch.float32) ** -1.0
    return (u * d) @ v + 1e-2 * torch.randn(count, rows, cols, generator=g, device="cuda")


def run(grad, mom, dtype, count, rows, cols, **kw):
    plan_kw = {k: kw.pop(k) for k in ("steps", "coefficients", "timeout_ms") if k in kw}
    plan = rg.moe_muon_plan_create(count, rows, cols, grad_dtype=dtype, **plan_kw)
    ws = torch.full((rg.moe_muon_workspace_bytes(plan),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in every type
    out = torch.full((count, rows, cols), float("nan"), dtype=torch.bfloat16, device="cuda")
    rg.moe_muon_update(plan, grad, mom, out, ws, **kw)
    assert rg.moe_muon_get_status(plan, ws) == rg.MOE_STATUS_OK
    return out


def rel(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


SHAPES = [(1, 1, 1), (2, 1, 9), (2, 7, 1), (5, 8, 8), (3, 33, 65), (2, 64, 64), (4, 100, 30), (2, 128, 256), (2, 255, 257),
          (1, 257, 255), (3, 300, 200), (1, 512, 1000), (1, 1031, 517), (700, 16, 24), (1, 24, 5000), (1, 5000, 24)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["flat", "decaying", "low rank"])
@pytest.mark.parametrize("count,rows,cols", SHAPES)
def test_update_matches_fp64(count, rows, cols, kind):
    grad = stack(count, rows, cols, kind, rows * 7 + cols)
    mom = stack(count, rows, cols, kind, rows + cols + 1) * 3
    ref, rm = plain(grad, mom, scale=0.2)
    out = run(grad, mom, "fp32", count, rows, cols, scale=0.2)
    assert rel(out, ref) <= TOL
    # one product and one sum in fp32
    assert float((mom.double() - rm).abs().max()) <= 2 ** -23 * float(rm.abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("momentum", [True, False])
def test_types_and_momentum_forms(dtype, nesterov, momentum):
    count, rows, cols = 3, 160, 120
    grad = (stack(count, rows, cols, "decaying", 1) * 1e-2).to(DTYPES[dtype])
    mom = stack(count, rows, cols, "flat", 2) * 1e-2 if momentum else None
    ref, rm = plain(grad, mom, mu=0.9, nesterov=nesterov)
    out = run(grad, mom, dtype, count, rows, cols, mu=0.9, nesterov=nesterov)
    assert rel(out, ref) <= TOL
    if momentum:
        assert float((mom.double() - rm).abs().max()) <= 2 ** -23 * float(rm.abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("steps,coefs", [(1, COEFS), (2, COEFS), (3, (1.875, -1.25, 0.375)), (10, (1.5, -0.5, 0.0))])
def test_steps_and_coefficients(steps, coefs):
    grad = stack(2, 90, 140, "flat", 4)
    ref, _ = plain(grad, None, steps=steps, coefs=coefs)
    out = run(grad, None, "fp32", 2, 90, 140, steps=steps, coefficients=coefs)
    # these coefficients damp errors (no gain above 1.9 a step); more steps add more roundings
    assert rel(out, ref) <= 2 * np.sqrt(4.0 * steps) * 2.0 ** -11 / np.sqrt(3.0) + 2.0 ** -9


@pytest.mark.gpu
def test_strided_gradients():
    count, rows, cols = 3, 48, 72
    for pad, extra, off in ((0, 0, 1), (8, 0, 0), (5, 3, 2), (24, 1, 4)):
        base = torch.randn(count * (rows + extra) * (cols + pad) + off, device="cuda").bfloat16()
        view = base[off:].view(count, rows + extra, cols + pad)[:, :rows, :cols]
        ref = run(view.contiguous(), None, "bf16", count, rows, cols)
        out = run(view.data_ptr(), None, "bf16", count, rows, cols, grad_row_stride=cols + pad,
                  grad_stride=(rows + extra) * (cols + pad))
        assert torch.equal(out, ref)


@pytest.mark.gpu
def test_zero_infinite_and_nan_matrices_keep_to_themselves():
    count, rows, cols = 5, 70, 90
    grad = stack(count, rows, cols, "flat", 8)
    ref = run(grad, None, "fp32", count, rows, cols)
    bad = grad.clone()
    bad[1] = 0
    bad[2, 3, 4] = float("inf")
    bad[3, 69, 89] = float("nan")
    out = run(bad, None, "fp32", count, rows, cols)
    assert torch.equal(out[0], ref[0]) and torch.equal(out[4], ref[4])
    assert bool((out[1] == 0).all()) and bool(torch.isnan(out[2]).all()) and bool(torch.isnan(out[3]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("power", [-140, -100, 60, 110])
def test_magnitudes_outside_the_squares_range(power):
    """Squares of these overflow or underflow fp32; the direction does not change
    (powers of two, though -140 leaves few bits: subnormal inputs)."""
    grad = torch.randint(-8, 9, (2, 40, 56), device="cuda").float()
    ref = run(grad, None, "fp32", 2, 40, 56)
    out = run(torch.ldexp(grad, torch.tensor(power, device="cuda")), None, "fp32", 2, 40, 56)
    assert torch.equal(out, ref)


@pytest.mark.gpu
def test_one_large_element_does_not_overflow():
    grad = torch.zeros(1, 64, 64, device="cuda")
    grad[0, 5, 9] = 3.0
    out = run(grad, None, "fp32", 1, 64, 64)
    want = 1.0
    for _ in range(5):
        want = COEFS[0] * want + COEFS[1] * want ** 3 + COEFS[2] * want ** 5
    assert abs(float(out[0, 5, 9]) - want) <= TOL * abs(want)
    assert int((out != 0).sum()) == 1


@pytest.mark.gpu
def test_repeats_streams_and_graphs_give_the_same_bits():
    count, rows, cols = 4, 300, 520
    grad = stack(count, rows, cols, "flat", 3).bfloat16()
    mom0 = stack(count, rows, cols, "flat", 5)
    mom = mom0.clone()
    ref = run(grad, mom, "bf16", count, rows, cols)
    plan = rg.moe_muon_plan_create(count, rows, cols)
    ws = torch.zeros(rg.moe_muon_workspace_bytes(plan), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(ref)
    m2 = mom0.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    rg.moe_muon_update(plan, grad, m2, out, ws, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(m2, mom)
    m2.copy_(mom0)
    out.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rg.moe_muon_update(plan, grad, m2, out, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(m2, mom)


@pytest.mark.gpu
def test_several_chunks_equal_single_matrices():
    """A stack larger than what is in flight at once."""
    count, rows, cols = 650, 20, 28
    grad = stack(count, rows, cols, "flat", 6)
    out = run(grad, None, "fp32", count, rows, cols)
    for i in (0, 607, 608, 649):
        assert torch.equal(out[i], run(grad[i:i + 1].contiguous(), None, "fp32", 1, rows, cols)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("count,rows,cols", [(3, 128, 64), (2, 128, 129), (2, 64, 256), (2, 20, 257), (2, 257, 20), (2, 100, 600),
                                             (1, 1500, 128), (3, 24, 1788), (2, 117, 3051), (2, 3051, 117), (1, 128, 4096),
                                             (1, 4097, 16), (1, 129, 1000), (40, 96, 512)])
def test_shapes_around_the_small_form(count, rows, cols):
    """Widths of a CTA's columns, cluster sizes, and the sizes beyond which the
    steps are launches of their own."""
    grad = stack(count, rows, cols, "decaying", rows + 3 * cols).bfloat16()
    mom = stack(count, rows, cols, "flat", rows * 2 + cols)
    m2 = mom.clone()
    ref, rm = plain(grad, mom)
    out = run(grad, mom, "bf16", count, rows, cols)
    assert rel(out, ref) <= TOL
    assert float((mom.double() - rm).abs().max()) <= 2 ** -23 * float(rm.abs().max())
    assert torch.equal(out, run(grad, m2, "bf16", count, rows, cols))


@pytest.mark.gpu
def test_several_chunks_of_the_general_form():
    count, rows, cols = 612, 129, 136
    grad = stack(count, rows, cols, "flat", 6).bfloat16()
    out = run(grad, None, "bf16", count, rows, cols)
    for i in (0, 607, 608, 611):
        assert torch.equal(out[i], run(grad[i:i + 1].contiguous(), None, "bf16", 1, rows, cols)[0])


@pytest.mark.gpu
@pytest.mark.parametrize("count,rows,cols", [(65536, 128, 300), (9000, 520, 512)])
def test_offsets_beyond_31_bits(count, rows, cols):
    """More than 2^31 values in the stack: the last matrices are those of calls of their own."""
    grad = torch.empty(count, rows, cols, dtype=torch.bfloat16, device="cuda")
    grad.uniform_(-1.0, 1.0)
    mom = torch.zeros(count, rows, cols, device="cuda")
    out = run(grad, mom, "bf16", count, rows, cols)
    for i in (0, count - 1):
        m1 = torch.zeros(1, rows, cols, device="cuda")
        assert torch.equal(out[i], run(grad[i:i + 1].contiguous(), m1, "bf16", 1, rows, cols)[0])
        assert torch.equal(mom[i], m1[0])


# ---------------------------------------------------------------- refusals (no GPU needed)
@pytest.fixture(scope="module")
def L():
    from routing_grouped_expert_gemm_gb300 import build as rgbuild
    rgbuild.build()
    return rg.lib()


@pytest.mark.parametrize("kw,code", [
    (dict(count=0), rg.MOE_ERR_UNSUPPORTED_SHAPE), (dict(count=65537), rg.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(rows=0), rg.MOE_ERR_UNSUPPORTED_SHAPE), (dict(cols=0), rg.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(rows=65537), rg.MOE_ERR_UNSUPPORTED_SHAPE), (dict(rows=65536, cols=32768), rg.MOE_ERR_UNSUPPORTED_SHAPE),
    (dict(steps=-1), rg.MOE_ERR_INVALID_ARG), (dict(steps=33), rg.MOE_ERR_INVALID_ARG),
    (dict(grad_dtype=3), rg.MOE_ERR_INVALID_ARG), (dict(grad_dtype=-1), rg.MOE_ERR_INVALID_ARG),
    (dict(coefficients=(1.0, float("nan"), 0.0)), rg.MOE_ERR_INVALID_ARG),
    (dict(coefficients=(float("inf"), 0.0, 0.0)), rg.MOE_ERR_INVALID_ARG),
])
def test_plan_refusals(L, kw, code):
    with pytest.raises(rg.MoEError) as ei:
        rg.moe_muon_plan_create(**{**dict(count=2, rows=16, cols=16), **kw})
    assert ei.value.code == code


def test_null_refusals(L):
    assert L.moe_muon_plan_create(None, None) == rg.MOE_ERR_INVALID_ARG
    assert L.moe_muon_workspace_bytes(None) == 0
    assert L.moe_muon_update(None, None, 0, 0, None, 0.9, 1, 1.0, None, None, 0, None) == rg.MOE_ERR_INVALID_ARG
    assert L.moe_muon_get_status(None, None, None, None) == rg.MOE_ERR_INVALID_ARG
    assert L.moe_muon_plan_destroy(None) == 0


@pytest.mark.gpu
def test_call_refusals():
    plan = rg.moe_muon_plan_create(2, 16, 24)
    g = torch.zeros(2, 16, 24, dtype=torch.bfloat16, device="cuda")
    m = torch.zeros(2, 16, 24, device="cuda")
    u = torch.zeros_like(g)
    ws = torch.zeros(rg.moe_muon_workspace_bytes(plan), dtype=torch.uint8, device="cuda")

    def code(*a, **kw):
        with pytest.raises(rg.MoEError) as ei:
            rg.moe_muon_update(plan, *a, **kw)
        return ei.value.code

    bad = rg.MOE_ERR_INVALID_ARG
    assert code(None, m, u, ws) == bad
    assert code(g, m, None, ws) == bad
    assert code(g, m, u, None, workspace_bytes=1 << 30) == bad
    assert code(g, m, u, ws, grad_row_stride=23) == bad
    assert code(g, m, u, ws, grad_stride=-1) == bad
    assert code(g.data_ptr() + 1, m, u, ws) == bad
    assert code(g, m.data_ptr() + 2, u, ws) == bad
    assert code(g, m, u, ws.data_ptr() + 16, workspace_bytes=1 << 30) == bad
    assert code(g, m, u, ws, mu=float("nan")) == bad
    assert code(g, m, u, ws, scale=float("inf")) == bad
    assert code(g, m, u, ws, nesterov=2) == bad
    assert code(g, m, u, ws, workspace_bytes=ws.numel() - 1) == rg.MOE_ERR_WORKSPACE_TOO_SMALL


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(128, 300), (60, 1000), (700, 90), (33, 2000), (100, 256), (300, 520)])
def test_a_matrix_does_not_depend_on_its_stack(rows, cols):
    """Alone, or among so many that another split over the SMs is chosen."""
    count = 90
    grad = stack(count, rows, cols, "decaying", 12).bfloat16()
    mom = stack(count, rows, cols, "flat", 13)
    m0 = mom.clone()
    out = run(grad, mom, "bf16", count, rows, cols)
    for i in (0, 41, 89):
        m1 = m0[i:i + 1].clone()
        assert torch.equal(out[i], run(grad[i:i + 1].contiguous(), m1, "bf16", 1, rows, cols)[0])
        assert torch.equal(mom[i], m1[0])


# ---------------------------------------------------------------- the coefficients' range
@pytest.mark.parametrize("steps,coefs", [
    (2, (6.0, 0.0, 0.0)),      # |X|_2 6 after a step: A's elements up to 18
    (1, (1.0, 40.0, 0.0)),     # B's elements up to 20
    (1, (1.0, 0.0, -40.0)),
    (3, (3.0, 0.0, 0.0)),      # 9 after two steps
    (32, (1.2, 0.0, 0.0)),
    (1, (1.0, 3e38, 3e38)),
    (32, (3e38, 3e38, 3e38)),
])
def test_coefficients_whose_iterates_leave_fp16_are_refused(L, steps, coefs):
    with pytest.raises(rg.MoEError) as ei:
        rg.moe_muon_plan_create(2, 16, 16, steps=steps, coefficients=coefs)
    assert ei.value.code == rg.MOE_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(64, 96), (96, 64), (200, 264), (264, 200)])
@pytest.mark.parametrize("steps,coefs", [(2, (5.2, 0.0, 0.0)), (1, (1.0, 28.0, 0.0)), (1, (100.0, 0.0, 0.0)),
                                         (3, (2.2, 0.0, 0.0))])
def test_coefficients_near_the_limit(rows, cols, steps, coefs):
    """One direction only, two of the short side's indices sharing it: the
    largest element that A and B can have beside their diagonals.  Nothing cancels
    here (all terms have one sign), so the file's tolerance holds."""
    short = torch.zeros(min(rows, cols), device="cuda")
    short[3] = short[min(rows, cols) - 5] = 1.0
    long = torch.randn(max(rows, cols), device="cuda")
    m = torch.outer(short, long) if rows <= cols else torch.outer(long, short)
    grad = torch.stack([m, torch.randn(rows, cols, device="cuda")])
    ref, _ = plain(grad, None, steps=steps, coefs=coefs)
    out = run(grad, None, "fp32", 2, rows, cols, steps=steps, coefficients=coefs)
    for i in range(2):
        assert rel(out[i], ref[i]) <= TOL


@pytest.mark.gpu
@pytest.mark.parametrize("power", [50, -50])
def test_norms_of_large_matrices_do_not_overflow(power):
    """2^28 and more elements just below 2^50, or 2^-50: the squares' sums reach
    2^128 where the elements are taken as they are (or times 2^100)."""
    rows, cols = 16384, 16640
    grad = (torch.randint(0, 2, (1, rows, cols), device="cuda", dtype=torch.int8) * 2 - 1).bfloat16() * (1 - 2.0 ** -8)
    assert float(grad[0, 0].abs().max()) < 1.0
    ref = run(grad, None, "bf16", 1, rows, cols, steps=1)
    out = run(grad * 2.0 ** power, None, "bf16", 1, rows, cols, steps=1)
    assert bool(torch.isfinite(ref).all()) and torch.equal(out, ref)


# ---------------------------------------------------------------- both forms
# (rows, cols, one launch): a cluster per matrix on chip, or the steps as launches of their own
FORMS = [(70, 90, True), (90, 70, True), (67, 131, True), (200, 264, False), (264, 200, False), (257, 131, False), (131, 257, False)]


def assert_form(rows, cols, one_launch, count=2, **kw):
    """The one-launch form's workspace holds the status only."""
    plan = rg.moe_muon_plan_create(count, rows, cols, **kw)
    assert (rg.moe_muon_workspace_bytes(plan) == 256) == one_launch


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,one_launch", FORMS)
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("nesterov,momentum", [(True, True), (False, True), (True, False)])
def test_types_and_momentum_in_both_forms(rows, cols, one_launch, dtype, nesterov, momentum):
    assert_form(rows, cols, one_launch, 3)
    grad = (stack(3, rows, cols, "decaying", 1) * 1e-2).to(DTYPES[dtype])
    mom = stack(3, rows, cols, "flat", 2) * 1e-2 if momentum else None
    ref, rm = plain(grad, mom, mu=0.9, nesterov=nesterov)
    out = run(grad, mom, dtype, 3, rows, cols, mu=0.9, nesterov=nesterov)
    assert rel(out, ref) <= TOL
    if momentum:
        assert float((mom.double() - rm).abs().max()) <= 2 ** -23 * float(rm.abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,one_launch", FORMS)
@pytest.mark.parametrize("steps,coefs", [(1, COEFS), (2, COEFS), (4, COEFS), (3, (1.875, -1.25, 0.375)), (10, (1.5, -0.5, 0.0))])
def test_steps_and_coefficients_in_both_forms(rows, cols, one_launch, steps, coefs):
    assert_form(rows, cols, one_launch)
    grad = stack(2, rows, cols, "flat", 4)
    ref, _ = plain(grad, None, steps=steps, coefs=coefs, scale=0.3)
    out = run(grad, None, "fp32", 2, rows, cols, steps=steps, coefficients=coefs, scale=0.3)
    # as in test_steps_and_coefficients
    assert rel(out, ref) <= 2 * np.sqrt(4.0 * steps) * 2.0 ** -11 / np.sqrt(3.0) + 2.0 ** -9


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,one_launch", FORMS)
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_strides_in_both_forms(rows, cols, one_launch, dtype):
    assert_form(rows, cols, one_launch, 3)
    mom0 = stack(3, rows, cols, "flat", 2)
    for pad, extra, off in ((0, 0, 1), (8, 0, 0), (5, 3, 2), (24, 1, 8)):
        base = torch.randn(3 * (rows + extra) * (cols + pad) + off, device="cuda").to(DTYPES[dtype])
        view = base[off:].view(3, rows + extra, cols + pad)[:, :rows, :cols]
        mom = mom0.clone()
        ref, rm = plain(view, mom)
        out = run(view.data_ptr(), mom, dtype, 3, rows, cols, grad_row_stride=cols + pad,
                  grad_stride=(rows + extra) * (cols + pad))
        assert rel(out, ref) <= TOL
        assert float((mom.double() - rm).abs().max()) <= 2 ** -23 * float(rm.abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,one_launch", FORMS)
def test_bad_matrices_keep_to_themselves_in_both_forms(rows, cols, one_launch):
    assert_form(rows, cols, one_launch, 5)
    grad = stack(5, rows, cols, "flat", 8)
    ref = run(grad, None, "fp32", 5, rows, cols)
    bad = grad.clone()
    bad[1] = 0
    bad[2, 3, 4] = float("-inf")
    bad[3, rows - 1, cols - 1] = float("nan")
    out = run(bad, None, "fp32", 5, rows, cols)
    assert torch.equal(out[0], ref[0]) and torch.equal(out[4], ref[4])
    assert bool((out[1] == 0).all()) and bool(torch.isnan(out[2]).all()) and bool(torch.isnan(out[3]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,one_launch", FORMS)
@pytest.mark.parametrize("power", [-140, -100, 45, 60, 110])
def test_magnitudes_in_both_forms(rows, cols, one_launch, power):
    """As test_magnitudes_outside_the_squares_range."""
    assert_form(rows, cols, one_launch)
    grad = torch.randint(-8, 9, (2, rows, cols), device="cuda").float()
    ref = run(grad, None, "fp32", 2, rows, cols)
    out = run(torch.ldexp(grad, torch.tensor(power, device="cuda")), None, "fp32", 2, rows, cols)
    assert torch.equal(out, ref)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,one_launch", FORMS)
def test_one_element_in_both_forms(rows, cols, one_launch):
    assert_form(rows, cols, one_launch, 1)
    grad = torch.zeros(1, rows, cols, device="cuda")
    grad[0, rows - 2, cols - 3] = 3.0
    out = run(grad, None, "fp32", 1, rows, cols)
    want = 1.0
    for _ in range(5):
        want = COEFS[0] * want + COEFS[1] * want ** 3 + COEFS[2] * want ** 5
    assert abs(float(out[0, rows - 2, cols - 3]) - want) <= TOL * abs(want)
    assert int((out != 0).sum()) == 1


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols,kind", [(2048, 7168, "decaying"), (7168, 2048, "flat"), (2049, 3333, "low rank")])
def test_large_matrices_match_fp64(rows, cols, kind):
    grad = stack(2, rows, cols, kind, 5).bfloat16()
    mom = stack(2, rows, cols, kind, 6)
    ref, rm = plain(grad, mom, scale=0.2)
    out = run(grad, mom, "bf16", 2, rows, cols, scale=0.2)
    assert rel(out, ref) <= TOL
    assert float((mom.double() - rm).abs().max()) <= 2 ** -23 * float(rm.abs().max())
