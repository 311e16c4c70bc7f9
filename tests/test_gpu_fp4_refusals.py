"""Refusals of the torch wrappers that take CUDA tensors to reach: operands and plans that do not belong together. Every one of
them is raised before anything is launched."""
import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq

pytestmark = pytest.mark.gpu


def raw(kind, rows, K, plan_experts=0):
    """Zero codes and scales of an operand of `rows` rows."""
    pitch, size = pnq.fp4_layout(kind, rows, K, 1, plan_experts)
    return torch.zeros(rows, pitch, dtype=torch.uint8, device="cuda"), torch.zeros(size, dtype=torch.uint8, device="cuda")


def plan_of(tokens, slots, experts, shift=0):
    ids = (torch.arange(tokens * slots, dtype=torch.int32, device="cuda").view(tokens, slots) + shift) % experts
    return pnq.expert_sort(ids, experts)


@pytest.mark.parametrize("kind", [pnq.NVFP4, pnq.MXFP4])
@pytest.mark.parametrize("rows", [1, 8, 999, 1001, 2000])
def test_an_operand_has_its_plans_rows(kind, rows):
    """A product by experts reads the plan's 1000 rows: an operand of fewer (or more) is no operand of that plan."""
    plan = plan_of(500, 2, 3)
    with pytest.raises(pnq.PnqError, match="1000 sorted rows"):
        pnq.Fp4Matrix(kind, rows, 64, *raw(kind, rows, 64, 3), plan=plan)
    m = pnq.Fp4Matrix(kind, 1000, 64, *raw(kind, 1000, 64, 3), plan=plan)
    assert m.rows == plan.rows and m.plan is plan


def test_products_refuse_another_plan():
    """Two layers of one model have plans of the same sizes: an operand sorted by one is not multiplied by the other. The
    same memory as another ExpertPlan is the same plan."""
    K, E = 64, 3
    first, second = plan_of(8, 2, E), plan_of(8, 2, E, shift=1)
    x = torch.randn(8, K, device="cuda")
    w = pnq.fp4_quantize(pnq.NVFP4, torch.randn(E, 40, K, device="cuda"))
    q = pnq.fp4_quantize(pnq.NVFP4, x, plan=first)
    for other in (second, plan_of(8, 2, E + 1), plan_of(16, 1, E), plan_of(4, 2, E)):
        with pytest.raises(pnq.PnqError, match="not an operand of this plan"):
            pnq.fp4_gemm_experts(q, w, other)
    want = pnq.fp4_gemm_experts(q, w, first)
    assert torch.equal(pnq.fp4_gemm_experts(q, w, pnq.ExpertPlan(8, 2, E, first.buffer)), want)
    pnq.fp4_quantize(pnq.NVFP4, x, plan=second, out=q)  # the operand is the second plan's from here on
    with pytest.raises(pnq.PnqError, match="not an operand of this plan"):
        pnq.fp4_gemm_experts(q, w, first)
    pnq.fp4_gemm_experts(q, w, second)


@pytest.mark.parametrize("g", [0.0, -1.0, float("nan"), float("inf"), 1e-45])
def test_a_refused_encode_leaves_out_as_it_was(g):
    """Codes, multiplier (one, or one per matrix) and plan of `out` stay those of the operand it was."""
    x = torch.randn(8, 64, device="cuda")
    first, second = plan_of(8, 2, 3), plan_of(8, 2, 3, shift=1)
    q = pnq.fp4_quantize(pnq.NVFP4, x, 0.25, plan=first)
    before = q.codes.clone()
    with pytest.raises(pnq.PnqError) as e:
        pnq.fp4_quantize(pnq.NVFP4, 2 * x, g, plan=second, out=q)
    assert e.value.status == pnq.Status.ERR_VALUE
    assert q.global_scale == 0.25 and q.plan is first and torch.equal(q.codes, before)
    m = pnq.fp4_quantize(pnq.NVFP4, x.view(2, 4, 64))
    m.global_scale = torch.tensor([0.5, 2.0], device="cuda")
    with pytest.raises(pnq.PnqError):
        pnq.fp4_quantize(pnq.NVFP4, x.view(2, 4, 64), g, out=m)
    assert torch.equal(m.global_scale, torch.tensor([0.5, 2.0], device="cuda"))
    pnq.fp4_quantize(pnq.NVFP4, x, 0.5, plan=second, out=q)
    assert q.global_scale == 0.5 and q.plan is second


@pytest.mark.parametrize("flags", [2, 3, -1, 1 << 32, (1 << 32) + 1, -(1 << 32)])
def test_unknown_flags(flags):
    """Flags past 32 bits too: their low bits are not taken for the whole."""
    q, w = pnq.fp4_quantize(pnq.NVFP4, torch.randn(8, 64, device="cuda")), pnq.fp4_quantize(pnq.NVFP4, torch.randn(3, 5, 64, device="cuda"))
    with pytest.raises(pnq.PnqError) as e:
        pnq.fp4_gemm(q, q, flags=flags)
    assert e.value.status == pnq.Status.ERR_FLAGS
    plan = plan_of(8, 2, 3)
    with pytest.raises(pnq.PnqError) as e:
        pnq.fp4_gemm_experts(pnq.fp4_quantize(pnq.NVFP4, torch.randn(8, 64, device="cuda"), plan=plan), w, plan, flags=flags)
    assert e.value.status == pnq.Status.ERR_FLAGS
