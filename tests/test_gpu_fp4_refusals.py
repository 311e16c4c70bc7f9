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
