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


def refused(match, call, *args, **kwargs):
    with pytest.raises(pnq.PnqError, match=match):
        call(*args, **kwargs)


def test_encode_and_decode_of_wrong_tensors():
    kind, plan = pnq.NVFP4, plan_of(8, 2, 3)
    x = torch.randn(8, 64, device="cuda")
    refused("consecutive", pnq.fp4_quantize, kind, torch.randn(64, 8, device="cuda").t())
    refused("elements apart", pnq.fp4_quantize, kind, x[:1].expand(4, 64))
    refused("contiguous", pnq.fp4_quantize, kind, torch.randn(2, 4, 128, device="cuda")[:, :, :64])
    refused("multiple of 16", pnq.fp4_quantize, kind, torch.randn(8, 72, device="cuda"))
    refused("multiple of 32", pnq.fp4_quantize, pnq.MXFP4, torch.randn(8, 48, device="cuda"))
    refused("dtype", pnq.fp4_quantize, kind, x.half())
    refused("the plan has 8 tokens", pnq.fp4_quantize, kind, x[:7], plan=plan)
    refused("16 rows", pnq.fp4_quantize, kind, x, plan=plan, sorted=True)
    refused("plan is missing", pnq.fp4_quantize, kind, x, sorted=True)
    refused("ExpertPlan", pnq.fp4_quantize, kind, x, plan=x)
    q = pnq.fp4_quantize(kind, x)
    for out in (pnq.fp4_quantize(pnq.MXFP4, x), pnq.fp4_quantize(kind, x[:7]), pnq.fp4_quantize(kind, torch.randn(8, 80, device="cuda")),
                pnq.fp4_quantize(kind, x.view(2, 4, 64)), pnq.fp4_quantize(kind, x, plan=plan)):
        refused("another type, shape", pnq.fp4_quantize, kind, x, out=out)
    refused("another type, shape", pnq.fp4_quantize, kind, x, plan=plan, out=q)
    refused("another type, shape", pnq.fp4_quantize, kind, x, plan=plan, out=pnq.fp4_quantize(kind, x, plan=plan_of(8, 2, 4)))
    refused("shape", pnq.fp4_dequantize, q, out=torch.empty(8, 63, device="cuda"))
    refused("dtype", pnq.fp4_dequantize, q, dtype=torch.float16)
    refused("contiguous", pnq.fp4_dequantize, q, out=torch.empty(64, 8, device="cuda").t())
    refused("CUDA", pnq.fp4_dequantize, q, out=torch.empty(8, 64))
    many = pnq.fp4_quantize(kind, x.view(2, 4, 64))
    refused(r"expected \(2,\)", setattr, many, "global_scale", torch.ones(3, device="cuda"))
    many.global_scale = torch.ones(2, device="cuda")
    refused("matrix by matrix", pnq.fp4_dequantize, many)
    codes, scales = raw(kind, 8, 64)
    refused("elements", pnq.Fp4Matrix, kind, 9, 64, codes, scales)
    refused("elements", pnq.Fp4Matrix, kind, 8, 64, codes, scales[1:])
    refused("dtype", pnq.Fp4Matrix, kind, 8, 64, codes.to(torch.int8), scales)
    refused("ERR_SHAPE", pnq.Fp4Matrix, kind, 8, 40, codes, scales)
    refused("ERR_SHAPE", pnq.Fp4Matrix, kind, -1, 64, codes, scales)
    refused("ERR_ALIGN", pnq.fp4_dequantize, pnq.Fp4Matrix(kind, 7, 64, codes.view(-1)[8:], scales))
    refused("elements", pnq.fp4_pack, kind, codes, scales[:31], 8, 64)
    refused("elements", pnq.fp4_pack, kind, codes.view(-1)[1:], scales, 8, 64)


def test_products_of_wrong_operands():
    kind, plan = pnq.NVFP4, plan_of(8, 2, 3)
    x, w3 = torch.randn(8, 64, device="cuda"), torch.randn(3, 5, 64, device="cuda")
    q, qp, w, we = pnq.fp4_quantize(kind, x), pnq.fp4_quantize(kind, x, plan=plan), pnq.fp4_quantize(kind, w3[0]), pnq.fp4_quantize(kind, w3)
    refused("operands differ", pnq.fp4_gemm, q, pnq.fp4_quantize(pnq.MXFP4, w3[0]))
    refused("operands differ", pnq.fp4_gemm, q, pnq.fp4_quantize(kind, torch.randn(5, 80, device="cuda")))
    refused("one matrix", pnq.fp4_gemm, q, we)
    refused("one matrix", pnq.fp4_gemm, we, w)
    refused("one matrix", pnq.fp4_gemm, qp, w)
    refused("shape", pnq.fp4_gemm, q, w, out=torch.empty(8, 6, device="cuda"))
    refused("dtype", pnq.fp4_gemm, q, w, dtype=torch.float16)
    refused("Fp4Matrix", pnq.fp4_gemm, q, x)
    refused("this plan's", pnq.fp4_gemm_experts, q, we, plan)
    refused("2 matrices", pnq.fp4_gemm_experts, qp, pnq.fp4_quantize(kind, w3[:2].contiguous()), plan)
    refused("operands differ", pnq.fp4_gemm_experts, qp, pnq.fp4_quantize(pnq.MXFP4, w3), plan)
    refused("shape", pnq.fp4_gemm_experts, qp, we, plan, out=torch.empty(15, 5, device="cuda"))
    refused("ExpertPlan", pnq.fp4_gemm_experts, qp, we, x)


def test_expert_calls_with_wrong_tensors():
    plan, ids = plan_of(8, 2, 3), torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    x, ys, w = torch.randn(8, 33, device="cuda"), torch.randn(16, 33, device="cuda"), torch.rand(8, 2, device="cuda")
    refused("dtype", pnq.expert_sort, ids.long(), 3)
    refused("contiguous", pnq.expert_sort, ids.t(), 3)
    refused("slots", pnq.expert_sort, torch.zeros(2, 65, dtype=torch.int32, device="cuda"), 3)
    refused("experts", pnq.expert_sort, ids, 0)
    refused("experts", pnq.expert_sort, ids, 1025)
    refused("another shape", pnq.expert_sort, ids, 4, plan)
    refused("elements", pnq.ExpertPlan, 8, 2, 3, torch.zeros(8 + 48 - 1, dtype=torch.int32, device="cuda"))
    refused("dtype", pnq.ExpertPlan, 8, 2, 3, torch.zeros(100, device="cuda"))
    for call, good in ((pnq.expert_gather, x), (pnq.expert_gather_backward, ys), (lambda t, p, **k: pnq.expert_combine(t, p, w, **k), ys),
                       (lambda t, p, **k: pnq.expert_combine_backward(x, t, p, w, **k), ys)):
        refused("shape", call, good[1:], plan)
        refused("dtype", call, good.double(), plan)
        refused("contiguous", call, torch.randn(33, len(good), device="cuda").t(), plan)
        refused("must be a torch.Tensor", call, good[0], plan)
        refused("ExpertPlan", call, good, x)
        refused("shape", call, good, plan, out=torch.empty(5, 33, device="cuda"))
    refused("dtype", pnq.expert_gather, x, plan, out=torch.empty(16, 33, dtype=torch.bfloat16, device="cuda"))
    refused("dtype", pnq.expert_combine, ys, plan, w, out=torch.empty(8, 33, dtype=torch.bfloat16, device="cuda"))
    refused("shape", pnq.expert_combine, ys, plan, w.t().contiguous())
    refused("dtype", pnq.expert_combine, ys, plan, w.double())
    refused("shape", pnq.expert_combine_backward, x[:7], ys, plan, w)
    refused("dtype", pnq.expert_combine_backward, x.bfloat16(), ys, plan, w)
    refused("shape", pnq.expert_combine_backward, x, ys, plan, w, dweights=torch.empty(8, 3, device="cuda"))
    torch.cuda.synchronize()
    assert pnq.device_error() == 0
