"""Plans that were never sorted, or were overwritten: whatever their arrays hold, the calls stay inside their buffers (guards on
both sides of every output, no device error), entries in range are used as ever, and the rest count as dropped."""
import numpy as np
import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq
from test_gpu_fp4 import route

pytestmark = pytest.mark.gpu

GUARD = 1024
FILLS = {"highest": 2 ** 31 - 1, "lowest": -2 ** 31, "minus two": -2, "one past": None, "noise": None}


def guarded(shape, dtype):
    """A zeroed tensor of `shape` and a check that the elements on both sides of it stayed as they were."""
    n = int(np.prod(shape))
    buf = torch.full((n + 2 * GUARD,), 7, dtype=dtype, device="cuda")
    t = buf[GUARD:GUARD + n].view(shape)
    t.zero_()
    return t, lambda: bool((buf[:GUARD] == 7).all()) and bool((buf[GUARD + n:] == 7).all())


def spoiled(T, k, E, how):
    n = T * k
    if how == "noise":
        fill = torch.from_numpy(np.random.default_rng(n).integers(-2 ** 31, 2 ** 31, 2 * (E + 1) + 3 * n).astype(np.int32)).cuda()
    else:
        fill = torch.full((2 * (E + 1) + 3 * n,), n if how == "one past" else FILLS[how], dtype=torch.int32, device="cuda")
    return pnq.ExpertPlan(T, k, E, fill)


@pytest.mark.parametrize("how", list(FILLS))
@pytest.mark.parametrize("T,k,E,K", [(3, 2, 4, 64), (40, 33, 70, 96), (3000, 4, 9, 288)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_plan_never_sorted(how, T, k, E, K, dtype):
    plan, n = spoiled(T, k, E, how), T * k
    x, rows = torch.ones(T, K, dtype=dtype, device="cuda"), torch.ones(n, K, dtype=dtype, device="cuda")
    weights = torch.ones(T, k, device="cuda")
    xs, a = guarded((n, K), dtype)
    pnq.expert_gather(x, plan, out=xs)
    y, b = guarded((T, K), dtype)
    pnq.expert_combine(rows, plan, weights, out=y)
    dx, c = guarded((T, K), dtype)
    pnq.expert_gather_backward(rows, plan, out=dx)
    dys, d = guarded((n, K), dtype)
    dw, e = guarded((T, k), torch.float32)
    pnq.expert_combine_backward(x, rows, plan, weights, out=dys, dweights=dw)
    checks = [a, b, c, d, e]
    for kind in (pnq.NVFP4, pnq.MXFP4):
        pitch, size = pnq.fp4_layout(kind, n, K, 1, E)
        codes, f = guarded((n, pitch), torch.uint8)
        scales, g = guarded((size,), torch.uint8)
        q = pnq.Fp4Matrix(kind, n, K, codes, scales, plan=plan)
        pnq.fp4_quantize(kind, x, plan=plan, out=q)
        pnq.fp4_quantize(kind, rows, plan=plan, sorted=True, out=q)
        v, h = guarded((n, K), dtype)
        pnq.fp4_dequantize(q, out=v)
        w = pnq.fp4_quantize(kind, torch.ones(E, 130, K, device="cuda"))
        z, i = guarded((n, 130), dtype)
        pnq.fp4_gemm_experts(q, w, plan, out=z)
        checks += [f, g, h, i]
        assert not z.any()
        if how not in ("noise", "one past"):  # n may be a scale row: the scales of few rows are spread over more
            assert not codes.any() and not v.any()
    assert pnq.device_error() == 0
    assert all(check() for check in checks)
    if how != "noise":  # every position is out of range
        assert not any(t.any() for t in (y, dx, dw))


def test_one_entry_overwritten():
    """A slot whose position is out of range counts as dropped; the other slots' results are those of the whole plan."""
    T, k, E, D = 50, 3, 6, 96
    plan = pnq.expert_sort(torch.from_numpy(route(T, k, E, 1)).cuda(), E)
    ys, weights = torch.randn(T * k, D, device="cuda"), torch.rand(T, k, device="cuda")
    want = pnq.expert_combine(ys, plan, weights)
    plan.position[7 * k + 1] = T * k
    got = pnq.expert_combine(ys, plan, weights)
    kept = plan.position[7 * k + torch.tensor([0, 2], device="cuda")].long()
    assert torch.allclose(got[7], (weights[7, [0, 2], None] * ys[kept]).sum(0), rtol=1e-6, atol=1e-6)
    got[7] = want[7]
    assert torch.equal(got, want)


def test_offsets_overwritten():
    """Offsets that fall, or that pass the rows, make a product of zeros; the plan's own offsets give its rows."""
    T, k, E, K, N = 200, 2, 5, 128, 96
    plan = pnq.expert_sort(torch.from_numpy(route(T, k, E, 2)).cuda(), E)
    q = pnq.fp4_quantize(pnq.NVFP4, torch.randn(T, K, device="cuda"), plan=plan)
    w = pnq.fp4_quantize(pnq.NVFP4, torch.randn(E, N, K, device="cuda"))
    want = pnq.fp4_gemm_experts(q, w, plan)
    assert want.any(1).all()
    for at, value in ((1, -1), (2, T * k + 1), (3, 2 ** 31 - 1), (E, 0), (0, 2 ** 30)):
        old = int(plan.offsets[at])
        plan.offsets[at] = value
        assert not pnq.fp4_gemm_experts(q, w, plan).any(), (at, value)
        plan.offsets[at] = old
        assert torch.equal(pnq.fp4_gemm_experts(q, w, plan), want)
    assert pnq.device_error() == 0
