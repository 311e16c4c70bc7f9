"""The expert calls and autograd: results require no gradient (and the documentation of each call says so), and the gradients
that the library has, wrapped in torch.autograd.Function as the documentation names it, are those of the same layer in
plain torch in 64 bits.

Bound: sums of k terms and dot products of D terms in fp32, (D / 32 + 16) 2^-24 of the sums of magnitudes, which random
values of size one keep below 1e-4 at these sizes."""
import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq
from test_gpu_fp4 import route

pytestmark = pytest.mark.gpu


class Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, plan):
        ctx.plan = plan
        return pnq.expert_gather(x, plan)

    @staticmethod
    def backward(ctx, dxs):
        return pnq.expert_gather_backward(dxs.contiguous(), ctx.plan), None


class Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ys, weights, plan):
        ctx.plan = plan
        ctx.save_for_backward(ys, weights)
        return pnq.expert_combine(ys, plan, weights)

    @staticmethod
    def backward(ctx, dy):
        ys, weights = ctx.saved_tensors
        return *pnq.expert_combine_backward(dy.contiguous(), ys, ctx.plan, weights), None


def layer_inputs(T, k, E, D):
    gen = torch.Generator(device="cuda").manual_seed(T)
    plan = pnq.expert_sort(torch.from_numpy(route(T, k, E, T, "drop")).cuda(), E)
    x = torch.randn(T, D, generator=gen, device="cuda", requires_grad=True)
    weights = torch.rand(T, k, generator=gen, device="cuda", requires_grad=True)
    return plan, x, weights


def test_results_stand_outside_autograd():
    plan, x, weights = layer_inputs(20, 2, 3, 64)
    xs = pnq.expert_gather(x, plan)
    assert not xs.requires_grad and not pnq.expert_combine(xs, plan, weights).requires_grad
    for call in (pnq.expert_gather, pnq.expert_combine):
        assert "requires no gradient" in call.__doc__
    for call in (pnq.fp4_gemm, pnq.fp4_gemm_experts):
        assert "gradient" in call.__doc__


@pytest.mark.parametrize("T,k,E,D", [(20, 2, 3, 64), (500, 4, 9, 192)])
def test_gradients_through_functions_of_the_pairs(T, k, E, D):
    plan, x, weights = layer_inputs(T, k, E, D)
    dy = torch.randn(T, D, device="cuda")
    Combine.apply(Gather.apply(x, plan).tanh(), weights, plan).backward(dy)
    x64, w64 = x.detach().double().requires_grad_(), weights.detach().double().requires_grad_()
    kept = (plan.position.view(T, k) >= 0).double()
    (x64.tanh()[:, None, :] * (w64 * kept)[..., None]).sum(1).backward(dy.double())
    assert torch.allclose(x.grad.double(), x64.grad, rtol=1e-5, atol=1e-4)
    assert torch.allclose(weights.grad.double(), w64.grad, rtol=1e-5, atol=1e-4)
