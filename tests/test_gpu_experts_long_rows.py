"""Expert rows of many elements by a warp per token (many tokens) and by a CTA (few): gradients of the weights against sums in
64 bits, and rows bit for bit the same whichever takes them.

Bound of dweights: a thread adds D / 32 terms (a warp per token, 16 tokens per SM or more), rounded up to the 8 of an access,
and 5 additions join the warp: (D / 32 + 16) 2^-24 of the sum of magnitudes; a CTA's threads add fewer."""
import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq
from test_gpu_fp4 import route

pytestmark = pytest.mark.gpu


def tensor(rows, D, dtype, offset, gen):
    buf = torch.zeros(rows * D + offset, dtype=dtype, device="cuda")
    t = buf[offset:].view(rows, D)
    t.copy_(torch.randn(rows, D, generator=gen, device="cuda"))
    return t


@pytest.mark.parametrize("D", [2048, 2049, 4100, 5120])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("T", [40, 5000])
def test_gradients_of_the_weights(D, dtype, offset, T):
    k, E = 3, 9
    gen = torch.Generator(device="cuda").manual_seed(D)
    plan = pnq.expert_sort(torch.from_numpy(route(T, k, E, D, "drop")).cuda(), E)
    ys, dy, w = tensor(T * k, D, dtype, offset, gen), tensor(T, D, dtype, offset, gen), torch.rand(T, k, generator=gen, device="cuda")
    dys, dw = pnq.expert_combine_backward(dy, ys, plan, w)
    at = plan.position.view(T, k).long()
    for j in range(k):
        there = at[:, j] >= 0
        terms = ys[at[there, j]].double() * dy[there].double()
        bound = (D / 32 + 16) * 2.0 ** -24 * terms.abs().sum(-1)
        assert bool(((dw[there, j].double() - terms.sum(-1)).abs() <= bound).all())
        assert not dw[~there, j].any()
    again = pnq.expert_combine_backward(dy, ys, plan, w)
    assert torch.equal(again[0], dys) and torch.equal(again[1], dw)


@pytest.mark.parametrize("D", [2048, 2049])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_do_not_depend_on_the_launch(D, dtype):
    """The first 40 tokens alone (a CTA each) and among 5000 (a warp each): the same bits of every row."""
    T, few, k, E = 5000, 40, 3, 9
    gen = torch.Generator(device="cuda").manual_seed(D)
    ids = torch.from_numpy(route(T, k, E, D, "drop")).cuda()
    x, w = tensor(T, D, dtype, 0, gen), torch.rand(T, k, generator=gen, device="cuda")
    plan, part = pnq.expert_sort(ids, E), pnq.expert_sort(ids[:few].contiguous(), E)
    xs, xp = pnq.expert_gather(x, plan), pnq.expert_gather(x[:few], part)
    y, yp = pnq.expert_combine(xs, plan, w), pnq.expert_combine(xp, part, w[:few])
    assert torch.equal(y[:few], yp)
    assert torch.equal(pnq.expert_gather_backward(xs, plan)[:few], pnq.expert_gather_backward(xp, part))
    dys, dp = pnq.expert_combine_backward(x, xs, plan, w)[0], pnq.expert_combine_backward(x[:few], xp, part, w[:few])[0]
    a, b = plan.position[:few * k].long(), part.position.long()
    assert torch.equal(a >= 0, b >= 0)
    assert torch.equal(dys[a[a >= 0]], dp[b[b >= 0]])
