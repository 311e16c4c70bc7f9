"""Routing of tokens whose choice scores are all nearer than fp32 tells, at the sizes where a thread holds several experts, a token has more than
32 slots, or the logits are bf16.

Such a token: logits x of the tested type, and a bias that is 0.7 - s(x) rounded to fp32, so that every c = s + bias is 0.7 but for that
rounding, 2^-25 at most either way. The kernel's fp32 tolerance is above 2^-24 + 2^-23 * 0.7 for either score (at least 1.4e-7, against a spread of
6e-8), so these tokens are certain to be done again with finer scores.

Those are s to some 2^-44 of itself (s <= 1), and a sum with the bias: c within 2^-43 of what it is, a group's score of two within 2^-42. What is
chosen is compared with the 64-bit scores within that: each place's score is the sorted one within twice the error, and the expert is the
sorted one wherever no other score lies that near (equal logits of equal biases are ties, which go to the lowest index)."""
import math

import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq
from test_gpu_route import bound, make, reference, scores

pytestmark = pytest.mark.gpu
NEAR = 2 * 2.0 ** -43


def near_bias(E, dtype, score, seed):
    """One token's logits in `dtype` and the bias that brings its choice scores together."""
    x = make(1, E, dtype, seed)[0].contiguous()
    s = scores(x, score)[0]
    bias = (0.7 - s).float()
    c = s + bias.double()
    assert float(c.max() - c.min()) <= 2.0 ** -24
    assert len(torch.unique(c)) > 0.9 * len(torch.unique(x))  # not ties
    return x, bias


def choice_scores(x, score, bias, groups, top_groups, best):
    """c in 64 bits with what the groups leave out at -infinity, and for each token whether its groups are told apart."""
    T, E = x.shape
    c = scores(x, score) + bias.double()
    clear = torch.ones(T, dtype=torch.bool, device=x.device)
    if groups > 1:
        each = c.view(T, groups, -1)
        total = torch.sort(each, dim=2, descending=True)[0][:, :, :best].sum(2)
        value, order = torch.sort(total, dim=1, descending=True, stable=True)
        if top_groups < groups:
            clear = value[:, top_groups - 1] - value[:, top_groups] > 2 * NEAR
        out = torch.ones(T, groups, dtype=torch.bool, device=x.device).scatter_(1, order[:, :top_groups], False)
        c = each.masked_fill(out[:, :, None], -math.inf).view(T, E)
    return c, clear


def check(x, k, score, bias, groups=1, top_groups=1, best=2, renormalize=True):
    T, E = x.shape
    ids, weights = pnq.expert_route(x, k, score=score, bias=bias, groups=groups, top_groups=top_groups, best=best, renormalize=renormalize)
    c, clear = choice_scores(x, score, bias, groups, top_groups, best)
    value, order = torch.sort(c, dim=1, descending=True, stable=True)
    at = ids.long()
    assert bool(((at >= 0) & (at < E)).all())
    assert bool((torch.sort(at, dim=1)[0].diff(dim=1) > 0).all())  # no expert twice
    got = c.gather(1, at)
    assert bool(((got - value[:, :k]).abs() <= NEAR)[clear].all())
    # apart from its neighbours in order, or an exact tie (the same logit and bias) decided by the index
    gap = (value[:, :-1] - value[:, 1:]).nan_to_num(nan=math.inf)  # -infinity after -infinity
    gap = torch.where(gap == 0, math.inf, gap)
    alone = torch.ones_like(value, dtype=torch.bool)
    alone[:, :-1] &= gap > NEAR
    alone[:, 1:] &= gap > NEAR
    sure = alone[:, :k] & clear[:, None]
    assert torch.equal(at[sure], order[:, :k][sure])
    w = scores(x, score).gather(1, at)
    if renormalize:
        w = w / w.sum(1, keepdim=True)
    assert bool(((weights.double() - w).abs() <= bound(x, E) * w + 1e-38).all())
    return int(sure.sum()) / k  # tokens' worth of places compared as they are


SIZES = [(64, 7, 1, 1), (33, 33, 1, 1), (90, 50, 3, 2), (100, 40, 5, 4), (256, 8, 1, 1), (256, 8, 8, 4), (257, 40, 1, 1), (1000, 64, 1, 1), (1000, 64, 8, 3), (1024, 33, 1, 1),
         (1024, 64, 32, 5)]


@pytest.mark.parametrize("E,k,groups,top", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", [pnq.SOFTMAX, pnq.SIGMOID])
def test_one_near_token(E, k, groups, top, dtype, score):
    told = 0.0  # two scores of a token, or of its groups, are within the error of each other once in some hundred tokens
    for seed in range(8):
        x, bias = near_bias(E, dtype, score, 100 + seed)
        for best in (1, 2):
            told += check(x, k, score, bias, groups, top, best, renormalize=seed % 2 == 0)
    assert told >= 12


@pytest.mark.parametrize("E,k,groups,top", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", [pnq.SOFTMAX, pnq.SIGMOID])
@pytest.mark.parametrize("T", [6, 4100])
def test_near_tokens_among_others(E, k, groups, top, dtype, score, T):
    """Few tokens (done again by the CTAs that met them) and many (by a kernel of their own), one in three near."""
    x, bias = near_bias(E, dtype, score, 7)
    rows = make(T, E, dtype, 8)[0].clone()
    rows[::3] = x
    assert check(rows, k, score, bias, groups, top) >= 0.6 * T


@pytest.mark.parametrize("T", [3, 4500])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", [pnq.SOFTMAX, pnq.SIGMOID])
def test_equal_groups(T, dtype, score):
    """A router that starts at zero: every score and every group is equal, and the lowest groups and experts are chosen, with equal weights."""
    for bias in (None, torch.zeros(256, device="cuda")):
        ids, w = pnq.expert_route(torch.zeros(T, 256, dtype=dtype, device="cuda"), 8, score=score, bias=bias, groups=8, top_groups=4, best=2,
                                  renormalize=True)
        assert torch.equal(ids, torch.arange(8, dtype=torch.int32, device="cuda").expand(T, 8)) and bool((w == 0.125).all())


def test_order_of_renormalised_sigmoids_with_experts_out():
    """The ids, in order, where logits and biases of -infinity, 200 and -200 leave fp32 scores that are 0 or 1."""
    x, bias = make(6, 48, torch.float32)
    x[0, 5:] = -math.inf
    x[1] = -math.inf
    x[2, :24] = -math.inf
    x[3, 47] = 200.0
    x[4] = -200.0
    x[4, 7] = -199.0
    bias[9] = -math.inf
    for groups in (1, 4):
        for b in (None, bias):
            rule = dict(score=pnq.SIGMOID, bias=b, groups=groups, top_groups=3 if groups > 1 else 1, renormalize=True)
            assert torch.equal(pnq.expert_route(x, 12, **rule)[0], reference(x, 12, **rule)[0])
