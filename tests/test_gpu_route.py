"""Routing to experts against its definition in 64 bits: ids exactly, weights and gradients within roundings of fp32.

Bounds in units of u = 2^-24. A softmax score: its exponential is within 2 ulp (4 u) and its argument's rounding adds |x - max| u; the sum of
E / 32 + 5 additions of such, a division, the scale. A renormalised weight: the same over at most 64 scores."""
import math

import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def scores(logits, score):
    x = logits.double()
    if score == pnq.SIGMOID:
        return torch.sigmoid(x)
    m = x.amax(1, keepdim=True)
    e = torch.where(x == -math.inf, 0.0, torch.exp(x - m))
    return e / e.sum(1, keepdim=True)


def reference(logits, k, score, bias=None, groups=1, top_groups=None, best=1, renormalize=False, scale=1.0):
    """(ids, weights in 64 bits), expert by expert."""
    T, E = logits.shape
    s = scores(logits, score)
    c = s.clone() if bias is None else s + bias.double()
    c[logits.double() == -math.inf] = -math.inf
    if bias is not None:
        c[:, bias == -math.inf] = -math.inf
    if groups > 1:
        top = torch.sort(c.view(T, groups, -1), dim=2, descending=True)[0][:, :, :best]
        total = torch.where(top == -math.inf, 0.0, top).sum(2)
        total[top[:, :, 0] == -math.inf] = -math.inf
        kept = torch.sort(total, dim=1, descending=True, stable=True)[1][:, :top_groups or groups]
        out = torch.ones(T, groups, dtype=torch.bool, device=c.device).scatter_(1, kept, False)
        c = c.view(T, groups, -1).masked_fill(out[:, :, None], -math.inf).view(T, E)
    value, ids = torch.sort(c, dim=1, descending=True, stable=True)
    value, ids = value[:, :k], ids[:, :k]
    gone = value == -math.inf
    w = s.gather(1, ids).masked_fill(gone, 0.0)
    if renormalize:
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
    return ids.masked_fill(gone, -1).to(torch.int32), scale * w


def bound(logits, E):
    """Relative, per token."""
    x = logits.double()
    spread = torch.where(x == -math.inf, x.amax(1, keepdim=True), x)
    spread = torch.where(spread.isinf().all(1, keepdim=True), 0.0, spread)  # a token without experts: its weights are zeros
    return ((spread.amax(1) - spread.amin(1)) * 2 + E / 32 + 5 + 40)[:, None] * U


def check(logits, k, **rule):
    ids, weights = pnq.expert_route(logits, k, **rule)
    want_ids, want = reference(logits, k, rule.pop("score", pnq.SOFTMAX), **rule)
    assert ids.dtype == torch.int32 and ids.shape == want_ids.shape
    assert torch.equal(ids, want_ids)
    assert bool(((weights.double() - want).abs() <= bound(logits, logits.shape[1]) * want.abs() + 1e-38).all())
    return ids, weights


def make(T, E, dtype, seed=0, stride=None):
    gen = torch.Generator(device="cuda").manual_seed(seed + 7 * T + E)
    x = torch.randn(T, stride or E, generator=gen, device="cuda") + torch.randn(stride or E, generator=gen, device="cuda") / 2
    return x.to(dtype)[:, :E], 0.2 * torch.randn(E, generator=gen, device="cuda")


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (5, 7, 3), (130, 31, 6), (9, 33, 33), (77, 60, 6), (12, 128, 8), (1, 129, 64), (33, 256, 8),
                                   (4, 257, 40), (6, 512, 10), (5, 1000, 64), (3, 1024, 33), (3001, 64, 6)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", [pnq.SOFTMAX, pnq.SIGMOID])
def test_route(T, E, k, dtype, score):
    for bias_on, renorm, extra in ((False, True, 0), (True, False, 0), (True, True, 3)):
        x, bias = make(T, E, dtype, stride=E + extra)
        check(x, k, score=score, bias=bias if bias_on else None, renormalize=renorm, scale=2.5 if renorm else 1.0)


@pytest.mark.parametrize("E,groups,top", [(256, 8, 4), (160, 8, 3), (64, 2, 1), (96, 32, 5), (90, 3, 2), (130, 10, 7), (32, 32, 9), (1024, 4, 2), (21, 7, 7)])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", [pnq.SOFTMAX, pnq.SIGMOID])
def test_groups(E, groups, top, best, score):
    k = min(8, E // groups * top)
    for T, dtype, bias_on in ((257, torch.float32, True), (31, torch.bfloat16, False)):
        x, bias = make(T, E, dtype)
        check(x, k, score=score, bias=bias if bias_on else None, groups=groups, top_groups=top, best=best, renormalize=True)


@pytest.mark.parametrize("score", [pnq.SOFTMAX, pnq.SIGMOID])
@pytest.mark.parametrize("groups", [1, 4])
def test_scores_nearer_than_fp32_tells(score, groups):
    """Biases that bring the choice scores of a token within 1e-8 to 1e-7 of each other: the order is that of the 64-bit scores."""
    for seed in range(40):
        x, _ = make(1, 64, torch.float32, seed)
        s = scores(x, score)[0]
        bias = (0.7 - s).float()  # c = 0.7 but for the rounding of the bias
        c = s + bias.double()
        assert float(c.max() - c.min()) < 1.3e-7 and len(torch.unique(c)) > 60
        check(x, 20, score=score, bias=bias, groups=groups, top_groups=min(2, groups), best=2)
        rows = torch.cat((make(50, 64, torch.float32, seed)[0], x))
        check(rows, 20, score=score, bias=bias, groups=groups, top_groups=min(2, groups), best=2)


@pytest.mark.parametrize("T", [3, 130, 4096, 4097, 10001])
@pytest.mark.parametrize("score", [pnq.SOFTMAX, pnq.SIGMOID])
@pytest.mark.parametrize("groups", [1, 4])
def test_many_tokens_of_near_scores(T, score, groups):
    """The same among many tokens: one in three, and all of a CTA's at the end, need more than fp32."""
    x, _ = make(1, 64, torch.float32, 11)
    bias = (0.7 - scores(x, score)[0]).float()
    rows, _ = make(T, 64, torch.float32, 12)
    rows[::3] = x
    rows[-40:] = x
    for dtype in (torch.float32, torch.bfloat16):
        check(rows.to(dtype), 7, score=score, bias=bias, groups=groups, top_groups=min(2, groups), best=2, renormalize=True)


def test_ties_go_to_the_lowest():
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.zeros(5, 100, dtype=dtype, device="cuda")
        x[1, 50:] = 1
        x[2, ::3] = -0.0
        x[3] = torch.arange(100, device="cuda") // 7
        for score in (pnq.SOFTMAX, pnq.SIGMOID):
            for bias in (None, torch.zeros(100, device="cuda")):
                for groups in (1, 5):
                    check(x, 40, score=score, bias=bias, groups=groups, top_groups=max(1, groups - 1), best=2, renormalize=True)


def test_experts_that_are_out():
    """Logits or biases of -infinity: not chosen, and slots without an expert are dropped; a row of them takes part in nothing."""
    x, bias = make(6, 48, torch.float32)
    x[0, 5:] = -math.inf
    x[1] = -math.inf
    x[2, :24] = -math.inf
    x[3, 47] = 200.0
    x[4] = -200.0
    x[4, 7] = -199.0
    bias[9] = -math.inf
    for score in (pnq.SOFTMAX, pnq.SIGMOID):
        for groups in (1, 4):
            for renorm in (False, True):
                for b in (None, bias):
                    if score == pnq.SIGMOID and renorm:  # the definition in 64 bits holds where fp32 scores would not
                        ids, w = pnq.expert_route(x, 12, score=score, bias=b, groups=groups, top_groups=3 if groups > 1 else 1, renormalize=True)
                        _, want = reference(x, 12, score, bias=b, groups=groups, top_groups=3 if groups > 1 else 1, renormalize=True)
                        assert bool(((w.double() - want).abs() <= 500 * U * want + 1e-38).all())
                    elif score == pnq.SOFTMAX or not renorm:
                        ids, w = check(x, 12, score=score, bias=b, groups=groups, top_groups=3 if groups > 1 else 1, renormalize=renorm)
                    assert bool((ids[1] == -1).all()) and bool((w[1] == 0).all())
                    assert bool(((ids == -1) == ((ids == -1) & (w == 0))).all())
    ids, w = pnq.expert_route(x, 12)
    plan = pnq.expert_sort(ids, 48)
    assert int(plan.offsets[-1]) == int((ids >= 0).sum())


def test_nan_stays_in_its_token():
    x, bias = make(5, 40, torch.float32)
    clean = pnq.expert_route(x, 6, bias=bias, renormalize=True)
    x[1, 3] = math.nan
    x[3, 39] = math.inf
    ids, w = pnq.expert_route(x, 6, bias=bias, renormalize=True)
    assert bool(w[[1, 3]].isnan().all()) and ids[1].tolist() == ids[3].tolist() == list(range(6))
    assert torch.equal(ids[[0, 2, 4]], clean[0][[0, 2, 4]]) and torch.equal(w[[0, 2, 4]], clean[1][[0, 2, 4]])
    ids, w = pnq.expert_route(x, 6, score=pnq.SIGMOID)
    assert bool(w[1].isnan().all()) and float(w[3, 0]) == 1.0 and int(ids[3, 0]) == 39
    bias[4] = math.nan
    ids, w = pnq.expert_route(x, 6, score=pnq.SIGMOID, bias=bias)
    assert bool(w.isnan().all()) and bool((ids >= 0).all())


def gradient(dweights, logits, ids, score, renormalize, scale):
    """By the formula in 64 bits, slot by slot."""
    x = logits.double()
    s = scores(logits, score)
    T, E = x.shape
    ok = (ids >= 0) & (ids < E)
    at = ids.clamp(0, E - 1).long()
    c = torch.where(ok, s.gather(1, at), 0.0)
    dw = torch.where(ok, dweights.double(), 0.0) * scale
    if renormalize:
        total = c.sum(1, keepdim=True).clamp(min=1e-300)
        dc = (dw - (dw * c).sum(1, keepdim=True) / total) / total
    else:
        dc = dw
    ds = torch.zeros_like(s).scatter_add_(1, at, torch.where(ok, dc, 0.0))
    size = torch.zeros_like(s).scatter_add_(1, at, torch.where(ok, dc.abs() + (dw.abs().sum(1, keepdim=True) / (total if renormalize else 1)), 0.0))
    if score == pnq.SIGMOID:
        return ds * s * (1 - s), size * s * (1 - s)
    return s * (ds - (ds * s).sum(1, keepdim=True)), s * (size + (size * s).sum(1, keepdim=True))


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 7, 3), (130, 31, 6), (9, 33, 33), (12, 128, 8), (33, 256, 8), (4, 257, 40), (5, 1000, 64), (2000, 64, 6)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", [pnq.SOFTMAX, pnq.SIGMOID])
@pytest.mark.parametrize("renorm", [False, True])
def test_gradient(T, E, k, dtype, score, renorm):
    x, bias = make(T, E, dtype, stride=E + 1)
    if T > 4 and E > 4:
        x[3, : E // 2] = -math.inf
        x[2] = -math.inf
    ids, _ = pnq.expert_route(x, k, score=score, bias=bias, renormalize=renorm, scale=1.5)
    dw = torch.randn(T, k, device="cuda")
    if T > 1:
        ids[0, 0] = -1 if k > 1 else ids[0, 0]
        ids[1, k - 1] = ids[1, 0]  # the same expert twice
    got = pnq.expert_route_backward(dw, x, ids, score=score, renormalize=renorm, scale=1.5)
    want, size = gradient(dw, x, ids, score, renorm, 1.5)
    want, size = torch.nan_to_num(want), torch.nan_to_num(size)
    assert got.dtype == dtype and bool(got.isfinite().all())
    step = torch.finfo(dtype).eps / 2
    assert bool(((got.double() - want).abs() <= (bound(torch.where(x.isinf().all(1, keepdim=True), 0.0, x), E) + 64 * U) * size + step * want.abs() * 1.01 + 1e-37).all())


def test_gradient_against_differences():
    h = 1e-6
    x, bias = make(3, 12, torch.float32)
    dw = torch.randn(3, 4, device="cuda")
    for score in (pnq.SOFTMAX, pnq.SIGMOID):
        for renorm in (False, True):
            ids, _ = pnq.expert_route(x, 4, score=score, bias=bias, renormalize=renorm)
            got = pnq.expert_route_backward(dw, x, ids, score=score, renormalize=renorm)

            def loss(z):
                w = scores(z, score).gather(1, ids.long())
                return ((w / w.sum(1, keepdim=True) if renorm else w) * dw.double()).sum()

            for i in range(3):
                for j in range(12):
                    step = torch.zeros(3, 12, dtype=torch.float64, device="cuda")
                    step[i, j] = h
                    d = float((loss(x.double() + step) - loss(x.double() - step)) / (2 * h))
                    assert float(got[i, j]) == pytest.approx(d, rel=1e-5, abs=1e-7)


def test_gradient_ignores_ids_outside():
    x, _ = make(4, 16, torch.float32)
    ids = torch.tensor([[0, 16, -5], [1 << 30, 3, 3], [-1, -1, -1], [15, 14, -(1 << 31)]], dtype=torch.int32, device="cuda")
    dw = torch.randn(4, 3, device="cuda")
    for score in (pnq.SOFTMAX, pnq.SIGMOID):
        for renorm in (False, True):
            got = pnq.expert_route_backward(dw, x, ids, score=score, renormalize=renorm)
            want, _ = gradient(dw, x, ids, score, renorm, 1.0)
            assert bool(((got.double() - want).abs() <= 100 * U).all())
            assert bool((got[2] == 0).all())


def test_routing_into_the_layer():
    """Router, sort, gather, combine and the gradients on the way back, as a layer uses them; captured and replayed."""
    T, E, k, D = 70, 24, 4, 96
    x, bias = make(T, E, torch.bfloat16)
    h = torch.randn(T, D, device="cuda")

    def step():
        ids, w = pnq.expert_route(x, k, score=pnq.SIGMOID, bias=bias, groups=4, top_groups=2, best=2, renormalize=True)
        plan = pnq.expert_sort(ids, E)
        ys = pnq.expert_gather(h, plan)
        y = pnq.expert_combine(ys, plan, w)
        dys, dw = pnq.expert_combine_backward(h, ys, plan, w)
        return y, pnq.expert_route_backward(dw, x, ids, score=pnq.SIGMOID, renormalize=True), ids, w

    y, dx, ids, w = step()
    # every expert passes its rows on, so y = h times a sum of weights that is 1, and the weights' gradients are all <h, h>: no pull on the logits
    assert bool(((y - h).abs() <= 8 * U * h.abs() * k).all())
    assert float(dx.float().abs().max()) <= 64 * U * float((h * h).sum(1).max())
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(make(T, E, torch.bfloat16, 3)[0])
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, step()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T", [100, 6000])
def test_captured_with_near_scores(T):
    """Captured, and replayed on other logits, at once with a second call on another stream: the same as called."""
    x, _ = make(1, 64, torch.float32, 11)
    bias = (0.7 - scores(x, pnq.SIGMOID)[0]).float()
    rows = make(T, 64, torch.float32, 5)[0].clone()
    other = make(T, 64, torch.float32, 6)[0].clone()
    other[::7] = x
    rule = dict(score=pnq.SIGMOID, bias=bias, groups=4, top_groups=2, best=2, renormalize=True)
    pnq.expert_route(rows, 6, **rule)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        out = pnq.expert_route(rows, 6, **rule)
    rows.copy_(other)
    torch.cuda.synchronize()
    for _ in range(3):
        graph.replay()
        second = pnq.expert_route(other, 6, stream=stream, **rule)
        torch.cuda.synchronize()
        want_ids, _ = reference(other, 6, **rule)
        for ids, w in (out, second):
            assert torch.equal(ids, want_ids) and torch.equal(w, second[1])
