"""Tokens to their experts and back on the GPU: the plan against a plain sort, rows and gradients against sums in 64 bits,
and the gradients against differences of the forward pass.

Bounds. Gathered rows are copies: equal. Sums over k slots in fp32: (k + 1) 2^-24 of the sum of magnitudes, plus half a unit
of the result's type (24 or 8 significant bits: 2^-24 or 2^-8 of its magnitude). <dy, y> in fp32 over D elements, summed in 256 threads and joined: (D / 256 + 16)
2^-24 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq
import fp4_reference as ref
from test_gpu_fp4 import route

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
ROUTES = [(1, 1, 1, "even"), (1, 8, 64, "even"), (7, 3, 5, "drop"), (33, 8, 256, "even"), (100, 2, 3, "one"), (50, 4, 6, "none"),
          (1000, 8, 128, "skew"), (4100, 6, 1024, "drop"), (20000, 8, 60, "skew"), (3, 64, 40, "even"), (70000, 1, 7, "drop")]


@pytest.mark.parametrize("T,k,E,how", ROUTES)
def test_sort(T, k, E, how):
    ids = route(T, k, E, seed=T + k, how=how)
    guard = torch.full((2 * (E + 1) + 3 * T * k + 32,), 99, dtype=torch.int32, device="cuda")
    plan = pnq.ExpertPlan(T, k, E, guard)
    pnq.expert_sort(torch.from_numpy(ids).cuda(), E, plan)
    want = ref.plan(ids, E)
    for name, w in zip(("offsets", "block_start", "order", "position", "scale_row"), want):
        assert np.array_equal(getattr(plan, name).cpu().numpy(), w), name
    assert bool((guard[-32:] == 99).all())


ROWS = [(1, 1, 1, "even", 1), (1, 8, 64, "even", 5120), (7, 3, 5, "drop", 33), (40, 9, 12, "drop", 264), (20, 17, 30, "even", 100),
        (100, 2, 3, "one", 1999), (50, 4, 6, "none", 64), (700, 8, 128, "skew", 520), (5, 3, 4, "even", 2052), (3000, 3, 9, "drop", 300),
        (2600, 9, 20, "drop", 67), (4, 2, 3, "even", 12290), (300, 2, 5, "drop", 1030)]


def rows_on_gpu(a, dtype, offset):
    """a [rows][D] as a contiguous CUDA tensor `offset` elements into its buffer, and its values in 64 bits."""
    buf = torch.zeros(a.size + offset, dtype=dtype, device="cuda")
    t = buf[offset:].view(a.shape)
    t.copy_(torch.from_numpy(a))
    return t, t.double().cpu().numpy()


@pytest.mark.parametrize("T,k,E,how,D", ROWS)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1])
def test_rows(T, k, E, how, D, dtype, offset):
    rng = np.random.default_rng(T + D)
    ids = route(T, k, E, seed=T, how=how)
    plan = pnq.expert_sort(torch.from_numpy(ids).cuda(), E)
    offsets, _, order, position, _ = ref.plan(ids, E)
    used, pos = int(offsets[-1]), position.reshape(T, k)
    token = order[:used] // k
    x, xv = rows_on_gpu(rng.standard_normal((T, D)), dtype, offset)
    ys, yv = rows_on_gpu(rng.standard_normal((T * k, D)), dtype, offset)
    ys[used:] = float("nan")  # rows that no slot has are not read
    weights = rng.random((T, k)).astype(np.float32)
    wd = torch.from_numpy(weights).cuda()
    wd[torch.from_numpy(pos < 0).cuda()] = float("nan")  # nor are dropped slots' weights
    half = HALF[dtype]

    xs = pnq.expert_gather(x, plan)
    assert torch.equal(xs[:used], x[torch.from_numpy(token).cuda()]) and not xs[used:].any()

    def close(got, want, size, terms):
        err = np.abs(got.double().cpu().numpy() - want)
        assert np.all(err <= terms * 2.0 ** -24 * size + half * (np.abs(want) + terms * 2.0 ** -24 * size) + 1e-40)

    kept = np.where(pos[..., None] >= 0, yv[np.maximum(pos, 0)], 0.0)
    close(pnq.expert_gather_backward(ys, plan), kept.sum(1), np.abs(kept).sum(1), k + 1)
    y = pnq.expert_combine(ys, plan, wd)
    close(y, (weights[..., None].astype(np.float64) * kept).sum(1), (weights[..., None] * np.abs(kept)).sum(1), k + 1)
    dys, dw = pnq.expert_combine_backward(x, ys, plan, wd)
    want = weights.reshape(-1)[order[:used]].astype(np.float64)[:, None] * xv[token]
    close(dys[:used], want, np.abs(want), 1)
    assert not dys[used:].any()
    err = np.abs(dw.double().cpu().numpy() - (kept * xv[:, None, :]).sum(-1))
    assert np.all(err <= (D / 256 + 16) * 2.0 ** -24 * (np.abs(kept) * np.abs(xv[:, None, :])).sum(-1))


def test_gradients_against_differences():
    """<dy, combine(ys, weights)> moves by <dys, delta> and <dweights, delta>; <dxs, gather(x)> by <dx, delta>: both maps
    are linear, so a difference quotient of any step is exact but for rounding (fp32, 64 terms of size one: 1e-4)."""
    T, k, E, D = 6, 3, 4, 40
    rng = np.random.default_rng(0)
    plan = pnq.expert_sort(torch.from_numpy(route(T, k, E, 1, "drop")).cuda(), E)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
    x, ys, dy, w, dxs = t(T, D), t(T * k, D), t(T, D), t(T, k), t(T * k, D)
    dys, dw = pnq.expert_combine_backward(dy, ys, plan, w)
    dx = pnq.expert_gather_backward(dxs, plan)
    dot = lambda a, b: float((a.double() * b.double()).sum())  # noqa: E731
    for _ in range(4):
        a, c, d = t(T * k, D), t(T, k), t(T, D)
        for h in (1.0, 0.25):
            f = lambda s: dot(dy, pnq.expert_combine(ys + s * h * a, plan, w))  # noqa: E731
            assert abs((f(1) - f(-1)) / (2 * h) - dot(dys, a)) <= 1e-4 * 64
            f = lambda s: dot(dy, pnq.expert_combine(ys, plan, w + s * h * c))  # noqa: E731
            assert abs((f(1) - f(-1)) / (2 * h) - dot(dw, c)) <= 1e-4 * 64
            f = lambda s: dot(dxs, pnq.expert_gather(x + s * h * d, plan))  # noqa: E731
            assert abs((f(1) - f(-1)) / (2 * h) - dot(dx, d)) <= 1e-4 * 64


def test_streams():
    """A plan and rows on a stream of their own."""
    ids = torch.from_numpy(route(500, 4, 9, 3)).cuda()
    x = torch.randn(500, 96, device="cuda")
    want = pnq.expert_gather(x, pnq.expert_sort(ids, 9))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = pnq.expert_gather(x, pnq.expert_sort(ids, 9, stream=s), stream=s)
    s.synchronize()
    assert torch.equal(got, want)
