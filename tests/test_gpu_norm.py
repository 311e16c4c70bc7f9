"""The norms and the 8-bit encode against their definitions in 64 bits.

Bounds, in units of u = 2^-24 (half a step of fp32). A thread adds at most `serial` squares in a row and their sum goes through five more
additions in its warp, and then five through the CTA, or one for each of the row's warps (at most D / 1024 of 32 lanes with 32 squares
each): the mean is within (serial + 10 + D / 1024) u of itself, its root within half of that, and root, reciprocal, the two products and the
division by 127 round at most 6 times more. bf16 results are off by another 2^-8 of themselves (eps / 2)."""
import math

import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-6


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rel(D):
    return ((max(32, -(-D // 1024)) + 10 + D // 1024) / 2 + 6) * U


def inputs(rows, D, dtype, wdtype, residual, seed=0, stride=None):
    gen = torch.Generator(device="cuda").manual_seed(seed + rows * 131 + D)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    loud = 1 + 6 * (torch.rand(stride or D, generator=gen, device="cuda") < 0.1)
    x = (r(rows, stride or D) * loud).to(dtype)[:, :D]
    res = (r(rows, stride or D) * loud).to(dtype)[:, (stride or D) - D:] if residual else None
    return x, (1 + 0.2 * r(D)).to(wdtype), res


def total_of(x, res):
    return x if res is None else (x.float() + res.float()).to(x.dtype)


def by_127(top):
    """fp32(top / 127): divided in 64 bits (torch divides an fp32 tensor by a number through its reciprocal; a quotient of 24 bits by 7 is never so near
    to the middle of two fp32 numbers that the second rounding matters)."""
    return (top.double() / 127).float()


def codes_of(p):
    """The definition in 64 bits: p holds fp32 values; the border between two codes is decided by exact products."""
    p = p.double()
    top = p.abs().amax(1, keepdim=True)
    low = torch.floor(torch.where(top > 0, 127 * p.abs() / top, 0.0))
    twice, middle = 254 * p.abs(), (2 * low + 1) * top
    q = low + ((twice > middle) | ((twice == middle) & (low % 2 == 1)))
    return (torch.sign(p) * torch.where(top > 0, q, 0.0)).to(torch.int8), top[:, 0]


SHAPES = [(1, 1), (1, 5120), (3, 7), (2, 2), (5, 96), (7, 255), (33, 256), (4, 257), (1000, 64), (9, 1999), (301, 2048), (17, 4100), (3, 8192),
          (2, 8193), (2, 16390), (3, 17408), (2, 32768), (2, 33001), (1, 70000), (2000, 96), (1700, 504), (900, 5120), (700, 8200), (650, 20480)]


@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm(rows, D, dtype):
    for wdtype, residual in ((torch.float32, True), (torch.bfloat16, False)):
        x, w, res = inputs(rows, D, dtype, wdtype, residual)
        y, total, rstd = pnq.rms_norm(x, w, EPS, res)
        assert torch.equal(total, total_of(x, res))
        t = total.double()
        r = 1 / torch.sqrt((t * t).mean(1) + EPS)
        assert bool(((rstd.double() - r).abs() <= rel(D) * r).all())
        want = t * r[:, None] * w.double()
        bound = (rel(D) + (half_step(dtype) if dtype != torch.float32 else 0)) * want.abs() * 1.01
        assert bool(((y.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("rows,D", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_int8(rows, D, dtype):
    for wdtype, residual in ((torch.float32, True), (torch.bfloat16, False)):
        x, w, res = inputs(rows, D, dtype, wdtype, residual)
        y = torch.empty(rows, D, dtype=dtype, device="cuda")
        codes, scales, total = pnq.rms_norm_int8(x, w, EPS, res, y=y)
        assert torch.equal(total, total_of(x, res))
        want, top = codes_of(total.float() * w.float())
        assert torch.equal(codes, want)
        t = total.double()
        s = top / torch.sqrt((t * t).mean(1) + EPS) / 127
        assert bool(((scales.double() - s).abs() <= rel(D) * s).all())
        assert torch.equal(y, pnq.rms_norm(x, w, EPS, res)[0])
        assert codes.stride(0) == -(-D // 16) * 16 or rows == 1
        assert torch.equal(pnq.int8_dequantize(codes, scales), codes.float() * scales[:, None])
        assert torch.equal(pnq.int8_dequantize(codes, scales, dtype=torch.bfloat16), (codes.float() * scales[:, None]).to(torch.bfloat16))


@pytest.mark.parametrize("rows,K", SHAPES + [(1500, 5120)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("extra", [0, 1, 8])
def test_quantize(rows, K, dtype, extra):
    x = inputs(rows, K, dtype, dtype, False, stride=K + extra)[0]
    codes, scales = pnq.int8_quantize(x)
    want, top = codes_of(x.float())
    assert torch.equal(codes, want)
    assert torch.equal(scales, by_127(top))


@pytest.mark.parametrize("rows,K", [(1, 1), (5, 127), (3, 128), (700, 129), (333, 2063), (2100, 1000), (9000, 1024), (40, 30001)])
@pytest.mark.parametrize("at,extra", [(0, 0), (0, 1), (1, 3), (4, 8)])
def test_decode_of_any_rows(rows, K, at, extra):
    """Codes `at` bytes into a buffer, rows K + extra bytes apart: code * scale in fp32, rounded once more for bf16; bytes behind a row are not read."""
    gen = torch.Generator(device="cuda").manual_seed(rows + K)
    buf = torch.randint(-128, 128, (at + rows * (K + extra) + 16,), generator=gen, device="cuda", dtype=torch.int8)
    codes, scales = buf[at: at + rows * (K + extra)].view(rows, K + extra)[:, :K], torch.rand(rows, generator=gen, device="cuda")
    want = codes.float() * scales[:, None]
    assert torch.equal(pnq.int8_dequantize(codes, scales), want)
    assert torch.equal(pnq.int8_dequantize(codes, scales, dtype=torch.bfloat16), want.to(torch.bfloat16))


def test_codes_on_the_borders():
    """Rows whose values lie on borders between codes, one step of fp32 to either side of them, and rows of every magnitude."""
    k = torch.arange(-127, 127, device="cuda", dtype=torch.float32) + 0.5
    up, down = torch.nextafter(k, k.new_full((), math.inf)), torch.nextafter(k, k.new_full((), -math.inf))
    base = torch.cat((k, up, down, k.new_tensor([127.0, -127.0, 0.0, -0.0])))
    for scale in [2.0 ** e for e in range(-148, 120, 3)] + [1.0 / 3, 1e-3, 1.2345e-30, 3.21e30]:
        x = (base * scale)[None].contiguous()
        codes, scales = pnq.int8_quantize(x)
        want, top = codes_of(x)
        assert torch.equal(codes, want), scale
        assert torch.equal(scales, by_127(top))
    b = torch.arange(-254, 255, device="cuda").to(torch.bfloat16)[None] / 2  # every border is a tie in bf16
    codes, _ = pnq.int8_quantize(b)
    assert torch.equal(codes, torch.round(b.float()).to(torch.int8))


def test_rows_without_values():
    """Rows of zeros, and NaN or infinities: they stay in their rows."""
    x = torch.randn(7, 300, device="cuda")
    clean = x.clone()
    x[1] = 0.0
    x[2, 5] = math.nan
    x[3, 299] = math.inf
    x[4, 0] = -math.inf
    w = torch.ones(300, device="cuda")
    want, want_scales, _ = pnq.rms_norm_int8(clean, w)
    for codes, scales in (pnq.rms_norm_int8(x, w)[:2], pnq.int8_quantize(x)):
        assert bool((codes[1:5] == 0).all()) and float(scales[1]) == 0.0
        assert bool(scales[2:5].isnan().all()) and bool(scales[[0, 1, 5, 6]].isfinite().all())
    codes, scales, _ = pnq.rms_norm_int8(x, w)
    assert torch.equal(codes[[0, 5, 6]], want[[0, 5, 6]]) and torch.equal(scales[[0, 5, 6]], want_scales[[0, 5, 6]])
    y, _, rstd = pnq.rms_norm(x, w)
    assert bool((y[1] == 0).all()) and float(rstd[1]) == pytest.approx(EPS ** -0.5, rel=1e-6)
    assert bool(y[2].isnan().all()) and bool(y[[0, 1, 5, 6]].isfinite().all())
    w[17] = math.nan
    codes, scales, _ = pnq.rms_norm_int8(clean, w)
    assert bool(scales.isnan().all()) and bool((codes == 0).all())


def test_rows_of_zeros_without_eps():
    """r is infinite there: y and the scale are NaN, the codes zero, and other rows do not see it."""
    x, w = torch.randn(3, 96, device="cuda"), torch.ones(96, device="cuda")
    x[1] = 0
    for rows in (x, x.repeat(400, 1)):
        y, _, rstd = pnq.rms_norm(rows, w, 0.0)
        codes, scales, _ = pnq.rms_norm_int8(rows, w, 0.0)
        assert bool(y[1].isnan().all()) and bool(rstd[1].isinf()) and bool(scales[1].isnan()) and not bool(codes[1].any())
        assert bool(y[[0, 2]].isfinite().all()) and bool(scales[[0, 2]].isfinite().all())
    assert float(pnq.int8_quantize(x)[1][1]) == 0.0


@pytest.mark.parametrize("rows,D", [(6, 2048), (6, 1999), (6, 40000), (2000, 2048), (1500, 5120), (2001, 264), (900, 17408), (1300, 999)])
def test_in_place_and_given_buffers(rows, D):
    x, w, res = inputs(rows, D, torch.bfloat16, torch.float32, True)
    y, total, rstd = pnq.rms_norm(x, w, EPS, res)
    pitch = -(-D // 16) * 16 + 32
    wide = torch.full((rows, pitch), 99, dtype=torch.int8, device="cuda")
    codes, scales, _ = pnq.rms_norm_int8(x, w, EPS, res)
    held = res.clone()
    c, s, t = pnq.rms_norm_int8(x, w, EPS, held, codes=wide[:, :D], scales=torch.empty(rows, device="cuda"), total=held)
    assert t is held and torch.equal(held, total) and torch.equal(c, codes) and torch.equal(s, scales)
    assert bool((wide[:, D:] == 99).all())
    xx, held = x.clone(), res.clone()
    yy, tt, rr = pnq.rms_norm(xx, w, EPS, held, out=xx, total=held)
    assert yy is xx and tt is held and torch.equal(xx, y) and torch.equal(held, total) and torch.equal(rr, rstd)


@pytest.mark.parametrize("rows,D", SHAPES + [(0, 40), (700, 512), (5000, 136), (64, 4096), (200, 999), (24, 130), (120, 8191)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward(rows, D, dtype):
    """Against the formula in 64 bits; the bound of dx counts the terms that cancel, that of dweight every term of its sum."""
    for wdtype, dt in ((torch.float32, True), (torch.bfloat16, False)):
        x, w, _ = inputs(rows, D, dtype, wdtype, False)
        gen = torch.Generator(device="cuda").manual_seed(5)
        dy = torch.randn(rows, D, generator=gen, device="cuda").to(dtype)
        dtotal = torch.randn(rows, D + 3, generator=gen, device="cuda").to(dtype)[:, 3:] if dt else None
        _, total, rstd = pnq.rms_norm(x, w, EPS)
        dx, dw = pnq.rms_norm_backward(dy, total, w, rstd, dtotal)
        r = rstd.double()[:, None]
        n, g = total.double() * r, dy.double() * w.double()
        mean, size = (g * n).sum(1, keepdim=True) / D, (g * n).abs().sum(1, keepdim=True) / D
        want = r * (g - n * mean) + (dtotal.double() if dt else 0)
        serial = max(32, -(-D // 1024))
        bound = r * (6 * g.abs() + n.abs() * (serial + 18) * size) * U + (half_step(dtype) + U) * want.abs() * 1.01 + 1e-30
        assert bool(((dx.double() - want).abs() <= bound).all())
        want = (dy.double() * n).sum(0)
        assert bool(((dw.double() - want).abs() <= (rows + 64) * U * (dy.double() * n).abs().sum(0) + 1e-30).all())
        again = pnq.rms_norm_backward(dy, total, w, rstd, dtotal)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


def test_backward_against_differences():
    """Central differences of sum(y dy) + sum(total dtotal) in 64 bits on the forward's definition."""
    rows, D, h = 3, 24, 1e-5
    x, w, res = inputs(rows, D, torch.float32, torch.float32, True)
    dy, dtotal = torch.randn(rows, D, device="cuda"), torch.randn(rows, D, device="cuda")
    _, total, rstd = pnq.rms_norm(x, w, EPS, res)
    dx, dw = pnq.rms_norm_backward(dy, total, w, rstd, dtotal)

    def loss(t, w):
        return ((t / torch.sqrt((t * t).mean(1, keepdim=True) + EPS) * w * dy.double()).sum() + (t * dtotal.double()).sum())

    t, ww = total.double(), w.double()
    for i in range(rows):
        for j in range(0, D, 5):
            step = torch.zeros_like(t)
            step[i, j] = h
            assert float(dx[i, j]) == pytest.approx(float((loss(t + step, ww) - loss(t - step, ww)) / (2 * h)), rel=1e-5, abs=1e-6)
    for j in range(D):
        step = torch.zeros_like(ww)
        step[j] = h
        assert float(dw[j]) == pytest.approx(float((loss(t, ww + step) - loss(t, ww - step)) / (2 * h)), rel=1e-5, abs=1e-6)


def test_backward_in_place():
    """dx may take dtotal's buffer, not dy's or the total's: those may be read for the weight's gradient after it is written."""
    for rows, D in ((40, 512), (3000, 512)):
        dy, t, dt = (torch.randn(rows, D, device="cuda") for _ in range(3))
        w, rstd = torch.randn(D, device="cuda"), torch.rand(rows, device="cuda")
        want = pnq.rms_norm_backward(dy, t, w, rstd, dt)
        got = pnq.rms_norm_backward(dy, t, w, rstd, dt, out=dt)
        assert got[0] is dt and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        for out in (dy, t):
            with pytest.raises(RuntimeError):
                pnq.rms_norm_backward(dy, t, w, rstd, out=out)


def test_capture_and_another_stream():
    """A captured norm with its gradients replays on new inputs; a call on another stream answers the same."""
    x, w, res = inputs(65, 1536, torch.bfloat16, torch.float32, True)
    dy = torch.randn_like(x)

    def step():
        y, total, rstd = pnq.rms_norm(x, w, EPS, res)
        return (y, total, *pnq.rms_norm_backward(dy, total, w, rstd), *pnq.rms_norm_int8(x, w, EPS, res))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(torch.randn_like(x))
    dy.copy_(torch.randn_like(x))
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, step()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, total, rstd = pnq.rms_norm(x, w, EPS, res, stream=side)
    dx, dw = pnq.rms_norm_backward(dy, total, w, rstd, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(out, (y, total, dx, dw)):
        assert torch.equal(a, b)
