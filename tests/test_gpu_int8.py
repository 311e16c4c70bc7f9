"""The product of 8-bit integers: bit for bit. Its sum is exact, so fp32(sum) * x_scale * w_scale, one rounding a step, is the one answer
whichever kernel takes the call. The reference multiplies the codes in fp64, where sums below 2^53 are exact."""
import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq

pytestmark = pytest.mark.gpu


def codes(gen, rows, K, pitch=None, at=0):
    """Codes of every value; rows `pitch` bytes apart, the first `at` bytes past 16, other bytes of the buffer not zero."""
    pitch = pitch or -(-K // 16) * 16
    buf = torch.randint(-128, 128, (rows * pitch + at + 16,), generator=gen, device="cuda", dtype=torch.int8)
    return buf[at: at + rows * pitch].view(rows, pitch)[:, :K]


def reference(x, xs, w, ws, dtype):
    s = torch.empty(x.shape[0], w.shape[0], dtype=torch.float32, device="cuda")
    xd = x.double()
    for n in range(0, w.shape[0], 4096):
        s[:, n:n + 4096] = (xd @ w[n:n + 4096].double().T).float()
    return ((s * xs[:, None]) * ws).to(dtype)


def check(M, N, K, seed=0, x_pitch=None, w_pitch=None, x_at=0, w_at=0, dtypes=(torch.float32,)):
    gen = torch.Generator(device="cuda").manual_seed(seed + M * 1009 + N * 31 + K)
    x, w = codes(gen, M, K, x_pitch, x_at), codes(gen, N, K, w_pitch, w_at)
    xs, ws = torch.rand(M, generator=gen, device="cuda"), torch.rand(N, generator=gen, device="cuda")
    for dtype in dtypes:
        out = torch.full((M * N + 64,), 7.0, dtype=dtype, device="cuda")
        y = pnq.int8_gemm(x, xs, w, ws, out=out[:M * N].view(M, N))
        assert torch.equal(y, reference(x, xs, w, ws, dtype)), (M, N, K, dtype)
        assert bool((out[M * N:] == 7.0).all())
    assert pnq.device_error() == 0


@pytest.mark.parametrize("M", [1, 2, 3, 5, 8, 9, 15, 16, 17, 31, 33, 64, 65, 100, 128, 129, 200, 257, 400])
@pytest.mark.parametrize("N,K", [(1, 16), (130, 64), (257, 1040), (1000, 208)])
def test_rows(M, N, K):
    check(M, N, K, dtypes=(torch.float32, torch.bfloat16))


@pytest.mark.parametrize("K", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 1023, 1024, 1025, 1040, 2047, 2048, 2049, 4095, 5120, 17408])
@pytest.mark.parametrize("M", [1, 4, 7, 24, 130])
def test_lengths(M, K):
    check(M, 150, K)


@pytest.mark.parametrize("M,N,K", [(1, 17408, 5120), (4, 5120, 17408), (33, 5120, 17408), (700, 1500, 5120), (1100, 520, 2064), (1, 1, 131071), (20, 140, 131071),
                                   (2, 300, 131071), (2049, 130, 64), (16, 151936, 256), (300, 17408, 640)])
def test_sizes(M, N, K):
    check(M, N, K, dtypes=(torch.bfloat16,))


@pytest.mark.parametrize("M", [1, 3, 8, 40, 300])
@pytest.mark.parametrize("K,x_pitch,w_pitch,x_at,w_at", [(100, 100, 100, 0, 0), (100, 101, 112, 3, 16), (64, 64, 64, 1, 5), (640, 700, 650, 7, 0), (1040, 1056, 1040, 16, 8)])
def test_strides_and_alignment(M, K, x_pitch, w_pitch, x_at, w_at):
    check(M, 270, K, x_pitch=x_pitch, w_pitch=w_pitch, x_at=x_at, w_at=w_at)


@pytest.mark.parametrize("M,N,K", [(65, 1001, 2063), (128, 640, 1024), (333, 384, 7168), (512, 100, 256), (64, 4096, 4096), (20, 151936, 128), (40, 151936, 640),
                                   (300, 130, 512)])
@pytest.mark.parametrize("x_at,x_extra", [(0, 0), (5, 0), (0, 16)])
def test_small_products(M, N, K, x_at, x_extra):
    """Few tiles or few stages each: kernels that widen x themselves, from its own rows or from a copy of them on 16 bytes."""
    check(M, N, K, x_at=x_at, x_pitch=-(-K // 16) * 16 + x_extra, dtypes=(torch.float32, torch.bfloat16))


@pytest.mark.parametrize("M", [1, 5, 20, 70, 300])
@pytest.mark.parametrize("K", [1024, 1040, 4096, 131071])
def test_largest_sums(M, K):
    """Sums of one sign, of the largest codes: -128 * -128 * 131071 is the largest that 32 bits take."""
    for a, b in ((-128, -128), (127, -128), (127, 127), (-128, 1)):
        x = torch.full((M, -(-K // 16) * 16), a, dtype=torch.int8, device="cuda")[:, :K]
        w = torch.full((133, -(-K // 16) * 16), b, dtype=torch.int8, device="cuda")[:, :K]
        w[::3, : K // 2] = -b if b != -128 else 127
        one = torch.ones(max(M, 133), device="cuda")
        assert torch.equal(pnq.int8_gemm(x, one[:M], w, one[:133]), reference(x, one[:M], w, one[:133], torch.float32))


def test_the_rows_do_not_matter():
    """A token's result is the same bit for bit alone and among others."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, w = codes(gen, 600, 5120), codes(gen, 300, 5120)
    xs, ws = torch.rand(600, generator=gen, device="cuda"), torch.rand(300, generator=gen, device="cuda")
    whole = pnq.int8_gemm(x, xs, w, ws)
    for m in (1, 2, 4, 8, 13, 30, 64, 128, 250):
        assert torch.equal(pnq.int8_gemm(x[:m], xs[:m], w, ws), whole[:m])


def test_scales_that_are_not_finite():
    gen = torch.Generator(device="cuda").manual_seed(2)
    for M in (3, 50):
        x, w = codes(gen, M, 64), codes(gen, 140, 64)
        xs, ws = torch.rand(M, device="cuda"), torch.rand(140, device="cuda")
        xs[1], ws[7], xs[2] = float("nan"), float("inf"), 0.0
        y, want = pnq.int8_gemm(x, xs, w, ws), reference(x, xs, w, ws, torch.float32)
        assert torch.equal(y.isnan(), want.isnan()) and torch.equal(torch.nan_to_num(y), torch.nan_to_num(want))


def test_nothing_to_multiply():
    for M, N in ((0, 5), (5, 0), (0, 0)):
        y = pnq.int8_gemm(torch.empty(M, 16, dtype=torch.int8, device="cuda"), torch.empty(M, device="cuda"),
                          torch.empty(N, 16, dtype=torch.int8, device="cuda"), torch.empty(N, device="cuda"))
        assert y.shape == (M, N)


def test_two_streams_and_a_graph():
    """Products at once on two streams, each with workspaces of its own, and two captured ones replayed at once."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    xs, ws = torch.rand(90, generator=gen, device="cuda"), torch.rand(1500, generator=gen, device="cuda")
    x = [codes(gen, 90, 2064) for _ in range(2)]
    w = codes(gen, 1500, 2064)
    want = [reference(v, xs, w, ws, torch.float32) for v in x]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        got = [pnq.int8_gemm(v, xs, w, ws, stream=s) for v, s in zip(x, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [], []
    for v in x:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(pnq.int8_gemm(v, xs, w, ws))
        graphs.append(g)
    for _ in range(4):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_a_block_of_a_model():
    """Norm -> 8-bit product -> norm of its result with the residual -> product, against the same in 64 bits on the decoded values. Each encode
    is checked on its own input; the product of the decoded values is off by the roundings of fp32 (scales and sum: 4 u) alone."""
    T, D, H = 37, 512, 1100
    gen = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    up, down = pnq.int8_quantize(r(H, D) * D ** -0.5), pnq.int8_quantize(r(D, H) * H ** -0.5)
    x, res, norm = r(T, D).to(torch.bfloat16), r(T, D).to(torch.bfloat16), 1 + 0.1 * r(D)
    codes_, scales, total = pnq.rms_norm_int8(x, norm, 1e-6, res)
    h = pnq.int8_gemm(codes_, scales, *up)
    want = (codes_.double() * scales.double()[:, None]) @ (up[0].double() * up[1].double()[:, None]).T
    size = (codes_.double().abs() * scales.double()[:, None]) @ (up[0].double().abs() * up[1].double()[:, None]).T
    assert bool(((h.double() - want).abs() <= 4 * 2.0 ** -24 * size).all())
    q = pnq.int8_quantize(h)
    y = pnq.int8_gemm(*q, *down, dtype=torch.bfloat16)
    want = (q[0].double() * q[1].double()[:, None]) @ (down[0].double() * down[1].double()[:, None]).T
    size = (q[0].double().abs() * q[1].double()[:, None]) @ (down[0].double().abs() * down[1].double()[:, None]).T
    assert bool(((y.double() - want).abs() <= 4 * 2.0 ** -24 * size + 2.0 ** -8 * want.abs()).all())
    again = pnq.rms_norm_int8(y, norm, 1e-6, total)
    assert torch.equal(again[2], (y.float() + total.float()).to(torch.bfloat16))
