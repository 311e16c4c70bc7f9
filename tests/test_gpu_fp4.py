"""4-bit microscaled operands on the GPU against references in 64 bits: encode and decode bit for bit, the layouts place
by place, products dense and by experts within the library's GEMV bound.

Bounds. Encode and decode: none (every rounding is defined). Products: codes and scales multiply exactly, so an fp32 result
carries the fp32 accumulation alone, |y - y_exact| <= 1e-5 sum |x w| (K / 64 additions of at most 2^-23 of the running
sum each come to 1e-5 of sum |x w| at K = 5400; the error grows like their square root in practice); a bf16 result adds
half a unit in the last of 8 bits, 2^-8 |y|."""
import numpy as np
import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq
import fp4_reference as ref

pytestmark = pytest.mark.gpu

TYPES = [pnq.NVFP4, pnq.MXFP4]
FLOATS = {"fp32": torch.float32, "bf16": torch.bfloat16}


def values_like(rows, K, seed, spread=4.0):
    """Values over several binades, with exact ties, zeros and groups of zeros among them (fp32, exact in bf16)."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, K)) * np.exp(spread * rng.standard_normal((rows, 1)))
    x = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).to(torch.float32).numpy()
    x[rng.random((rows, K)) < 0.05] = 0.0
    x[rng.random((rows, K)) < 0.02] = -0.0
    ties = rng.random((rows, K)) < 0.2
    x[ties] = np.round(x[ties] * 4) / 4
    for r in range(0, rows, 3):
        x[r, 32 * (r % max(1, K // 32)):][:32] = 0.0
    return x


def on_gpu(x, dtype, offset=0, stride=None):
    """x on the GPU as `dtype`, `offset` elements into a buffer, rows `stride` elements apart."""
    rows, K = x.shape
    stride = stride or K
    buf = torch.full((offset + rows * stride + 64,), 77.0, dtype=dtype, device="cuda")
    view = torch.as_strided(buf, (rows, K), (stride, 1), offset)
    view.copy_(torch.from_numpy(x))
    return view


def read_operand(m, tiled_rows=None):
    """(codes, scale words) of an operand as numpy, place by place."""
    groups = m.K // ref.GROUP[m.type]
    packed = m.codes.cpu().numpy().reshape(m.matrices * m.rows, -1)
    rows = ref.matrix_rows(m.rows, m.matrices) if tiled_rows is None else tiled_rows
    return ref.codes_of(packed, m.K), ref.scales_of(m.scales.cpu().numpy(), rows, groups)


SHAPES = [(1, 16), (2, 32), (3, 48), (5, 64), (33, 96), (31, 272), (128, 128), (130, 288), (300, 1040), (7, 4128)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("dtype", list(FLOATS))
@pytest.mark.parametrize("rows,K", SHAPES)
@pytest.mark.parametrize("g", [1.0, 0.0173])
def test_quantize_bits(kind, dtype, rows, K, g):
    if K % ref.GROUP[kind]:
        K = K // 32 * 32 + 32
    x = values_like(rows, K, seed=rows * 1000 + K)
    for offset, stride in ((0, K), (8, K + 8), (1, K + 3)):
        xd = on_gpu(x, FLOATS[dtype], offset, stride)
        m = pnq.fp4_quantize(kind, xd, g)
        codes, words = read_operand(m)
        want_codes, want_words = ref.quantize(x, kind, g)
        assert np.array_equal(words, want_words)
        assert np.array_equal(codes, want_codes)
        v = pnq.fp4_dequantize(m).cpu().numpy()
        want = (ref.values(want_codes, want_words, kind).astype(np.float32) * np.float32(g)).astype(np.float32)
        assert np.array_equal(v.view(np.uint32), want.view(np.uint32))
        vb = pnq.fp4_dequantize(m, torch.bfloat16)
        assert torch.equal(vb.cpu(), torch.from_numpy(want).to(torch.bfloat16))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("dtype", list(FLOATS))
@pytest.mark.parametrize("rows,K", [(2600, 1040), (1301, 2080), (900, 4128), (3000, 96)])
def test_quantize_bits_many_rows(kind, dtype, rows, K):
    """Enough rows that a warp takes 1024 elements at a time, K that ends inside them; plain, and through a plan both from
    tokens and from sorted rows."""
    if K % ref.GROUP[kind]:
        K = K // 32 * 32 + 32
    x = values_like(rows, K, seed=K)
    xd = torch.from_numpy(x).cuda().to(FLOATS[dtype])
    want_codes, want_words = ref.quantize(x, kind, 0.31)
    codes, words = read_operand(pnq.fp4_quantize(kind, xd, 0.31))
    assert np.array_equal(codes, want_codes) and np.array_equal(words, want_words)
    E, k = 5, 3
    ids = route(rows, k, E, seed=K, how="drop")
    plan = pnq.expert_sort(torch.from_numpy(ids).cuda(), E)
    offsets, _, order, _, scale_row = ref.plan(ids, E)
    used = int(offsets[-1])
    token = order[:used] // k
    xs = torch.full((rows * k, K), float("nan"), dtype=FLOATS[dtype], device="cuda")
    xs[:used] = xd[torch.from_numpy(token).cuda()]
    for m in (pnq.fp4_quantize(kind, xd, 0.31, plan=plan), pnq.fp4_quantize(kind, xs, 0.31, plan=plan, sorted=True)):
        codes, words = read_operand(m, np.maximum(scale_row, 0))
        assert np.array_equal(codes[:used], want_codes[token]) and np.array_equal(words[:used], want_words[token])


def neighbours(x, dtype):
    """Exact values x > 0 of a type and their neighbours: [..., 3] as fp32."""
    bits = np.asarray(x, np.float32).view(np.int32)[..., None]
    step = 1 if dtype == "fp32" else 1 << 16
    return (bits + np.array([-step, 0, step], np.int32)).view(np.float32)


@pytest.mark.parametrize("dtype", list(FLOATS))
@pytest.mark.parametrize("copies", [1, 13])
def test_quantize_at_thresholds(dtype, copies):
    """Every E4M3 scale with elements at, just below and just above every threshold between two codes, of both signs; and
    group maxima at, below and above every threshold between two scales."""
    scales = ref.E4M3[1:127]
    t = neighbours(scales[:, None] * np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]), dtype).reshape(126, 21)
    x = np.zeros((126, 32), np.float32)
    x[:, 0] = x[:, 16] = 6 * scales
    x[:, 1:16], x[:, 17:23] = t[:, :15], t[:, 15:]
    x = np.concatenate((x, -x))
    top = neighbours(6 * (ref.E4M3[:126] + ref.E4M3[1:127]) / 2, dtype).reshape(-1)
    y = np.zeros((top.size, 32), np.float32)
    y[:, 5], y[:, 31] = top, -top
    x = np.tile(np.concatenate((x, y)), (copies, 1))
    codes, words = read_operand(pnq.fp4_quantize(pnq.NVFP4, on_gpu(x, FLOATS[dtype]), 1.0))
    want_codes, want_words = ref.quantize(x, pnq.NVFP4, 1.0)
    assert np.array_equal(words, want_words)
    assert np.array_equal(codes, want_codes)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("dtype", list(FLOATS))
@pytest.mark.parametrize("rows,K", [(3, 96), (70, 1312), (2600, 1056), (900, 4128)])
@pytest.mark.parametrize("offset,pad", [(1, 1), (2, 2), (4, 4), (3, 0)])
def test_quantize_unaligned_rows(kind, dtype, rows, K, offset, pad):
    """Rows on any of the type's own boundaries, few and many, K that ends inside a warp's elements; non-finite values lie
    between the rows and are not read into them."""
    x = values_like(rows, K, seed=K + pad)
    buf = torch.full((offset + rows * (K + pad) + 64,), float("nan"), dtype=FLOATS[dtype], device="cuda")
    xd = torch.as_strided(buf, (rows, K), (K + pad, 1), offset)
    xd.copy_(torch.from_numpy(x))
    codes, words = read_operand(pnq.fp4_quantize(kind, xd, 0.31))
    want_codes, want_words = ref.quantize(x, kind, 0.31)
    assert np.array_equal(words, want_words)
    assert np.array_equal(codes, want_codes)
    ids = route(rows, 2, 5, seed=K, how="drop")
    plan = pnq.expert_sort(torch.from_numpy(ids).cuda(), 5)
    offsets, _, order, _, scale_row = ref.plan(ids, 5)
    used = int(offsets[-1])
    codes, words = read_operand(pnq.fp4_quantize(kind, xd, 0.31, plan=plan), np.maximum(scale_row, 0))
    token = order[:used] // 2
    assert np.array_equal(codes[:used], want_codes[token]) and np.array_equal(words[:used], want_words[token])


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("dtype", list(FLOATS))
@pytest.mark.parametrize("rows,K", [(3, 96), (70, 1312), (2600, 1056)])
@pytest.mark.parametrize("offset", [0, 1, 2, 4, 8])
def test_dequantize_into_any_alignment(kind, dtype, rows, K, offset):
    """Outputs on every boundary of their type, few rows and many, groups of NaN among them; nothing is written beside them."""
    x = values_like(rows, K, seed=rows)
    x[rows // 2, 40] = np.inf
    codes, words = ref.quantize(x, kind, 0.31)
    want = torch.from_numpy((ref.values(codes, words, kind).astype(np.float32) * np.float32(0.31)).astype(np.float32)).to(FLOATS[dtype])
    buf = torch.full((offset + rows * K + 16,), 77.0, dtype=FLOATS[dtype], device="cuda")
    out = buf[offset:offset + rows * K].view(rows, K)
    pnq.fp4_dequantize(pnq.fp4_quantize(kind, on_gpu(x, torch.float32), 0.31), out=out)
    assert torch.equal(out.cpu().nan_to_num(nan=99.0), want.nan_to_num(nan=99.0)) and out.isnan().sum() == ref.GROUP[kind]
    assert bool((buf[:offset] == 77).all()) and bool((buf[offset + rows * K:] == 77).all())


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("slots", [1, 7, 33, 64])
@pytest.mark.parametrize("tokens", [3, 2500])
def test_quantize_every_slot(kind, slots, tokens):
    """Any number of slots, over 32 too, few tokens and many."""
    K, E = 160, 70
    x = values_like(tokens, K, seed=slots)
    ids = route(tokens, slots, E, seed=slots, how="even")
    ids[0] = -1
    plan = pnq.expert_sort(torch.from_numpy(ids).cuda(), E)
    offsets, _, order, _, scale_row = ref.plan(ids, E)
    used = int(offsets[-1])
    m = pnq.fp4_quantize(kind, torch.from_numpy(x).cuda(), 1.0, plan=plan)
    want_codes, want_words = ref.quantize(x, kind, 1.0)
    codes, words = read_operand(m, np.maximum(scale_row, 0))
    token = order[:used] // slots
    assert np.array_equal(codes[:used], want_codes[token]) and np.array_equal(words[:used], want_words[token])


@pytest.mark.parametrize("kind", TYPES)
def test_quantize_edges(kind):
    """Ties of every scale and code, subnormal and huge magnitudes, saturation, infinities and NaN."""
    G = ref.GROUP[kind]
    rng = np.random.default_rng(1)
    rows = []
    for e in list(range(-140, 128, 3)):
        base = np.ldexp(rng.uniform(1, 2, G), e)
        rows.append(base)
        rows.append(np.ldexp(np.array([6.0] + list(np.resize([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -5.0], G - 1))), e - 3))
    for mid in np.concatenate(((ref.E4M3[1:] + ref.E4M3[:-1]) / 2, ref.E4M3[1:])):  # amax / 6 on a tie and on a value
        rows.append(np.r_[6.0 * mid, rng.uniform(-6, 6, G - 1) * mid])
    for bad in (np.inf, -np.inf, np.nan):
        rows.append(np.r_[np.ones(G - 1), bad])
    rows.append(np.full(G, 3.4e38))
    rows.append(np.zeros(G))
    rows.append(np.r_[1e-45, np.zeros(G - 1)])
    with np.errstate(over="ignore"):
        x = np.array(rows).astype(np.float32)
    x = np.concatenate((x, x[::-1]), 1)  # two groups a row: a NaN group leaves its neighbour alone
    m = pnq.fp4_quantize(kind, torch.from_numpy(x).cuda())
    codes, words = read_operand(m)
    want_codes, want_words = ref.quantize(x, kind, 1.0)
    assert np.array_equal(words, want_words)
    assert np.array_equal(codes, want_codes)
    v = pnq.fp4_dequantize(m).cpu().numpy()
    assert np.array_equal(v, ref.values(codes, words, kind).astype(np.float32), equal_nan=True)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("matrices,rows,K", [(1, 5, 64), (3, 129, 160), (4, 128, 96)])
def test_quantize_matrices(kind, matrices, rows, K):
    x = values_like(matrices * rows, K, seed=3)
    m = pnq.fp4_quantize(kind, torch.from_numpy(x).cuda().view(matrices, rows, K), 0.5)
    codes, words = read_operand(m)
    want_codes, want_words = ref.quantize(x, kind, 0.5)
    assert np.array_equal(codes, want_codes) and np.array_equal(words, want_words)
    assert pnq.fp4_dequantize(m).shape == (matrices * rows, K)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("matrices,rows,K", [(1, 1, 32), (1, 200, 48), (3, 130, 272), (2, 77, 320)])
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_pack(kind, matrices, rows, K, offset):
    G = ref.GROUP[kind]
    K = -(-K // G) * G
    rng = np.random.default_rng(2)
    n = matrices * rows
    codes = rng.integers(0, 256, (n, K // 2), dtype=np.uint8)
    words = rng.integers(0, 255, (n, K // G), dtype=np.uint8)
    buf = torch.zeros(offset + codes.size, dtype=torch.uint8, device="cuda")
    buf[offset:] = torch.from_numpy(codes.reshape(-1)).cuda()
    m = pnq.fp4_pack(kind, buf[offset:], torch.from_numpy(words).cuda(), rows, K, 0.25, matrices)
    got = m.codes.cpu().numpy().reshape(n, -1)[:, :K // 2]
    assert np.array_equal(got, codes)
    tiled = m.scales.cpu().numpy()
    assert np.array_equal(ref.scales_of(tiled, ref.matrix_rows(rows, matrices), K // G), words)
    used = ref.tiled_place(ref.matrix_rows(rows, matrices)[:, None], np.arange(K // G)[None, :], K // G)
    rest = np.ones(tiled.size, bool)
    rest[used] = False
    assert not tiled[rest].any()  # padding words are zero


def operand(kind, rows, K, seed, matrices=1, spread=1.0):
    """A random operand on the GPU and its values in 64 bits (global multiplier 1)."""
    x = values_like(matrices * rows, K, seed, spread)
    m = pnq.fp4_quantize(kind, torch.from_numpy(x).cuda().view(matrices, rows, K) if matrices > 1 else torch.from_numpy(x).cuda())
    codes, words = ref.quantize(x, kind, 1.0)
    return m, ref.values(codes, words, kind)


def check_product(y, x, w, alpha, dtype, what=""):
    want = alpha * (x @ w.T)
    bound = abs(alpha) * (1e-5 * (np.abs(x) @ np.abs(w).T) + 1e-6)
    if dtype == torch.bfloat16:
        bound = bound + np.abs(want) * 2.0 ** -8
    err = np.abs(y.to(torch.float64).cpu().numpy() - want)
    assert np.all(err <= bound), (what, float((err / bound).max()))


GEMMS = [(5, 7, 16), (1, 1, 32), (1, 128, 64), (2, 129, 96), (3, 127, 272), (17, 64, 1056), (33, 300, 4128), (64, 256, 512),
         (65, 257, 544), (100, 130, 288), (129, 500, 320), (200, 33, 64), (256, 256, 256), (300, 1001, 2080), (513, 384, 800)]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M,N,K", GEMMS)
@pytest.mark.parametrize("dtype", list(FLOATS))
def test_gemm(kind, M, N, K, dtype):
    if K % ref.GROUP[kind]:
        K += 16
    x, xv = operand(kind, M, K, seed=M + 7 * N)
    w, wv = operand(kind, N, K, seed=N + 11 * K)
    x.global_scale, w.global_scale = 0.75, -0.125
    guard = torch.full((M * N + 64,), 5.0, dtype=FLOATS[dtype], device="cuda")
    out = guard[:M * N].view(M, N)
    y = pnq.fp4_gemm(x, w, out=out)
    torch.cuda.synchronize()
    assert pnq.device_error() == 0
    assert y is out and bool((guard[M * N:] == 5.0).all())
    check_product(y, xv, wv, 0.75 * -0.125, FLOATS[dtype], (kind, M, N, K))


@pytest.mark.parametrize("kind", TYPES)
def test_gemm_one_hot_rows(kind):
    """x = one value a row picks single weights: the products come back exactly."""
    K, N = 192, 150
    w, wv = operand(kind, N, K, seed=5)
    x = np.zeros((K, K), np.float32)
    x[np.arange(K), np.arange(K)] = 6.0  # amax 6: scale 1 (NVFP4, MXFP4), code 6
    y = pnq.fp4_gemm(pnq.fp4_quantize(kind, torch.from_numpy(x).cuda()), w)
    assert np.array_equal(y.cpu().numpy(), (6.0 * wv.T).astype(np.float32))


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M", [3, 200])
def test_gemm_nan_groups_stay_in_their_rows(kind, M):
    K, N = 160, 140
    x = values_like(M, K, 1)
    w = values_like(N, K, 2, 1.0)
    x[M // 2, 70] = np.inf
    w[N - 1, 3] = np.nan
    y = pnq.fp4_gemm(pnq.fp4_quantize(kind, torch.from_numpy(x).cuda()), pnq.fp4_quantize(kind, torch.from_numpy(w).cuda()))
    bad = np.isnan(y.cpu().numpy())
    want = np.zeros((M, N), bool)
    want[M // 2, :] = True
    want[:, N - 1] = True
    assert np.array_equal(bad, want)


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M,N,K", [(1, 5120, 17408), (16, 17408, 5120)])
def test_gemm_projection_sizes(kind, M, N, K):
    """The decode projections at full size; sampled weight rows."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    xm = pnq.fp4_quantize(kind, torch.randn(M, K, generator=gen, device="cuda"))
    wm = pnq.fp4_quantize(kind, torch.randn(N, K, generator=gen, device="cuda"))
    y = pnq.fp4_gemm(xm, wm)
    rows = np.r_[0:3, 127:130, N // 2:N // 2 + 3, N - 3:N]
    xv = pnq.fp4_dequantize(xm).double().cpu().numpy()
    wv = pnq.fp4_dequantize(wm)[torch.from_numpy(rows).cuda()].double().cpu().numpy()
    check_product(y[:, torch.from_numpy(rows).cuda()], xv, wv, 1.0, torch.float32)


def random_operand(kind, rows, K, seed, matrices=1):
    """A large random operand (codes of normal values) and its values, both on the GPU in 64 bits."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(matrices * rows, K, generator=gen, device="cuda")
    m = pnq.fp4_quantize(kind, x.view(matrices, rows, K) if matrices > 1 else x)
    return m, pnq.fp4_dequantize(m).double()  # bit for bit the definition's values (test_quantize_bits)


def check_on_gpu(y, x, w, dtype):
    want = x @ w.T
    bound = 1e-5 * (x.abs() @ w.abs().T) + 1e-6
    if dtype == torch.bfloat16:
        bound += want.abs() * 2.0 ** -8
    assert bool(((y.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M,N,K", [(700, 9000, 2048), (513, 17408, 1056), (2051, 5121, 1312), (300, 17409, 288), (1000, 1025, 8224),
                                   (20, 5120, 8192), (50, 3000, 6176), (128, 2049, 4128), (9, 1024, 17408)])
@pytest.mark.parametrize("dtype", list(FLOATS))
def test_gemm_every_shape_of_tile(kind, M, N, K, dtype):
    """Sizes that take CTA pairs, single tiles of every width, and K split over clusters of every size."""
    x, xv = random_operand(kind, M, K, M + N)
    w, wv = random_operand(kind, N, K, N + K)
    y = pnq.fp4_gemm(x, w, dtype=FLOATS[dtype])
    assert pnq.device_error() == 0
    check_on_gpu(y, xv, wv, FLOATS[dtype])


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,k,E,N,K", [(1700, 2, 8, 300, 544), (900, 4, 7, 1408, 1056), (60, 1, 16, 700, 4128), (513, 8, 64, 200, 288),
                                       (900, 2, 5, 385, 4128), (2000, 3, 3, 1000, 4352)])
def test_gemm_experts_large(kind, T, k, E, N, K):
    """Many rows per expert (256-column tiles), tiles that several experts' loads leave ragged."""
    ids = route(T, k, E, seed=T, how="skew" if E > 8 else "drop")
    plan = pnq.expert_sort(torch.from_numpy(ids).cuda(), E)
    offsets, _, order, _, _ = ref.plan(ids, E)
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn(T, K, generator=gen, device="cuda", dtype=torch.bfloat16)
    xm = pnq.fp4_quantize(kind, x, plan=plan)
    xv = pnq.fp4_dequantize(xm).double()
    token = torch.from_numpy(order[:offsets[-1]] // k).cuda()
    assert torch.equal(xv[:offsets[-1]], pnq.fp4_dequantize(pnq.fp4_quantize(kind, x)).double()[token])
    w, wv = random_operand(kind, N, K, E, matrices=E)
    y = pnq.fp4_gemm_experts(xm, w, plan)
    assert pnq.device_error() == 0 and not y[offsets[-1]:].any()
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        check_on_gpu(y[lo:hi], xv[lo:hi], wv[e * N:(e + 1) * N], torch.float32)


@pytest.mark.parametrize("M", [1, 40, 600])
def test_static_weights_chain(M):
    """Products with static weights (copied before the kernel ahead of them ends) in a chain where each encodes the last
    one's result: bit for bit the chain without the flag."""
    kind, N = pnq.NVFP4, 2048
    ws = [random_operand(kind, N, N, i)[0] for i in range(3)]
    x0 = torch.randn(M, N, device="cuda")

    def chain(flags):
        x = x0
        for i in range(12):
            x = pnq.fp4_gemm(pnq.fp4_quantize(kind, x, 0.25), ws[i % 3], flags=flags) * 0.02
        return x

    want = chain(0)
    for _ in range(3):
        assert torch.equal(chain(pnq.GEMV_STATIC_WEIGHTS), want)
    assert pnq.device_error() == 0 and bool(want.isfinite().all())


def route(T, k, E, seed, how="even"):
    rng = np.random.default_rng(seed)
    if how == "one":
        ids = np.full((T, k), E - 1)
    elif how == "none":
        ids = np.full((T, k), -1)
    elif how == "skew":
        ids = np.minimum(rng.geometric(0.3, (T, k)) - 1, E - 1)
    else:
        ids = rng.integers(0, E, (T, k))
    if how == "drop":
        ids[rng.random((T, k)) < 0.3] = -1
        ids[rng.random((T, k)) < 0.1] = E + 5
    return ids.astype(np.int32)


EXPERTS = [(1, 1, 1, 40, 64, "even"), (1, 8, 16, 130, 96, "even"), (5, 2, 3, 128, 160, "skew"), (40, 4, 9, 200, 288, "drop"),
           (70, 3, 2, 129, 320, "skew"), (300, 2, 4, 257, 544, "skew"), (260, 1, 3, 150, 96, "one"), (9, 3, 5, 60, 64, "none"),
           (700, 2, 3, 140, 288, "drop"), (33, 8, 1000, 70, 64, "even")]


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,k,E,N,K,how", EXPERTS)
@pytest.mark.parametrize("dtype", list(FLOATS))
def test_gemm_experts(kind, T, k, E, N, K, how, dtype):
    ids = route(T, k, E, seed=T + E, how=how)
    offsets, blocks, order, position, scale_row = ref.plan(ids, E)
    plan = pnq.expert_sort(torch.from_numpy(ids).cuda(), E)
    x = values_like(T, K, seed=T, spread=1.0)
    xm = pnq.fp4_quantize(kind, torch.from_numpy(x).cuda(), 0.5, plan=plan)
    used = int(offsets[-1])
    codes, words = read_operand(xm, np.maximum(scale_row, 0))
    want_codes, want_words = ref.quantize(x, kind, 0.5)
    token = order[:used] // k
    assert np.array_equal(codes[:used], want_codes[token]) and np.array_equal(words[:used], want_words[token])
    xv = ref.values(want_codes, want_words, kind)
    # the same rows, sorted already (NaN past the rows in use: they are not read)
    xs = np.full((T * k, K), np.nan, np.float32)
    xs[:used] = x[token]
    sm = pnq.fp4_quantize(kind, torch.from_numpy(xs).cuda(), 0.5, plan=plan, sorted=True)
    codes, words = read_operand(sm, np.maximum(scale_row, 0))
    assert np.array_equal(codes[:used], want_codes[token]) and np.array_equal(words[:used], want_words[token])
    back = pnq.fp4_dequantize(xm).cpu().numpy()
    assert np.array_equal(back[:used], (xv[token] * 0.5).astype(np.float32)) and not back[used:].any()

    w, wv = operand(kind, N, K, seed=E, matrices=E)
    per = torch.linspace(0.5, 2.0, E, device="cuda")
    for scale in (0.25, per):
        w.global_scale = scale
        guard = torch.full((T * k * N + 64,), 5.0, dtype=FLOATS[dtype], device="cuda")
        y = pnq.fp4_gemm_experts(xm, w, plan, out=guard[:T * k * N].view(T * k, N))
        torch.cuda.synchronize()
        assert pnq.device_error() == 0
        assert bool((guard[T * k * N:] == 5.0).all())
        assert not y[used:].any()
        for e in range(E):
            lo, hi = offsets[e], offsets[e + 1]
            if hi > lo:
                alpha = 0.5 * (0.25 if scale is not per else float(per[e]))
                check_product(y[lo:hi], xv[token[lo:hi]], wv[e * N:(e + 1) * N], alpha, FLOATS[dtype], (kind, T, k, E, e))


def test_long_rows_pass_32_bits():
    """Operands whose code offsets pass 2^31: the last rows' codes against the same rows encoded apart, their products
    (how K is split depends on the shape, so not bit for bit) against the sums in 64 bits."""
    kind, rows, K = pnq.NVFP4, 70_000, 65_536  # 2.3 GB of codes
    gen = torch.Generator(device="cuda").manual_seed(1)
    row = torch.randn(256, K, generator=gen, device="cuda", dtype=torch.bfloat16)
    x = row.repeat(-(-rows // 256), 1)[:rows]
    m = pnq.fp4_quantize(kind, x)
    last = pnq.fp4_quantize(kind, x[-300:].contiguous())
    v = torch.randn(3, K, generator=gen, device="cuda")
    vm = pnq.fp4_quantize(kind, v)
    assert torch.equal(m.codes[-300:], last.codes)
    vv, lv = (pnq.fp4_dequantize(t).double().cpu().numpy() for t in (vm, last))
    check_product(pnq.fp4_gemm(vm, m)[:, -300:], vv, lv, 1.0, torch.float32)
    check_product(pnq.fp4_gemm(m, vm)[-300:], lv, vv, 1.0, torch.float32)


def test_streams_and_graph():
    """Calls on a stream of their own, and captured in a graph, give the same bits."""
    kind, M, N, K = pnq.NVFP4, 40, 384, 512
    x = torch.from_numpy(values_like(M, K, 1, 1.0)).cuda()
    w = pnq.fp4_quantize(kind, torch.from_numpy(values_like(N, K, 2, 1.0)).cuda())
    q = pnq.fp4_quantize(kind, x)
    want = pnq.fp4_gemm(q, w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = pnq.fp4_gemm(pnq.fp4_quantize(kind, x, stream=s), w, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pnq.fp4_quantize(kind, x, out=q)
        pnq.fp4_gemm(q, w, out=out)
    x.mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, 2.0 * want)


def test_another_stream_keeps_its_tensors():
    """Calls on a stream that is behind: inputs freed after the call, and results made on that stream, are not handed to
    the current stream's allocations while the work is still to come."""
    kind, rows, K = pnq.NVFP4, 700, 2048
    w = pnq.fp4_quantize(kind, torch.randn(256, K, device="cuda"))
    x0 = torch.randn(rows, K, device="cuda")
    want = pnq.fp4_gemm(pnq.fp4_quantize(kind, x0), w)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        x = x0.clone()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)  # about 10 ms
        q = pnq.fp4_quantize(kind, x, stream=s)
        y = pnq.fp4_gemm(q, w, stream=s)
        del x, q
        junk = [torch.full((rows, K), 3.0, device="cuda") for _ in range(4)] + \
               [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (rows * K // 2, rows * K // 16) * 4]
        s.synchronize()
        assert torch.equal(y, want)
        del junk


def test_empty():
    w = pnq.fp4_quantize(pnq.NVFP4, torch.randn(5, 64, device="cuda"))
    q = pnq.fp4_quantize(pnq.NVFP4, torch.randn(0, 64, device="cuda"))
    assert pnq.fp4_gemm(q, w).shape == (0, 5)
    assert pnq.fp4_gemm(w, q).shape == (5, 0)
    assert pnq.fp4_dequantize(q).shape == (0, 64)
    plan = pnq.expert_sort(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), 3)
    assert plan.offsets.tolist() == [0, 0, 0, 0]
    xq = pnq.fp4_quantize(pnq.NVFP4, torch.randn(0, 64, device="cuda"), plan=plan)
    we = pnq.fp4_quantize(pnq.NVFP4, torch.randn(3, 7, 64, device="cuda"))
    assert pnq.fp4_gemm_experts(xq, we, plan).shape == (0, 7)
