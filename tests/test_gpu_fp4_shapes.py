"""Dense products through every kernel that a size can lead to: each width of tile, CTA pairs, and K split over every number of
CTAs. Which kernel a size takes is asked of the library (pnq_fp4_gemm_shape) and asserted, so that a changed estimate cannot
take one out of these tests unseen.

Bound: codes and scales multiply exactly; the K / 64 additions to a sum round or truncate by at most 2^-23 of its magnitude
each, (K / 64) 2^-23 sum |x w| or, for short sums, 1e-5 of it; half a unit of 8 bits, 2^-8 |y|, for bf16."""
import ctypes

import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq
from test_gpu_fp4 import random_operand, route

pytestmark = pytest.mark.gpu

TYPES = [pnq.NVFP4, pnq.MXFP4]
FLOATS = [torch.float32, torch.bfloat16]

# sizes that end inside a tile on every side, the cheapest first
CANDIDATES = sorted(((M, N, K) for M in (3, 29, 40, 61, 97, 129, 150, 201, 257, 300, 500, 700, 1000)
                     for N in (129, 700, 1025, 2049, 3001, 4001, 5121, 9001)
                     for K in (288, 1056, 4128, 6176, 8224, 10272, 17440, 32800)), key=lambda s: s[0] * s[1] * s[2])
SPLITS = [(32, s) for s in range(1, 9)] + [(64, s) for s in range(1, 9)] + [(128, s) for s in (1, 2, 3, 4, 5, 6, 8)]


def shape_of(M, N, K, kind=pnq.NVFP4):
    """(columns, CTAs of a tile, CTAs that share K) of a dense product."""
    torch.zeros(1, device="cuda")  # a context
    out = [ctypes.c_int32() for _ in range(3)]
    assert pnq.fp4_lib().pnq_fp4_gemm_shape(kind, M, N, K, *[ctypes.byref(v) for v in out]) == 0
    return tuple(v.value for v in out)


def check(y, x, w, K, dtype):
    want = x @ w.T
    bound = max(1e-5, K / 64 * 2.0 ** -23) * (x.abs() @ w.abs().T) + 1e-6
    if dtype == torch.bfloat16:
        bound += want.abs() * 2.0 ** -8
    assert bool(((y.double() - want).abs() <= bound).all())


def guarded_product(x, w, dtype, flags=0):
    M, N = x.rows, w.rows
    buf = torch.full((M * N + 64,), 5.0, dtype=dtype, device="cuda")
    y = pnq.fp4_gemm(x, w, out=buf[:M * N].view(M, N), flags=flags)
    assert pnq.device_error() == 0 and bool((buf[M * N:] == 5.0).all())
    return y


@pytest.mark.parametrize("columns,split", SPLITS)
@pytest.mark.parametrize("kind", TYPES)
def test_every_width_and_split(columns, split, kind):
    sizes = [s for s in CANDIDATES if shape_of(*s, kind) == (columns, 1, split)][:2]
    assert sizes, "no size leads to this kernel any more"
    for M, N, K in sizes:
        x, xv = random_operand(kind, M, K, M + N)
        w, wv = random_operand(kind, N, K, N + K)
        for dtype in FLOATS:
            check(guarded_product(x, w, dtype), xv, wv, K, dtype)


@pytest.mark.parametrize("M,N,K", [(129, 17409, 1056), (500, 5121, 1056), (2100, 9001, 4128), (8191, 301, 1056), (4097, 9100, 544)])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("dtype", FLOATS)
def test_dense_pairs(M, N, K, kind, dtype):
    """CTA pairs with remainders in M (in the second CTA's half, and one row past a tile), N (either CTA's half) and K; the
    same bits with static weights, copied early by both CTAs."""
    assert shape_of(M, N, K, kind) == (256, 2, 1)
    x, xv = random_operand(kind, M, K, M + N)
    w, wv = random_operand(kind, N, K, N + K)
    y = guarded_product(x, w, dtype)
    check(y, xv, wv, K, dtype)
    for _ in range(2):
        assert torch.equal(guarded_product(x, w, dtype, pnq.GEMV_STATIC_WEIGHTS), y)


def test_static_weights_chain_of_pairs():
    """Pairs with static weights in a chain where each product's rows are the last one's results, encoded: bit for bit the
    chain without the flag."""
    kind, M, N = pnq.NVFP4, 2050, 5120
    assert shape_of(M, N, N) == (256, 2, 1)
    ws = [random_operand(kind, N, N, i)[0] for i in range(2)]
    x0 = torch.randn(M, N, device="cuda")

    def chain(flags):
        x = x0
        for i in range(6):
            x = pnq.fp4_gemm(pnq.fp4_quantize(kind, x, 0.25), ws[i % 2], flags=flags) * 0.012
        return x

    want = chain(0)
    assert torch.equal(chain(pnq.GEMV_STATIC_WEIGHTS), want)
    assert pnq.device_error() == 0 and bool(want.isfinite().all())


@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,k,E,N,K", [(900, 2, 5, 385, 4128), (1700, 2, 8, 300, 544), (900, 4, 7, 1408, 1056), (50, 1, 16, 130, 1056)])
def test_experts_to_bf16(kind, T, k, E, N, K):
    """The experts' kernels (pairs, 256, 128 and 64 columns) with bf16 results."""
    ids = torch.from_numpy(route(T, k, E, seed=T, how="drop")).cuda()
    plan = pnq.expert_sort(ids, E)
    x = pnq.fp4_quantize(kind, torch.randn(T, K, device="cuda"), plan=plan)
    w, wv = random_operand(kind, N, K, E, matrices=E)
    xv, offsets = pnq.fp4_dequantize(x).double(), plan.offsets.tolist()
    buf = torch.full((T * k * N + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
    y = pnq.fp4_gemm_experts(x, w, plan, out=buf[:T * k * N].view(T * k, N))
    assert pnq.device_error() == 0 and bool((buf[T * k * N:] == 5.0).all()) and not y[offsets[-1]:].any()
    for e in range(E):
        lo, hi = offsets[e], offsets[e + 1]
        check(y[lo:hi], xv[lo:hi], wv[e * N:(e + 1) * N], K, torch.bfloat16)
