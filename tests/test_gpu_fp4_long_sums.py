"""Products whose terms have one sign, where the additions' errors do not cancel: the bound that include/pnq.h states, by every
way to sum (one CTA, K split over a cluster, pairs).

Bound: an addition to the running sum is off by one unit of its 24 bits at most, 2^-23 of it, and the running sum is at most
the whole one: K / 64 such errors; 16 more units stand for the roundings inside a step of 64, the sum over a cluster and
the scaling. Short sums: 1e-5."""
import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq
from test_gpu_fp4_shapes import shape_of

pytestmark = pytest.mark.gpu


def uniform(rows, K):
    return torch.rand(rows, K, device="cuda")


def uneven(rows, K):
    """Groups of very different size: within a step the small terms are cut off against the large ones."""
    size = torch.exp(3 * torch.randn(rows, K // 32, 1, device="cuda"))
    return (torch.randn(rows, K // 32, 32, device="cuda").abs() * size).reshape(rows, K)


def swamped(rows, K):
    """One term of 2^22, and steps of 64 terms that come to three quarters of a unit of it: a sum that is cut off stays
    where it is, the worst there is for one rounding a step."""
    x = torch.full((rows, K), 1.5 * 2.0 ** -4, device="cuda")
    x[:, :32] = 0.0
    x[:, 0] = 2048.0
    return x


def swamping(rows, K):
    w = torch.full((rows, K), 2.0 ** -4, device="cuda")
    w[:, :32] = 0.0
    w[:, 0] = 2048.0
    return w


@pytest.mark.parametrize("kind", [pnq.NVFP4, pnq.MXFP4])
@pytest.mark.parametrize("M,N,K,split", [(16, 17408, 17408, 1), (16, 3000, 17408, None), (3, 200, 65536, 8), (200, 9000, 65536, 1),
                                         (300, 17408, 17408, 1), (16, 17408, 262144, 1)])
@pytest.mark.parametrize("terms", ["uniform", "uneven", "swamped"])
def test_terms_of_one_sign(kind, M, N, K, split, terms):
    got = shape_of(M, N, K, kind)[2]
    assert got == split if split else got > 1
    torch.manual_seed(K + M)
    make = {"uniform": (uniform, uniform), "uneven": (uneven, uneven), "swamped": (swamped, swamping)}[terms]
    x, w = pnq.fp4_quantize(kind, make[0](M, K)), pnq.fp4_quantize(kind, make[1](N, K))
    y = pnq.fp4_gemm(x, w).double()
    xv, wv = pnq.fp4_dequantize(x).double(), pnq.fp4_dequantize(w)[:300].double()
    want = xv @ wv.T  # no term is negative: the sum of magnitudes too
    assert bool(((y[:, :300] - want).abs() <= max(1e-5, (K / 64 + 16) * 2.0 ** -23) * want + 1e-6).all())
