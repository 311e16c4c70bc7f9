"""Refusals of the torch wrappers of the norms, the 8-bit rows and products, and the routing that take CUDA tensors to reach. Every one is
raised before anything is launched."""
import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq

pytestmark = pytest.mark.gpu


def t(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def i8(*shape):
    return t(*shape, dtype=torch.int8)


NORM = [
    (lambda: pnq.rms_norm(t(2, 16), t(15)), "weight has shape"), (lambda: pnq.rms_norm(t(2, 16), t(1, 16)), "weight has shape"),
    (lambda: pnq.rms_norm(t(16), t(16)), r"\[rows\]\[columns\]"), (lambda: pnq.rms_norm(t(2, 0), t(0)), "no elements"),
    (lambda: pnq.rms_norm(t(16, 2).T, t(16)), "must be consecutive"), (lambda: pnq.rms_norm(t(2, 16), t(32)[::2]), "contiguous"),
    (lambda: pnq.rms_norm(t(2, 16), t(16), 1e-6, t(3, 16)), "another shape or dtype"),
    (lambda: pnq.rms_norm(t(2, 16), t(16), 1e-6, t(2, 16, dtype=torch.bfloat16)), "another shape or dtype"),
    (lambda: pnq.rms_norm(t(2, 16), t(16), out=t(2, 15)), "out has shape"), (lambda: pnq.rms_norm(t(2, 16), t(16), out=t(2, 16, dtype=torch.bfloat16)), "out has dtype"),
    (lambda: pnq.rms_norm(t(2, 16), t(16), total=t(2, 16)), "total is x"), (lambda: pnq.rms_norm(t(2, 16), t(16), 1e-6, t(2, 16), total=t(2, 32)[:, :16]), "contiguous"),
    (lambda: pnq.rms_norm(t(1, 16).expand(4, 16), t(16)), "elements apart"),
    (lambda: pnq.rms_norm_int8(t(2, 20), t(20), codes=i8(2, 20)), "16 bytes"), (lambda: pnq.rms_norm_int8(t(2, 16), t(16), codes=i8(2, 32)), "codes have shape"),
    (lambda: pnq.rms_norm_int8(t(2, 16), t(16), codes=t(2, 16)), "dtype"), (lambda: pnq.rms_norm_int8(t(2, 16), t(16), scales=t(3)), "scales has shape"),
    (lambda: pnq.rms_norm_int8(t(2, 16), t(16), y=t(2, 17)), "y has shape"),
    (lambda: pnq.rms_norm_backward(t(2, 16), t(2, 17), t(17), t(2)), "dy has another"), (lambda: pnq.rms_norm_backward(t(2, 16), t(2, 16), t(16), t(3)), "rstd has shape"),
    (lambda: pnq.rms_norm_backward(t(2, 16), t(2, 16), t(16), t(2), t(2, 15)), "dtotal has another"),
    (lambda: pnq.rms_norm_backward(t(2, 16), t(2, 16), t(16), t(2), dweight=t(15)), "dweight has shape"),
    (lambda: pnq.int8_quantize(t(2, 16, 4)), r"\[rows\]\[columns\]"), (lambda: pnq.int8_quantize(t(4, 0)), "no elements"),
    (lambda: pnq.int8_quantize(t(2, 16), codes=i8(33)[1:].view(2, 16)), "16 bytes"),
    (lambda: pnq.int8_dequantize(i8(2, 16), t(3)), "scales has shape"), (lambda: pnq.int8_dequantize(i8(2, 16), t(2), dtype=torch.float16), "dtype"),
    (lambda: pnq.int8_gemm(i8(2, 16), t(2), i8(3, 17), t(3)), "operands differ"), (lambda: pnq.int8_gemm(i8(2, 16), t(3), i8(3, 16), t(3)), "x_scales has shape"),
    (lambda: pnq.int8_gemm(i8(2, 16), t(2), i8(3, 16), t(2)), "w_scales has shape"), (lambda: pnq.int8_gemm(i8(2, 0), t(2), i8(3, 0), t(3)), "131071"),
    (lambda: pnq.int8_gemm(i8(1, 131072), t(1), i8(1, 131072), t(1)), "131071"), (lambda: pnq.int8_gemm(i8(16, 2).T, t(2), i8(3, 16), t(3)), "consecutive"),
    (lambda: pnq.int8_gemm(i8(2, 16), t(2), i8(3, 16), t(3), out=t(2, 4)), "out has shape"), (lambda: pnq.int8_gemm(i8(2, 16), t(2), i8(3, 16), t(3), dtype=torch.int32), "dtype"),
    (lambda: pnq.expert_route(t(2, 8), 9), "slots"), (lambda: pnq.expert_route(t(2, 8), 0), "slots"), (lambda: pnq.expert_route(t(2, 1025), 2), "experts"),
    (lambda: pnq.expert_route(t(2, 8), 2, groups=3), "groups"), (lambda: pnq.expert_route(t(2, 8), 3, groups=4, top_groups=1), "slots"),
    (lambda: pnq.expert_route(t(2, 8), 2, groups=4, top_groups=5), "top_groups"), (lambda: pnq.expert_route(t(2, 8), 2, best=3), "best"),
    (lambda: pnq.expert_route(t(2, 8), 2, score=7), "score"), (lambda: pnq.expert_route(t(2, 8), 2, bias=t(7)), "bias has shape"),
    (lambda: pnq.expert_route(t(2, 8), 2, bias=t(8, dtype=torch.bfloat16)), "bias has dtype"), (lambda: pnq.expert_route(t(2, 8), 2, scale=float("nan")), "pnq_expert_route"),
    (lambda: pnq.expert_route(t(2, 8), 2, ids=t(2, 2)), "ids has dtype"), (lambda: pnq.expert_route(t(2, 8), 2, weights=t(2, 3)), "weights has shape"),
    (lambda: pnq.expert_route_backward(t(2, 2), t(2, 8), t(2, 3, dtype=torch.int32)), "dweights has shape"),
    (lambda: pnq.expert_route_backward(t(2, 2), t(3, 8), t(2, 2, dtype=torch.int32)), "ids has shape"),
    (lambda: pnq.expert_route_backward(t(2, 2), t(2, 8), t(2, 2, dtype=torch.int64)), "ids has dtype"),
]


@pytest.mark.parametrize("call,match", NORM)
def test_refusals(call, match):
    with pytest.raises(pnq.PnqError, match=match):
        call()


@pytest.mark.parametrize("eps", [-1.0, float("nan"), float("inf")])
def test_eps(eps):
    with pytest.raises(pnq.PnqError) as e:
        pnq.rms_norm(t(2, 16), t(16), eps)
    assert e.value.status == pnq.Status.ERR_VALUE


def test_no_rows():
    """Nothing to do is no error: empty results, and a weight's gradient of zeros."""
    y, total, rstd = pnq.rms_norm(t(0, 16), t(16))
    assert y.shape == total.shape == (0, 16) and rstd.shape == (0,)
    assert [tuple(v.shape) for v in pnq.rms_norm_int8(t(0, 16), t(16))] == [(0, 16), (0,), (0, 16)]
    assert pnq.int8_dequantize(*pnq.int8_quantize(t(0, 7))).shape == (0, 7)
    dx, dw = pnq.rms_norm_backward(t(0, 16), t(0, 16), t(16), t(0))
    assert dx.shape == (0, 16) and bool((dw == 0).all())
    ids, w = pnq.expert_route(t(0, 8), 3)
    assert ids.shape == w.shape == (0, 3)
    assert pnq.expert_route_backward(w, t(0, 8), ids).shape == (0, 8)


def test_results_require_no_gradient():
    """Outside autograd, as the expert layer's calls."""
    x, w = t(4, 16).requires_grad_(), t(16).requires_grad_()
    for out in (*pnq.rms_norm(x, w)[::2], *pnq.rms_norm_int8(x, w)[:2], *pnq.int8_quantize(x), *pnq.expert_route(x, 2)):
        assert not out.requires_grad
