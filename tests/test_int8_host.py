"""Refusals of the C ABI of the norms, the 8-bit rows and products, and the routing: all before anything is launched, so that
addresses that are none do no harm; and of their torch wrappers on host tensors."""
import ctypes

import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq
from block_quantized_weight_pn3t_gb300 import Status

A = 1 << 20  # an aligned address that nothing reads
F32, BF16 = 0, 1
INF = float("inf")
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    return pnq.fp4_lib()


def rule(**kw):
    r = dict(experts=8, slots=2, score=0, groups=1, top_groups=1, best=1, renormalize=0, scale=1.0) | kw
    return pnq.RouteRule(**r)


@pytest.mark.parametrize("kw,status", [
    (dict(experts=0), "SHAPE"), (dict(experts=1025), "SHAPE"), (dict(slots=0), "SHAPE"), (dict(slots=9), "SHAPE"), (dict(slots=65, experts=100), "SHAPE"),
    (dict(groups=3), "SHAPE"), (dict(groups=0), "SHAPE"), (dict(groups=64, experts=64), "SHAPE"), (dict(groups=4, top_groups=5), "SHAPE"),
    (dict(groups=4, top_groups=0), "SHAPE"), (dict(groups=4, top_groups=1, slots=3), "SHAPE"), (dict(best=0), "SHAPE"), (dict(best=3), "SHAPE"),
    (dict(score=2), "TYPE"), (dict(score=-1), "TYPE"), (dict(scale=NAN), "VALUE"), (dict(scale=INF), "VALUE")])
def test_route_rules(lib, kw, status):
    want = getattr(Status, "ERR_" + status)
    r = rule(**kw)
    assert lib.pnq_expert_route(F32, A, 2048, 4, ctypes.byref(r), None, A, A, None) == want
    assert lib.pnq_expert_route_backward(F32, A, A, 2048, A, 4, ctypes.byref(r), A, None) == want


def test_route_arguments(lib):
    r = ctypes.byref(rule())
    fwd = lambda **k: lib.pnq_expert_route(*(dict(t=F32, x=A, ld=8, n=4, r=r, b=None, i=A, w=A, s=None) | k).values())  # noqa: E731
    bwd = lambda **k: lib.pnq_expert_route_backward(*(dict(t=F32, d=A, x=A, ld=8, i=A, n=4, r=r, o=A, s=None) | k).values())  # noqa: E731
    for f in (fwd, bwd):
        assert f(t=2) == Status.ERR_TYPE and f(r=None) == Status.ERR_NULL
        assert f(ld=7) == Status.ERR_SHAPE and f(n=-1) == Status.ERR_SHAPE and f(n=1 << 30) == Status.ERR_SHAPE
        assert f(n=0, x=None, i=None) == Status.OK
        assert f(x=None) == Status.ERR_NULL and f(i=None) == Status.ERR_NULL
        assert f(x=A + 2) == Status.ERR_ALIGN and f(t=BF16, x=A + 1) == Status.ERR_ALIGN and f(i=A + 1) == Status.ERR_ALIGN
    assert fwd(w=None) == Status.ERR_NULL and fwd(b=A + 2) == Status.ERR_ALIGN
    assert bwd(d=None) == Status.ERR_NULL and bwd(o=None) == Status.ERR_NULL and bwd(o=A + 2) == Status.ERR_ALIGN


def test_norm_arguments(lib):
    def norm(**k):
        return lib.pnq_rms_norm(*(dict(t=F32, x=A, ldx=64, r=A, ldr=64, rows=4, D=64, wt=F32, w=A, eps=1e-6, total=A, y=A, rstd=A, c=A, pitch=64,
                                       s=A, st=None) | k).values())
    assert norm(t=3) == Status.ERR_TYPE and norm(wt=-1) == Status.ERR_TYPE
    for bad in (dict(rows=-1), dict(D=0), dict(ldx=63), dict(ldr=63), dict(pitch=63), dict(pitch=72), dict(rows=(1 << 30) + 1), dict(ldx=1 << 62)):
        assert norm(**bad) == Status.ERR_SHAPE, bad
    for eps in (-1e-6, NAN, INF):
        assert norm(eps=eps) == Status.ERR_VALUE
    for bad in (dict(x=None), dict(w=None), dict(s=None), dict(c=None), dict(total=None, y=None, rstd=None, c=None, s=None)):
        assert norm(**bad) == Status.ERR_NULL, bad
    for bad in (dict(x=A + 2), dict(r=A + 2), dict(w=A + 2), dict(total=A + 2), dict(y=A + 2), dict(rstd=A + 2), dict(c=A + 8), dict(s=A + 2),
                dict(t=BF16, x=A + 1)):
        assert norm(**bad) == Status.ERR_ALIGN, bad
    assert norm(rows=0, x=None, w=None) == Status.OK


def test_norm_backward_arguments(lib):
    size = ctypes.c_uint64()
    assert lib.pnq_rms_norm_backward_scratch_bytes(4, 64, ctypes.byref(size)) == Status.OK and size.value == 4 * 64 * 4
    assert lib.pnq_rms_norm_backward_scratch_bytes(4, 0, ctypes.byref(size)) == Status.ERR_SHAPE
    assert lib.pnq_rms_norm_backward_scratch_bytes(4, 64, None) == Status.ERR_NULL

    def back(**k):
        return lib.pnq_rms_norm_backward(*(dict(t=F32, dy=A, ldy=64, tot=A, ldt=64, wt=F32, w=A, rstd=A, dt=A, ldd=64, rows=4, D=64, dx=A, dw=A, scr=A,
                                                n=1024, st=None) | k).values())
    assert back(t=3) == Status.ERR_TYPE and back(wt=2) == Status.ERR_TYPE
    for bad in (dict(ldy=63), dict(ldt=1), dict(ldd=63), dict(rows=-1), dict(D=0)):
        assert back(**bad) == Status.ERR_SHAPE, bad
    for bad in (dict(dy=None), dict(tot=None), dict(w=None), dict(rstd=None), dict(dx=None), dict(scr=None)):
        assert back(**bad) == Status.ERR_NULL, bad
    for bad in (dict(dy=A + 2), dict(tot=A + 2), dict(dt=A + 2), dict(dx=A + 2), dict(dw=A + 2), dict(scr=A + 2), dict(rstd=A + 1)):
        assert back(**bad) == Status.ERR_ALIGN, bad
    assert back(n=1023) == Status.ERR_SCRATCH
    assert back(rows=0, dw=None) == Status.OK


def test_int8_arguments(lib):
    q = lambda **k: lib.pnq_int8_quantize(*(dict(t=F32, x=A, ld=40, rows=4, K=40, c=A, p=48, s=A, st=None) | k).values())  # noqa: E731
    d = lambda **k: lib.pnq_int8_dequantize(*(dict(c=A, p=40, s=A, rows=4, K=40, t=F32, o=A, st=None) | k).values())  # noqa: E731
    assert q(t=2) == Status.ERR_TYPE and d(t=2) == Status.ERR_TYPE
    for bad in (dict(ld=39), dict(p=40), dict(p=32), dict(rows=-1), dict(K=0)):
        assert q(**bad) == Status.ERR_SHAPE, bad
    for bad in (dict(p=39), dict(rows=-1), dict(K=0)):
        assert d(**bad) == Status.ERR_SHAPE, bad
    for name in "xcs":
        assert q(**{name: None}) == Status.ERR_NULL
    for name in "cso":
        assert d(**{name: None}) == Status.ERR_NULL
    assert q(x=A + 2) == Status.ERR_ALIGN and q(c=A + 8) == Status.ERR_ALIGN and q(s=A + 2) == Status.ERR_ALIGN
    assert d(s=A + 2) == Status.ERR_ALIGN and d(o=A + 2) == Status.ERR_ALIGN
    assert q(rows=0, x=None) == Status.OK and d(rows=0, c=None) == Status.OK


def test_gemm_arguments(lib):
    def gemm(**k):
        return lib.pnq_int8_gemm(*(dict(x=A, ldx=40, xs=A, M=4, w=A, ldw=48, ws=A, N=8, K=40, t=F32, y=A, scr=A, n=1 << 40, st=None) | k).values())
    assert gemm(t=5) == Status.ERR_TYPE
    for bad in (dict(K=0), dict(K=131072, ldx=131072, ldw=131072), dict(ldx=39), dict(ldw=39), dict(M=-1), dict(N=-1), dict(M=1 << 30, N=1 << 30)):
        assert gemm(**bad) == Status.ERR_SHAPE, bad
    for name in ("x", "xs", "w", "ws", "y"):
        assert gemm(**{name: None}) == Status.ERR_NULL
    assert gemm(xs=A + 2) == Status.ERR_ALIGN and gemm(ws=A + 1) == Status.ERR_ALIGN and gemm(y=A + 2) == Status.ERR_ALIGN
    assert gemm(t=BF16, y=A + 1) == Status.ERR_ALIGN
    assert gemm(M=0, x=None) == Status.OK and gemm(N=0, w=None) == Status.OK
    size = ctypes.c_uint64()
    assert lib.pnq_int8_gemm_scratch_bytes(4, A, 48, 8, 0, ctypes.byref(size)) == Status.ERR_SHAPE
    assert lib.pnq_int8_gemm_scratch_bytes(4, A, 48, 8, 40, None) == Status.ERR_NULL
    assert lib.pnq_int8_gemm_scratch_bytes(1, A, 48, 8, 40, ctypes.byref(size)) == Status.OK and size.value == 0
    assert lib.pnq_int8_gemm_scratch_bytes(600, A, 48, 8, 40, ctypes.byref(size)) == Status.OK
    if size.value:
        assert gemm(M=600, n=size.value - 1) == Status.ERR_SCRATCH and gemm(M=600, scr=None, n=0) == Status.ERR_NULL
        assert gemm(M=600, scr=A + 8, n=size.value) == Status.ERR_ALIGN


@pytest.mark.parametrize("call", [
    lambda: pnq.rms_norm(torch.zeros(2, 16), torch.zeros(16)), lambda: pnq.rms_norm_int8(torch.zeros(2, 16), torch.zeros(16)),
    lambda: pnq.int8_quantize(torch.zeros(2, 16)), lambda: pnq.expert_route(torch.zeros(2, 16), 2),
    lambda: pnq.int8_dequantize(torch.zeros(2, 16, dtype=torch.int8), torch.zeros(2)),
    lambda: pnq.int8_gemm(torch.zeros(2, 16, dtype=torch.int8), torch.zeros(2), torch.zeros(2, 16, dtype=torch.int8), torch.zeros(2)),
    lambda: pnq.expert_route_backward(torch.zeros(2, 2), torch.zeros(2, 16), torch.zeros(2, 2, dtype=torch.int32))])
def test_host_tensors_are_refused(call):
    with pytest.raises(pnq.PnqError, match="CUDA"):
        call()


@pytest.mark.parametrize("call", [lambda: pnq.rms_norm(torch.zeros(2, 16, dtype=torch.float16), torch.zeros(16)), lambda: pnq.int8_quantize([1.0]),
                                  lambda: pnq.int8_quantize(torch.zeros(2, 16, dtype=torch.int8)), lambda: pnq.expert_route(torch.zeros(2, 4, dtype=torch.int32), 2),
                                  lambda: pnq.int8_gemm(torch.zeros(2, 16), torch.zeros(2), torch.zeros(2, 16), torch.zeros(2))])
def test_other_types_are_refused(call):
    with pytest.raises(pnq.PnqError, match="dtype|torch.Tensor"):
        call()


def test_calls_with_bad_keywords():
    for call in (pnq.rms_norm, pnq.rms_norm_int8, pnq.rms_norm_backward, pnq.int8_quantize, pnq.int8_dequantize, pnq.int8_gemm, pnq.expert_route,
                 pnq.expert_route_backward):
        with pytest.raises(TypeError):
            call()
        with pytest.raises(TypeError):
            call(nothing=1)
