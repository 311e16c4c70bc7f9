"""Results of the norms and the routing's gradient that stand partly where an operand does, or two results in one place: refused by the
C ABI before anything is launched, so that addresses that are none do no harm."""
import ctypes

import pytest

import block_quantized_weight_pn3t_gb300 as pnq
from block_quantized_weight_pn3t_gb300 import Status

F32, BF16 = 0, 1
M = 1 << 20  # buffers a megabyte apart; rows = 4 of D = 64 fp32 take 1024 bytes


@pytest.fixture(scope="module")
def lib():
    return pnq.fp4_lib()


def norm(lib, **k):
    a = dict(t=F32, x=1 * M, ldx=64, r=2 * M, ldr=64, rows=4, D=64, wt=F32, w=3 * M, eps=1e-6, total=4 * M, y=5 * M, rstd=6 * M, c=7 * M, pitch=64,
             s=8 * M, st=None) | k
    return lib.pnq_rms_norm(*a.values())


@pytest.mark.parametrize("bad", [
    dict(total=5 * M), dict(y=4 * M + 1020), dict(y=4 * M - 1020),                      # y and total in one place
    dict(y=1 * M + 256), dict(y=1 * M + 4), dict(y=1 * M - 4), dict(total=2 * M + 256),  # a row or an element off
    dict(y=2 * M + 1020), dict(total=1 * M - 1020),
    dict(y=1 * M, ldx=65), dict(total=2 * M, ldr=128), dict(y=1 * M + 3 * 4000, ldx=1000), dict(y=1 * M + 3 * 4000 + 252, ldx=1000),
    dict(t=BF16, y=1 * M + 2), dict(t=BF16, y=1 * M + 510), dict(rows=1, total=5 * M)])
def test_norm(lib, bad):
    assert norm(lib, **bad) == Status.ERR_VALUE


@pytest.mark.parametrize("bad", [
    dict(dx=1 * M), dict(dx=2 * M), dict(dx=1 * M + 256), dict(dx=2 * M - 1020), dict(dx=1 * M + 12000, ldy=1000), dict(dx=1 * M, rows=1), dict(dx=1 * M, ldy=80, dw=None),
    dict(dx=5 * M + 4), dict(dx=5 * M, ldd=65), dict(dx=5 * M - 1020)])
def test_norm_gradient(lib, bad):
    a = dict(t=F32, dy=1 * M, ldy=64, tot=2 * M, ldt=64, wt=F32, w=3 * M, rstd=4 * M, dt=5 * M, ldd=64, rows=4, D=64, dx=6 * M, dw=7 * M, scr=8 * M, n=1 << 20,
             st=None) | bad
    assert lib.pnq_rms_norm_backward(*a.values()) == Status.ERR_VALUE


@pytest.mark.parametrize("bad", [dict(o=2 * M + 32), dict(o=2 * M - 4), dict(ld=9, o=2 * M), dict(ld=9, o=2 * M + 3 * 36 + 28), dict(t=BF16, o=2 * M + 62)])
def test_routing_gradient(lib, bad):
    rule = pnq.RouteRule(experts=8, slots=2, score=0, groups=1, top_groups=1, best=1, renormalize=0, scale=1.0)
    a = dict(t=F32, d=1 * M, x=2 * M, ld=8, i=3 * M, n=4, r=ctypes.byref(rule), o=4 * M, s=None) | bad
    assert lib.pnq_expert_route_backward(*a.values()) == Status.ERR_VALUE
