"""Refusals of pnq_fp4_gemm_shape (no GPU needed: bad arguments are reported before the device is asked)."""
import ctypes
import os

import pytest

import block_quantized_weight_pn3t_gb300 as pnq
from block_quantized_weight_pn3t_gb300 import Status


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(pnq.lib_path()):
        from block_quantized_weight_pn3t_gb300 import build
        build.build()
    return pnq.fp4_lib()


def test_refusals(lib):
    out = [ctypes.c_int32() for _ in range(3)]

    def call(type_=pnq.NVFP4, M=4, N=8, K=64, refs=tuple(ctypes.byref(v) for v in out)):
        return lib.pnq_fp4_gemm_shape(type_, M, N, K, *refs)

    assert call(type_=pnq.PN3T) == Status.ERR_TYPE
    for bad in (dict(M=0), dict(N=0), dict(M=-1), dict(N=-1), dict(K=0), dict(K=72), dict(type_=pnq.MXFP4, K=48),
                dict(M=2 ** 29, N=2 ** 29)):
        assert call(**bad) == Status.ERR_SHAPE, bad
    for i in range(3):
        refs = [ctypes.byref(v) for v in out]
        refs[i] = None
        assert call(refs=refs) == Status.ERR_NULL
