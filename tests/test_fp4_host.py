"""Refusals of the 4-bit operand and expert-layer calls (no GPU needed): every bad argument is reported before the device is
touched, by the C ABI with its status and by the Python wrappers with PnqError. Sizes that the ABI reports are checked
against the layout's definition."""
import ctypes
import os

import pytest
import torch

import block_quantized_weight_pn3t_gb300 as pnq
from block_quantized_weight_pn3t_gb300 import PnqError, Status

FAKE = 0x10000  # never dereferenced: every call below fails its argument check first, or has nothing to do
F32, BF16 = 0, 1
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(pnq.lib_path()):
        from block_quantized_weight_pn3t_gb300 import build
        build.build()
    return pnq.fp4_lib()


class Plan(ctypes.Structure):
    """struct pnq_expert_plan of include/pnq.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("offsets", "block_start", "order", "position", "scale_row")] + \
        [("tokens", ctypes.c_int64), ("slots", ctypes.c_int32), ("experts", ctypes.c_int32)]


def plan(tokens=4, slots=2, experts=3, **other):
    p = Plan(FAKE, FAKE, FAKE, FAKE, FAKE, tokens, slots, experts)
    for k, v in other.items():
        setattr(p, k, v)
    return p


def test_layout(lib):
    def size(*args):
        pitch, n = ctypes.c_uint64(0), ctypes.c_uint64(0)
        return lib.pnq_fp4_layout(*args, ctypes.byref(pitch), ctypes.byref(n)), pitch.value, n.value

    assert size(pnq.NVFP4, 130, 2064, 3, 0) == (0, 1040, 3 * 2 * 33 * 512)
    assert size(pnq.MXFP4, 128, 96, 1, 0) == (0, 48, 512)
    assert size(pnq.NVFP4, 0, 16, 1, 0) == (0, 16, 0)
    # rows of a plan: any distribution fits, and the bound is met by the worst one (one row short of a block each)
    assert size(pnq.MXFP4, 129 + 1, 32, 1, 2) == (0, 16, 3 * 512)
    assert size(pnq.MXFP4, 5, 32, 1, 100) == (0, 16, 5 * 512)
    for args in ((pnq.PN3T, 4, 64, 1, 0), (pnq.NVFP4_DIV, 4, 64, 1, 0)):
        assert size(*args)[0] == Status.ERR_TYPE
    for args in ((pnq.NVFP4, 4, 24, 1, 0), (pnq.MXFP4, 4, 48, 1, 0), (pnq.NVFP4, 4, 0, 1, 0), (pnq.NVFP4, -1, 64, 1, 0),
                 (pnq.NVFP4, 4, 64, 0, 0), (pnq.NVFP4, 2 ** 31, 64, 1, 0), (pnq.NVFP4, 2 ** 20, 2 ** 30, 1, 0),
                 (pnq.NVFP4, 4, 64, 2, 3), (pnq.NVFP4, 4, 64, 1, 1025), (pnq.NVFP4, 4, 64, 1, -1),
                 (pnq.NVFP4, 2 ** 29, 64, 2 ** 29, 0)):
        assert size(*args)[0] == Status.ERR_SHAPE, args
    assert lib.pnq_fp4_layout(pnq.NVFP4, 4, 64, 1, 0, None, ctypes.byref(ctypes.c_uint64())) == Status.ERR_NULL


def test_quantize_refusals(lib):
    def call(type_=pnq.NVFP4, xt=F32, X=FAKE, ldx=64, rows=4, K=64, matrices=1, g=1.0, p=None, flags=0, codes=FAKE, scales=FAKE):
        return lib.pnq_fp4_quantize(type_, xt, X, ldx, rows, K, matrices, g, ctypes.byref(p) if p else None, flags, codes, scales,
                                    None)

    assert call(type_=pnq.PN4T) == Status.ERR_TYPE
    assert call(xt=2) == Status.ERR_TYPE
    assert call(K=72) == Status.ERR_SHAPE and call(ldx=63) == Status.ERR_SHAPE and call(rows=-1) == Status.ERR_SHAPE
    assert call(ldx=2 ** 62) == Status.ERR_SHAPE
    for g in (0.0, -1.0, INF, NAN, 1e-45):
        assert call(g=g) == Status.ERR_VALUE, g
    assert call(X=None) == Status.ERR_NULL and call(codes=None) == Status.ERR_NULL and call(scales=None) == Status.ERR_NULL
    assert call(X=FAKE + 2) == Status.ERR_ALIGN and call(xt=BF16, X=FAKE + 1) == Status.ERR_ALIGN
    assert call(codes=FAKE + 8) == Status.ERR_ALIGN and call(scales=FAKE + 4) == Status.ERR_ALIGN
    assert call(rows=0) == Status.OK
    assert call(p=plan(tokens=5)) == Status.ERR_SHAPE and call(p=plan(), matrices=2) == Status.ERR_SHAPE
    assert call(flags=2) == Status.ERR_FLAGS and call(flags=1) == Status.ERR_FLAGS  # sorted rows need a plan
    assert call(p=plan(), flags=1) == Status.ERR_SHAPE                              # 4 rows, the plan has 8
    assert call(p=plan(tokens=0), rows=0, flags=1) == Status.OK
    assert call(p=plan(slots=0)) == Status.ERR_SHAPE and call(p=plan(slots=65)) == Status.ERR_SHAPE
    assert call(p=plan(experts=0)) == Status.ERR_SHAPE and call(p=plan(experts=1025)) == Status.ERR_SHAPE
    assert call(p=plan(position=0)) == Status.ERR_NULL and call(p=plan(offsets=0)) == Status.ERR_NULL
    assert call(p=plan(order=FAKE + 2)) == Status.ERR_ALIGN


def test_dequantize_and_pack_refusals(lib):
    def deq(type_=pnq.NVFP4, codes=FAKE, scales=FAKE, rows=4, K=64, p=None, ot=F32, out=FAKE):
        return lib.pnq_fp4_dequantize(type_, codes, scales, rows, K, 1, 1.0, ctypes.byref(p) if p else None, ot, out, None)

    assert deq(type_=7) == Status.ERR_TYPE and deq(ot=5) == Status.ERR_TYPE
    assert deq(K=8) == Status.ERR_SHAPE and deq(p=plan()) == Status.ERR_SHAPE
    assert deq(codes=None) == Status.ERR_NULL and deq(out=None) == Status.ERR_NULL
    assert deq(scales=FAKE + 8) == Status.ERR_ALIGN and deq(out=FAKE + 2) == Status.ERR_ALIGN
    assert deq(rows=0) == Status.OK and deq(rows=0, p=plan(tokens=0)) == Status.OK

    def pack(codes=FAKE, scales=FAKE, rows=4, K=64, co=FAKE, so=FAKE):
        return lib.pnq_fp4_pack(pnq.NVFP4, codes, scales, rows, K, 1, co, so, None)

    assert pack(K=40) == Status.ERR_SHAPE and pack(K=48) == Status.ERR_SHAPE  # 48: not in place
    assert pack(codes=None) == Status.ERR_NULL and pack(so=None) == Status.ERR_NULL
    assert pack(so=FAKE + 1) == Status.ERR_ALIGN and pack(codes=FAKE + 1, co=FAKE + 1) == Status.ERR_ALIGN
    assert pack(rows=0) == Status.OK


def test_gemm_refusals(lib):
    def call(type_=pnq.NVFP4, xc=FAKE, xs=FAKE, M=4, wc=FAKE, ws=FAKE, N=8, K=64, yt=F32, Y=FAKE, flags=0):
        return lib.pnq_fp4_gemm(type_, xc, xs, M, wc, ws, N, K, 1.0, yt, Y, flags, None)

    assert call(type_=pnq.NVFP4_DIV) == Status.ERR_TYPE and call(yt=3) == Status.ERR_TYPE
    assert call(K=0) == Status.ERR_SHAPE and call(M=-1) == Status.ERR_SHAPE and call(N=-1) == Status.ERR_SHAPE
    assert call(type_=pnq.MXFP4, K=48) == Status.ERR_SHAPE and call(M=2 ** 29, N=2 ** 29) == Status.ERR_SHAPE
    assert call(flags=2) == Status.ERR_FLAGS
    for name in ("xc", "xs", "wc", "ws", "Y"):
        assert call(**{name: None}) == Status.ERR_NULL, name
    for name in ("xc", "xs", "wc", "ws"):
        assert call(**{name: FAKE + 8}) == Status.ERR_ALIGN, name
    assert call(Y=FAKE + 2) == Status.ERR_ALIGN and call(yt=BF16, Y=FAKE + 1) == Status.ERR_ALIGN
    assert call(M=0, xc=None) == Status.OK and call(N=0, wc=None) == Status.OK

    def experts(p=None, type_=pnq.NVFP4, xc=FAKE, N=8, K=64, wg=None, yt=F32, Y=FAKE, flags=0):
        p = p or plan()
        return lib.pnq_fp4_gemm_experts(type_, xc, FAKE, ctypes.byref(p), FAKE, FAKE, N, K, 1.0, wg, yt, Y, flags, None)

    assert lib.pnq_fp4_gemm_experts(pnq.NVFP4, FAKE, FAKE, None, FAKE, FAKE, 8, 64, 1.0, None, 0, FAKE, 0, None) == Status.ERR_NULL
    assert experts(type_=1) == Status.ERR_TYPE and experts(yt=9) == Status.ERR_TYPE
    assert experts(plan(experts=0)) == Status.ERR_SHAPE and experts(K=8) == Status.ERR_SHAPE and experts(N=-2) == Status.ERR_SHAPE
    assert experts(plan(tokens=2 ** 30)) == Status.ERR_SHAPE
    assert experts(xc=None) == Status.ERR_NULL and experts(Y=None) == Status.ERR_NULL
    assert experts(wg=FAKE + 2) == Status.ERR_ALIGN and experts(flags=8) == Status.ERR_FLAGS
    assert experts(plan(tokens=0)) == Status.OK and experts(N=0) == Status.OK


def test_expert_refusals(lib):
    ref = lambda p: ctypes.byref(p)  # noqa: E731
    assert lib.pnq_expert_sort(FAKE, None, None) == Status.ERR_NULL
    assert lib.pnq_expert_sort(None, ref(plan()), None) == Status.ERR_NULL
    assert lib.pnq_expert_sort(FAKE + 1, ref(plan()), None) == Status.ERR_ALIGN
    assert lib.pnq_expert_sort(FAKE, ref(plan(experts=2000)), None) == Status.ERR_SHAPE
    assert lib.pnq_expert_sort(FAKE, ref(plan(tokens=-1)), None) == Status.ERR_SHAPE
    two = {"gather": lambda t, D, p, a, b: lib.pnq_expert_gather(t, a, D, p, b, None),
           "gather_backward": lambda t, D, p, a, b: lib.pnq_expert_gather_backward(t, a, D, p, b, None),
           "combine": lambda t, D, p, a, b: lib.pnq_expert_combine(t, a, D, p, FAKE, b, None),
           "combine_backward": lambda t, D, p, a, b: lib.pnq_expert_combine_backward(t, a, FAKE, D, p, FAKE, b, None, None)}
    for name, call in two.items():
        assert call(2, 8, ref(plan()), FAKE, FAKE) == Status.ERR_TYPE, name
        assert call(F32, 0, ref(plan()), FAKE, FAKE) == Status.ERR_SHAPE, name
        assert call(F32, 8, None, FAKE, FAKE) == Status.ERR_NULL, name
        assert call(F32, 8, ref(plan()), None, FAKE) == Status.ERR_NULL, name
        assert call(F32, 8, ref(plan()), FAKE, None) == Status.ERR_NULL, name
        assert call(F32, 8, ref(plan()), FAKE + 2, FAKE) == Status.ERR_ALIGN, name
        assert call(BF16, 8, ref(plan()), FAKE, FAKE + 1) == Status.ERR_ALIGN, name
        assert call(F32, 8, ref(plan(tokens=0)), None, None) == Status.OK, name
    assert lib.pnq_expert_combine(F32, FAKE, 8, ref(plan()), None, FAKE, None) == Status.ERR_NULL
    assert lib.pnq_expert_combine(BF16, FAKE, 8, ref(plan()), FAKE + 2, FAKE, None) == Status.ERR_ALIGN
    assert lib.pnq_expert_combine_backward(F32, FAKE, FAKE, 8, ref(plan()), FAKE, FAKE, FAKE + 1, None) == Status.ERR_ALIGN


def test_wrapper_refusals(lib):
    """The torch wrappers refuse what the ABI cannot see: devices, dtypes, strides and shapes."""
    x = torch.zeros(4, 64)
    with pytest.raises(PnqError, match="CUDA"):
        pnq.fp4_quantize(pnq.NVFP4, x)
    with pytest.raises(PnqError, match="dtype"):
        pnq.fp4_quantize(pnq.NVFP4, x.to(torch.float16))
    with pytest.raises(PnqError, match="microscaled"):
        pnq.fp4_quantize(pnq.PN3T, x)
    with pytest.raises(PnqError, match="torch.Tensor"):
        pnq.fp4_quantize(pnq.NVFP4, x[0])
    with pytest.raises(PnqError, match="CUDA"):
        pnq.Fp4Matrix(pnq.NVFP4, 4, 64, torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8))
    with pytest.raises(PnqError, match="elements"):
        pnq.Fp4Matrix(pnq.NVFP4, 4, 64, torch.zeros(3, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8))
    with pytest.raises(PnqError, match="ERR_SHAPE"):
        pnq.fp4_layout(pnq.MXFP4, 4, 48)
    with pytest.raises(PnqError, match="ids"):
        pnq.expert_sort(torch.zeros(4, dtype=torch.int32), 3)
    with pytest.raises(PnqError, match="dtype"):
        pnq.expert_sort(torch.zeros(4, 2), 3)
    with pytest.raises(PnqError, match="CUDA"):
        pnq.ExpertPlan(4, 2, 3, torch.zeros(100, dtype=torch.int32))
    with pytest.raises(PnqError, match="Fp4Matrix"):
        pnq.fp4_gemm(x, x)
    with pytest.raises(PnqError, match="codes"):
        pnq.fp4_pack(pnq.NVFP4, torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8), 4, 64)
