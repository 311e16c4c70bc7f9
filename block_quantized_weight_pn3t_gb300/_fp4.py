"""4-bit microscaled operands (NVFP4, MXFP4) and the expert layer around their product: the torch wrappers of
the pnq_fp4_* and pnq_expert_* entry points (formats, layouts and rounding steps are stated in ``include/pnq.h``). They are
compiled (csrc/pnq_torch.cpp): they check tensors, allocate results and make one call of the library.

    q = fp4_quantize(NVFP4, x, g)                    # activations -> operand
    w = fp4_pack(NVFP4, codes, scales, N, K, g_w)    # row-major weights -> operand, once
    y = fp4_gemm(q, w)                               # Y = X W^T

    plan = expert_sort(ids, experts)                 # ids [tokens][slots]
    q = fp4_quantize(NVFP4, x, g, plan=plan)         # tokens encoded once, written in expert order
    ys = fp4_gemm_experts(q, w, plan)                # every row times its expert's matrix
    h = fp4_quantize(NVFP4, hs, g, plan=plan, sorted=True)   # rows in expert order already (between two products)
    y = expert_combine(ys, plan, weights)            # back to tokens, router weights applied

They stand outside autograd: results require no gradient. The gather and the combine have theirs as calls,
    dys, dweights = expert_combine_backward(dy, ys, plan, weights)
    dx = expert_gather_backward(dxs, plan)
"""
from __future__ import annotations

import ctypes
import os

import torch  # noqa: F401  (the libraries that _native.so is linked to)

from . import _binding as b

_NATIVE = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_native.so")
if not os.path.exists(_NATIVE):
    raise b.PnqError(f"{_NATIVE} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")

from ._native import (Fp4Matrix, ExpertPlan, fp4_layout, fp4_quantize, fp4_dequantize, fp4_pack, fp4_gemm,  # noqa: E402,F401
                      fp4_gemm_experts, expert_sort, expert_gather, expert_gather_backward, expert_combine,
                      expert_combine_backward)

MXFP4 = 1006
FP4_GROUP = {b.NVFP4: 16, MXFP4: 32}

_P, _I64, _I, _F, _U = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_uint
_SIGNATURES = {
    "pnq_fp4_layout": [_I, _I64, _I64, _I64, _I64, ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_uint64)],
    "pnq_fp4_quantize": [_I, _I, _P, _I64, _I64, _I64, _I64, _F, _P, _U, _P, _P, _P],
    "pnq_fp4_dequantize": [_I, _P, _P, _I64, _I64, _I64, _F, _P, _I, _P, _P],
    "pnq_fp4_pack": [_I, _P, _P, _I64, _I64, _I64, _P, _P, _P],
    "pnq_fp4_gemm": [_I, _P, _P, _I64, _P, _P, _I64, _I64, _F, _I, _P, _U, _P],
    "pnq_fp4_gemm_shape": [_I, _I64, _I64, _I64, *[ctypes.POINTER(ctypes.c_int32)] * 3],
    "pnq_fp4_gemm_experts": [_I, _P, _P, _P, _P, _P, _I64, _I64, _F, _P, _I, _P, _U, _P],
    "pnq_expert_sort": [_P, _P, _P],
    "pnq_expert_gather": [_I, _P, _I64, _P, _P, _P],
    "pnq_expert_gather_backward": [_I, _P, _I64, _P, _P, _P],
    "pnq_expert_combine": [_I, _P, _I64, _P, _P, _P, _P],
    "pnq_expert_combine_backward": [_I, _P, _P, _I64, _P, _P, _P, _P, _P],
}
_lib = None


def fp4_lib() -> ctypes.CDLL:
    """The library with the signatures of these entry points set (raw addresses; the wrappers above are faster)."""
    global _lib
    if _lib is None:
        L = b.lib()
        for name, args in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = _I
            fn.argtypes = args
        _lib = L
    return _lib
