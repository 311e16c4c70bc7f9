"""4-bit microscaled operands (NVFP4, MXFP4) and the expert layer around their product: argument marshalling for
the pnq_fp4_* and pnq_expert_* entry points (formats, layouts and rounding steps are stated in ``include/pnq.h``).

    q = fp4_quantize(NVFP4, x, g)                    # activations -> operand
    w = fp4_pack(NVFP4, codes, scales, N, K, g_w)    # row-major weights -> operand, once
    y = fp4_gemm(q, w)                               # Y = X W^T

    plan = expert_sort(ids, experts)                 # ids [tokens][slots]
    q = fp4_quantize(NVFP4, x, g, plan=plan)         # tokens encoded once, written in expert order
    ys = fp4_gemm_experts(q, w, plan)                # every row times its expert's matrix
    y = expert_combine(ys, plan, weights)            # back to tokens, router weights applied
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _binding as b
from ._binding import NVFP4, PnqError

MXFP4 = 1006
FP4_GROUP = {NVFP4: 16, MXFP4: 32}
_FLOAT = {torch.float32: 0, torch.bfloat16: 1}


# struct pnq_expert_plan of include/pnq.h: five device addresses, tokens, slots, experts
_PLAN = struct.Struct("@5Pqii")


_P, _I64, _I, _F, _U = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_uint
_SIGNATURES = {
    "pnq_fp4_layout": [_I, _I64, _I64, _I64, _I64, ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_uint64)],
    "pnq_fp4_quantize": [_I, _I, _P, _I64, _I64, _I64, _I64, _F, _P, _P, _P, _P],
    "pnq_fp4_dequantize": [_I, _P, _P, _I64, _I64, _I64, _F, _P, _I, _P, _P],
    "pnq_fp4_pack": [_I, _P, _P, _I64, _I64, _I64, _P, _P, _P],
    "pnq_fp4_gemm": [_I, _P, _P, _I64, _P, _P, _I64, _I64, _F, _I, _P, _U, _P],
    "pnq_fp4_gemm_experts": [_I, _P, _P, _P, _P, _P, _I64, _I64, _F, _P, _I, _P, _U, _P],
    "pnq_expert_sort": [_P, _P, _P],
    "pnq_expert_gather": [_I, _P, _I64, _P, _P, _P],
    "pnq_expert_gather_backward": [_I, _P, _I64, _P, _P, _P],
    "pnq_expert_combine": [_I, _P, _I64, _P, _P, _P, _P],
    "pnq_expert_combine_backward": [_I, _P, _P, _I64, _P, _P, _P, _P, _P],
}


_lib = None


def fp4_lib() -> ctypes.CDLL:
    """The library with the signatures of these entry points set."""
    global _lib
    if _lib is None:
        L = b.lib()
        for name, args in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = _I
            fn.argtypes = args
        _lib = L
    return _lib


# The wrappers run once per call of a decode step, so they look at each tensor once and keep addresses, sizes and
# devices as plain integers; a check that fails is looked at again, slowly, for its message.

_raw_stream = torch._C._cuda_getCurrentRawStream  # handle of the current stream of a device


def _group(type_: int) -> int:
    try:
        return FP4_GROUP[type_]
    except (KeyError, TypeError):
        raise PnqError(f"type {type_!r} is not a 4-bit microscaled format", int(b.Status.ERR_TYPE)) from None


def _float_type(dtype, what: str) -> int:
    try:
        return _FLOAT[dtype]
    except KeyError:
        raise PnqError(f"{what} has dtype {dtype}; expected float32 or bfloat16") from None


def _refuse(t, what: str, dtype, shape=None, numel: int | None = None, device: int | None = None):
    """Raise the PnqError that says what is wrong with t."""
    b._require(t, what, (dtype,), numel)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise PnqError(f"{what} has shape {tuple(t.shape)}; expected {tuple(shape)}")
    raise PnqError(f"{what} is on {t.device}; the other tensors are on cuda:{device}")


def _matrix(t, what: str, dtype, rows: int, cols: int, device: int) -> int:
    """Address of a contiguous [rows][cols] tensor of `dtype` on CUDA device `device`, or a refusal."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == (rows, cols) and t.get_device() == device
            and t.is_contiguous()):
        _refuse(t, what, dtype, (rows, cols), None, device)
    return t.data_ptr()


def _bytes(t, what: str, numel: int) -> None:
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.uint8 and t.is_cuda and t.numel() >= numel and t.is_contiguous()):
        _refuse(t, what, torch.uint8, None, numel)


_layouts: dict = {}


def fp4_layout(type_: int, rows: int, K: int, matrices: int = 1, plan_experts: int = 0):
    """(pitch of a row of codes, bytes of the tiled scales) of an operand."""
    key = (type_, rows, K, matrices, plan_experts)
    hit = _layouts.get(key)
    if hit is None:
        _group(type_)
        pitch, size = ctypes.c_uint64(0), ctypes.c_uint64(0)
        rc = fp4_lib().pnq_fp4_layout(type_, rows, K, matrices, plan_experts, ctypes.byref(pitch), ctypes.byref(size))
        if rc:
            raise PnqError("pnq_fp4_layout", rc)
        if len(_layouts) > 4096:
            _layouts.clear()
        hit = _layouts[key] = (pitch.value, size.value)
    return hit


class Fp4Matrix:
    """A 4-bit microscaled operand: `matrices` matrices of `rows` x `K`. codes: uint8 [matrices * rows][pitch];
    scales: uint8, the tiled scale words; global_scale: a float, or for expert weights a CUDA fp32 tensor
    [matrices]. plan: the ExpertPlan whose sorted rows it holds (None otherwise)."""
    __slots__ = ("type", "rows", "K", "global_scale", "matrices", "plan", "device", "device_index", "codes_ptr", "scales_ptr", "_codes",
                 "_scales", "_buffer")

    def __init__(self, type_: int, rows: int, K: int, codes, scales, global_scale=1.0, matrices: int = 1, plan=None):
        pitch, size = fp4_layout(type_, rows, K, matrices, 0 if plan is None else plan.experts)
        _bytes(codes, "codes", matrices * rows * pitch)
        _bytes(scales, "scales", size)
        dev = codes.get_device()
        if scales.get_device() != dev:
            _refuse(scales, "scales", torch.uint8, None, size, dev)
        if isinstance(global_scale, torch.Tensor):
            if not (global_scale.dtype is torch.float32 and global_scale.shape == (matrices,) and
                    global_scale.get_device() == dev and global_scale.is_contiguous()):
                _refuse(global_scale, "global_scale", torch.float32, (matrices,), None, dev)
        else:
            global_scale = float(global_scale)
        self.type, self.rows, self.K, self.matrices = type_, rows, K, matrices
        self.global_scale, self.plan, self.device, self.device_index = global_scale, plan, codes.device, dev
        self._codes, self._scales, self._buffer = codes, scales, None
        self.codes_ptr, self.scales_ptr = codes.data_ptr(), scales.data_ptr()

    @classmethod
    def _empty(cls, type_: int, rows: int, K: int, matrices: int, plan, device):
        """Room for an operand, codes and scales in one allocation."""
        pitch, size = fp4_layout(type_, rows, K, matrices, 0 if plan is None else plan.experts)
        self = cls.__new__(cls)
        self.type, self.rows, self.K, self.matrices, self.plan = type_, rows, K, matrices, plan
        self._buffer = buffer = torch.empty(matrices * rows * pitch + size, dtype=torch.uint8, device=device)
        self._codes = self._scales = None
        self.device, self.device_index = device, buffer.get_device()
        self.codes_ptr = buffer.data_ptr()
        self.scales_ptr = self.codes_ptr + matrices * rows * pitch  # rows of whole 16 bytes: still aligned
        return self

    def _layout(self):
        return fp4_layout(self.type, self.rows, self.K, self.matrices, 0 if self.plan is None else self.plan.experts)

    @property
    def codes(self):
        if self._codes is None:
            n, pitch = self.matrices * self.rows, self._layout()[0]
            self._codes = self._buffer[:n * pitch].view(n, pitch)
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            pitch, size = self._layout()
            at = self.matrices * self.rows * pitch
            self._scales = self._buffer[at:at + size]
        return self._scales


class ExpertPlan:
    """How the (token, slot) choices of an expert layer are sorted by expert: one int32 CUDA buffer that holds, one
    after the other, offsets [experts + 1], block_start [experts + 1], order [n], position [n] and scale_row [n]
    (n = tokens * slots; meanings in ``include/pnq.h``, pnq_expert_plan)."""
    __slots__ = ("tokens", "slots", "experts", "rows", "buffer", "device_index", "ref")

    def __init__(self, tokens: int, slots: int, experts: int, buffer=None, device=None):
        n = tokens * slots
        size = 2 * (experts + 1) + 3 * n
        if buffer is None:
            buffer = torch.empty(size, dtype=torch.int32, device=device)
        elif not (isinstance(buffer, torch.Tensor) and buffer.dtype is torch.int32 and buffer.is_cuda and buffer.numel() >= size
                and buffer.is_contiguous()):
            _refuse(buffer, "plan buffer", torch.int32, None, size)
        self.tokens, self.slots, self.experts, self.rows, self.buffer = tokens, slots, experts, n, buffer
        self.device_index = buffer.get_device()
        at = buffer.data_ptr()
        order = at + 8 * (experts + 1)
        self.ref = _PLAN.pack(at, at + 4 * (experts + 1), order, order + 4 * n, order + 8 * n, tokens, slots, experts)

    def _part(self, first: int, count: int):
        return self.buffer.narrow(0, first, count)

    @property
    def offsets(self):
        return self._part(0, self.experts + 1)

    @property
    def block_start(self):
        return self._part(self.experts + 1, self.experts + 1)

    @property
    def order(self):
        return self._part(2 * (self.experts + 1), self.rows)

    @property
    def position(self):
        return self._part(2 * (self.experts + 1) + self.rows, self.rows)

    @property
    def scale_row(self):
        return self._part(2 * (self.experts + 1) + 2 * self.rows, self.rows)


# ---- operands ------------------------------------------------------------------------------------

def fp4_quantize(type_: int, x, global_scale: float = 1.0, plan: ExpertPlan | None = None, out: Fp4Matrix | None = None,
                 stream=None) -> Fp4Matrix:
    """Encode x (CUDA bf16 or fp32, [rows][K], or [matrices][rows][K] contiguous; 2-D rows may be strided) for the
    global multiplier. With a plan, x holds the plan's tokens and the operand its sorted rows. out: an operand of
    the same shape to write into."""
    G = _group(type_)
    if not isinstance(x, torch.Tensor) or x.dim() not in (2, 3):
        raise PnqError("x must be a torch.Tensor [rows][K] or [matrices][rows][K]")
    xt = _float_type(x.dtype, "x")
    if not x.is_cuda:
        raise PnqError(f"x must be a CUDA tensor (device {x.device})")
    shape = x.shape
    if len(shape) == 2:
        matrices, (rows, K) = 1, shape
        ldx, step = x.stride()
        if rows <= 1:
            ldx = K
    else:
        matrices, rows, K = shape
        if not x.is_contiguous():
            raise PnqError("x [matrices][rows][K] must be contiguous")
        ldx, step = K, 1
    if step != 1 and K > 1 and rows * matrices:
        raise PnqError("the elements of a row of x must be consecutive")
    if ldx < K:
        raise PnqError(f"rows of x are {ldx} elements apart; at least K = {K} is wanted")
    if K == 0 or K % G:
        raise PnqError(f"K = {K} is not a positive multiple of {G}", int(b.Status.ERR_SHAPE))
    dev = x.get_device()
    out_rows = rows
    if plan is not None:
        if matrices != 1 or rows != plan.tokens:
            raise PnqError(f"x has shape {tuple(shape)}; the plan has {plan.tokens} tokens")
        if plan.device_index != dev:
            raise PnqError(f"x is on cuda:{dev}, the plan on cuda:{plan.device_index}")
        out_rows = plan.rows
    g = float(global_scale)
    if out is None:
        out = Fp4Matrix._empty(type_, out_rows, K, matrices, plan, x.device)
    elif (out.type, out.rows, out.K, out.matrices, out.plan.experts if out.plan is not None else 0) != \
            (type_, out_rows, K, matrices, plan.experts if plan is not None else 0) or out.device_index != dev:
        raise PnqError("out is an operand of another type, shape or device")
    out.global_scale, out.plan = g, plan
    rc = (_lib or fp4_lib()).pnq_fp4_quantize(type_, xt, x.data_ptr(), ldx, rows, K, matrices, g,
                                              None if plan is None else plan.ref, out.codes_ptr, out.scales_ptr,
                                              _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        raise PnqError("pnq_fp4_quantize", rc)
    return out


def fp4_dequantize(m: Fp4Matrix, dtype=torch.float32, out=None, stream=None):
    """The values an operand stands for, fp32 or bf16 [matrices * rows][K] (of a plan's operand: its sorted rows,
    zeros past the rows in use). The operand's global_scale must be one float."""
    if isinstance(m.global_scale, torch.Tensor):
        raise PnqError("an operand with a global scale per matrix is read back matrix by matrix")
    dev, n = m.device_index, m.matrices * m.rows
    if out is None:
        ot = _float_type(dtype, "out")
        out = torch.empty((n, m.K), dtype=dtype, device=m.device)
        at = out.data_ptr()
    else:
        ot = _float_type(out.dtype, "out")
        at = _matrix(out, "out", out.dtype, n, m.K, dev)
    rc = (_lib or fp4_lib()).pnq_fp4_dequantize(m.type, m.codes_ptr, m.scales_ptr, m.rows, m.K, m.matrices, m.global_scale,
                                                None if m.plan is None else m.plan.ref, ot, at,
                                                _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        raise PnqError("pnq_fp4_dequantize", rc)
    return out


def fp4_pack(type_: int, codes, scales, rows: int, K: int, global_scale=1.0, matrices: int = 1, stream=None) -> Fp4Matrix:
    """Row-major weights (codes uint8 [matrices * rows][K / 2], scale words uint8 [matrices * rows][K / group]) as an
    operand, once, when they are loaded. Where K is a multiple of 32 and the codes are 16-byte aligned they are kept
    as they are, not copied."""
    G = _group(type_)
    pitch, size = fp4_layout(type_, rows, K, matrices)
    n = matrices * rows
    _bytes(codes, "codes", n * K // 2)
    _bytes(scales, "scales", n * K // G)
    dev = codes.get_device()
    if scales.get_device() != dev:
        _refuse(scales, "scales", torch.uint8, None, 0, dev)
    keep = K % 32 == 0 and codes.data_ptr() % 16 == 0
    out_codes = codes if keep else torch.empty((n, pitch), dtype=torch.uint8, device=codes.device)
    tiled = torch.empty(size, dtype=torch.uint8, device=codes.device)
    rc = fp4_lib().pnq_fp4_pack(type_, codes.data_ptr(), scales.data_ptr(), rows, K, matrices, out_codes.data_ptr(),
                                tiled.data_ptr(), _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        raise PnqError("pnq_fp4_pack", rc)
    return Fp4Matrix(type_, rows, K, out_codes, tiled, global_scale, matrices)


def _operands(x: Fp4Matrix, w: Fp4Matrix) -> int:
    """The CUDA device of two operands that can be multiplied."""
    if not isinstance(x, Fp4Matrix) or not isinstance(w, Fp4Matrix):
        raise PnqError("both operands must be Fp4Matrix")
    if x.type != w.type or x.K != w.K:
        raise PnqError(f"operands differ: type {x.type}, K = {x.K} and type {w.type}, K = {w.K}")
    if x.matrices != 1 or isinstance(x.global_scale, torch.Tensor):
        raise PnqError("the activations are one matrix with one global scale")
    if x.device_index != w.device_index:
        raise PnqError(f"operands are on cuda:{x.device_index} and cuda:{w.device_index}")
    return x.device_index


def _result(out, rows: int, N: int, dtype, x: Fp4Matrix):
    """(result, element type, address)."""
    if out is None:
        ft = _float_type(dtype, "the result")
        out = torch.empty((rows, N), dtype=dtype, device=x.device)
        return out, ft, out.data_ptr()
    if not isinstance(out, torch.Tensor):
        raise PnqError("out must be a torch.Tensor")
    return out, _float_type(out.dtype, "out"), _matrix(out, "out", out.dtype, rows, N, x.device_index)


def fp4_gemm(x: Fp4Matrix, w: Fp4Matrix, dtype=torch.float32, out=None, flags: int = 0, stream=None):
    """Y[m][n] = sum_k X[m][k] W[n][k] of two operands of one type; fp32 or bf16 [M][N]."""
    dev = _operands(x, w)
    if w.matrices != 1 or isinstance(w.global_scale, torch.Tensor) or x.plan is not None or w.plan is not None:
        raise PnqError("fp4_gemm takes one matrix each; expert layers go through fp4_gemm_experts")
    out, ft, at = _result(out, x.rows, w.rows, dtype, x)
    rc = (_lib or fp4_lib()).pnq_fp4_gemm(x.type, x.codes_ptr, x.scales_ptr, x.rows, w.codes_ptr, w.scales_ptr, w.rows, x.K,
                                          x.global_scale * w.global_scale, ft, at, flags,
                                          _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        raise PnqError("pnq_fp4_gemm", rc)
    return out


def fp4_gemm_experts(x: Fp4Matrix, w: Fp4Matrix, plan: ExpertPlan, dtype=torch.float32, out=None, flags: int = 0,
                     stream=None):
    """Every sorted row of x (made with `plan`) times its expert's matrix of w (matrices = the plan's experts): fp32 or
    bf16 [tokens * slots][N], zeros past the rows in use."""
    dev = _operands(x, w)
    if x.plan is not plan and (x.plan is None or not isinstance(plan, ExpertPlan) or
                               (x.plan.tokens, x.plan.slots, x.plan.experts) != (plan.tokens, plan.slots, plan.experts)):
        raise PnqError("x is not an operand of this plan's sorted rows")
    if plan is None or w.matrices != plan.experts or w.plan is not None:
        raise PnqError(f"w has {w.matrices} matrices; one for each of the plan's experts is wanted")
    if plan.device_index != dev:
        raise PnqError(f"the operands are on cuda:{dev}, the plan on cuda:{plan.device_index}")
    out, ft, at = _result(out, plan.rows, w.rows, dtype, x)
    per = isinstance(w.global_scale, torch.Tensor)
    rc = (_lib or fp4_lib()).pnq_fp4_gemm_experts(
        x.type, x.codes_ptr, x.scales_ptr, plan.ref, w.codes_ptr, w.scales_ptr, w.rows, x.K,
        x.global_scale if per else x.global_scale * w.global_scale, w.global_scale.data_ptr() if per else None, ft, at, flags,
        _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        raise PnqError("pnq_fp4_gemm_experts", rc)
    return out


# ---- tokens to their experts and back ----------------------------------------------------------------

def expert_sort(ids, experts: int, plan: ExpertPlan | None = None, stream=None) -> ExpertPlan:
    """The plan of ids (CUDA int32 [tokens][slots]: the expert of each choice; one outside 0 .. experts - 1 is dropped):
    stable, so equal experts keep the order of their slots."""
    if not (isinstance(ids, torch.Tensor) and ids.dim() == 2):
        raise PnqError("ids must be a torch.Tensor [tokens][slots]")
    tokens, slots = ids.shape
    if not (ids.dtype is torch.int32 and ids.is_cuda and ids.is_contiguous()):
        _refuse(ids, "ids", torch.int32)
    if not 1 <= slots <= 64 or not 1 <= experts <= 1024:
        raise PnqError(f"{slots} slots and {experts} experts; 1..64 and 1..1024 are wanted", int(b.Status.ERR_SHAPE))
    dev = ids.get_device()
    if plan is None:
        plan = ExpertPlan(tokens, slots, experts, device=ids.device)
    elif (plan.tokens, plan.slots, plan.experts) != (tokens, slots, experts) or plan.device_index != dev:
        raise PnqError("the plan is of another shape or device")
    rc = (_lib or fp4_lib()).pnq_expert_sort(ids.data_ptr(), plan.ref,
                                             _raw_stream(dev) if stream is None else stream.cuda_stream)
    if rc:
        raise PnqError("pnq_expert_sort", rc)
    return plan


def _rows(t, what: str, rows: int, plan: ExpertPlan):
    """(element type, D, address) of a contiguous CUDA [rows][D] tensor on the plan's device."""
    if not (isinstance(t, torch.Tensor) and t.dim() == 2):
        raise PnqError(f"{what} must be a torch.Tensor [rows][D]")
    D = t.shape[1]
    return _float_type(t.dtype, what), D, _matrix(t, what, t.dtype, rows, D, plan.device_index)


def _rows_out(out, like, rows: int, D: int, plan: ExpertPlan):
    """(out or a new one like `like`, address)."""
    if out is None:
        out = like.new_empty((rows, D))
        return out, out.data_ptr()
    return out, _matrix(out, "out", like.dtype, rows, D, plan.device_index)


def expert_gather(x, plan: ExpertPlan, out=None, stream=None):
    """Sorted rows of x (fp32 or bf16 [tokens][D]): [tokens * slots][D], zeros past the rows in use."""
    ft, D, src = _rows(x, "x", plan.tokens, plan)
    out, dst = _rows_out(out, x, plan.rows, D, plan)
    rc = (_lib or fp4_lib()).pnq_expert_gather(ft, src, D, plan.ref, dst,
                                               _raw_stream(plan.device_index) if stream is None else stream.cuda_stream)
    if rc:
        raise PnqError("pnq_expert_gather", rc)
    return out


def expert_gather_backward(dxs, plan: ExpertPlan, out=None, stream=None):
    """Gradient of expert_gather: dx [tokens][D], each token's rows summed in fp32 in slot order."""
    ft, D, src = _rows(dxs, "dxs", plan.rows, plan)
    out, dst = _rows_out(out, dxs, plan.tokens, D, plan)
    rc = (_lib or fp4_lib()).pnq_expert_gather_backward(ft, src, D, plan.ref, dst,
                                                        _raw_stream(plan.device_index) if stream is None else stream.cuda_stream)
    if rc:
        raise PnqError("pnq_expert_gather_backward", rc)
    return out


def expert_combine(ys, plan: ExpertPlan, weights, out=None, stream=None):
    """y[t] = sum over t's slots of weights[t][j] * its row of ys ([tokens * slots][D]; weights fp32 [tokens][slots])."""
    ft, D, src = _rows(ys, "ys", plan.rows, plan)
    w = _matrix(weights, "weights", torch.float32, plan.tokens, plan.slots, plan.device_index)
    out, dst = _rows_out(out, ys, plan.tokens, D, plan)
    rc = (_lib or fp4_lib()).pnq_expert_combine(ft, src, D, plan.ref, w, dst,
                                                _raw_stream(plan.device_index) if stream is None else stream.cuda_stream)
    if rc:
        raise PnqError("pnq_expert_combine", rc)
    return out


def expert_combine_backward(dy, ys, plan: ExpertPlan, weights, out=None, dweights=None, stream=None):
    """Gradients of expert_combine: (dys [tokens * slots][D], dweights fp32 [tokens][slots])."""
    ft, D, src = _rows(ys, "ys", plan.rows, plan)
    grad = _matrix(dy, "dy", ys.dtype, plan.tokens, D, plan.device_index)
    w = _matrix(weights, "weights", torch.float32, plan.tokens, plan.slots, plan.device_index)
    out, dst = _rows_out(out, ys, plan.rows, D, plan)
    if dweights is None:
        dweights = torch.empty((plan.tokens, plan.slots), dtype=torch.float32, device=ys.device)
        dw = dweights.data_ptr()
    else:
        dw = _matrix(dweights, "dweights", torch.float32, plan.tokens, plan.slots, plan.device_index)
    rc = (_lib or fp4_lib()).pnq_expert_combine_backward(
        ft, grad, src, D, plan.ref, w, dst, dw, _raw_stream(plan.device_index) if stream is None else stream.cuda_stream)
    if rc:
        raise PnqError("pnq_expert_combine_backward", rc)
    return out, dweights
