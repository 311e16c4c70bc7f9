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

import torch

from . import _binding as b
from ._binding import NVFP4, PnqError

MXFP4 = 1006
FP4_GROUP = {NVFP4: 16, MXFP4: 32}
_FLOAT = {torch.float32: 0, torch.bfloat16: 1}


class pnq_expert_plan(ctypes.Structure):
    _fields_ = [("offsets", ctypes.c_void_p), ("block_start", ctypes.c_void_p), ("order", ctypes.c_void_p),
                ("position", ctypes.c_void_p), ("scale_row", ctypes.c_void_p), ("tokens", ctypes.c_int64),
                ("slots", ctypes.c_int32), ("experts", ctypes.c_int32)]


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


def _stream(stream, device: int) -> int:
    """The handle of `stream`, or of the current stream of CUDA device `device` (the calls' tensors')."""
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device)


def _call(name: str, *args) -> None:
    rc = getattr(fp4_lib(), name)(*args)
    if rc:
        raise PnqError(name, rc)


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


def _require(t, what: str, dtypes, shape=None, numel: int | None = None) -> None:
    b._require(t, what, dtypes, numel)
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise PnqError(f"{what} has shape {tuple(t.shape)}; expected {tuple(shape)}")


def _same_device(first, *others) -> int:
    """The CUDA device index that all the tensors are on."""
    for t in others:
        if t is not None and t.device != first.device:
            raise PnqError(f"tensors are on {first.device} and {t.device}; one device is wanted")
    return first.get_device()


_layouts: dict = {}


def fp4_layout(type_: int, rows: int, K: int, matrices: int = 1, plan_experts: int = 0):
    """(pitch of a row of codes, bytes of the tiled scales) of an operand."""
    key = (type_, rows, K, matrices, plan_experts)
    hit = _layouts.get(key)
    if hit is None:
        _group(type_)
        pitch, size = ctypes.c_uint64(0), ctypes.c_uint64(0)
        _call("pnq_fp4_layout", type_, rows, K, matrices, plan_experts, ctypes.byref(pitch), ctypes.byref(size))
        if len(_layouts) > 4096:
            _layouts.clear()
        hit = _layouts[key] = (pitch.value, size.value)
    return hit


class Fp4Matrix:
    """A 4-bit microscaled operand: `matrices` matrices of `rows` x `K`. codes: uint8 [matrices * rows][pitch];
    scales: uint8, the tiled scale words; global_scale: a float, or for expert weights a CUDA fp32 tensor
    [matrices]. plan: the ExpertPlan whose sorted rows it holds (None otherwise)."""
    __slots__ = ("type", "rows", "K", "codes", "scales", "global_scale", "matrices", "plan")

    def __init__(self, type_: int, rows: int, K: int, codes, scales, global_scale=1.0, matrices: int = 1, plan=None):
        pitch, size = fp4_layout(type_, rows, K, matrices, 0 if plan is None else plan.experts)
        _require(codes, "codes", (torch.uint8,), numel=matrices * rows * pitch)
        _require(scales, "scales", (torch.uint8,), numel=size)
        _same_device(codes, scales)
        if isinstance(global_scale, torch.Tensor):
            _require(global_scale, "global_scale", (torch.float32,), shape=(matrices,))
            _same_device(codes, global_scale)
        else:
            global_scale = float(global_scale)
        self.type, self.rows, self.K, self.matrices = type_, rows, K, matrices
        self.codes, self.scales, self.global_scale, self.plan = codes, scales, global_scale, plan

    @property
    def device(self):
        return self.codes.device


class ExpertPlan:
    """How the (token, slot) choices of an expert layer are sorted by expert: one int32 CUDA buffer that holds, one
    after the other, offsets [experts + 1], block_start [experts + 1], order [n], position [n] and scale_row [n]
    (n = tokens * slots; meanings in ``include/pnq.h``, pnq_expert_plan)."""
    __slots__ = ("tokens", "slots", "experts", "buffer", "descriptor", "ref")

    def __init__(self, tokens: int, slots: int, experts: int, buffer=None, device=None):
        n = tokens * slots
        size = 2 * (experts + 1) + 3 * n
        if buffer is None:
            buffer = torch.empty(size, dtype=torch.int32, device=device)
        _require(buffer, "plan buffer", (torch.int32,), numel=size)
        self.tokens, self.slots, self.experts, self.buffer = tokens, slots, experts, buffer
        at = buffer.data_ptr()
        order = at + 8 * (experts + 1)
        self.descriptor = pnq_expert_plan(at, at + 4 * (experts + 1), order, order + 4 * n, order + 8 * n, tokens, slots,
                                          experts)
        self.ref = ctypes.addressof(self.descriptor)

    @property
    def rows(self) -> int:
        """Sorted rows the plan has room for: tokens * slots."""
        return self.tokens * self.slots

    def _part(self, first: int, count: int):
        return self.buffer[first:first + count]

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
    K = x.shape[-1]
    rows, matrices = x.shape[-2], (x.shape[0] if x.dim() == 3 else 1)
    if x.dim() == 3 and not x.is_contiguous():
        raise PnqError("x [matrices][rows][K] must be contiguous")
    ldx = x.stride(-2)
    if x.numel() and K > 1 and x.stride(-1) != 1:
        raise PnqError("the elements of a row of x must be consecutive")
    if rows <= 1:
        ldx = K if matrices == 1 else rows * K
    if ldx < K:
        raise PnqError(f"rows of x are {ldx} elements apart; at least K = {K} is wanted")
    if K == 0 or K % G:
        raise PnqError(f"K = {K} is not a positive multiple of {G}", int(b.Status.ERR_SHAPE))
    if plan is not None:
        if matrices != 1 or rows != plan.tokens:
            raise PnqError(f"x has shape {tuple(x.shape)}; the plan has {plan.tokens} tokens")
        _same_device(x, plan.buffer)
        out_rows, experts = plan.rows, plan.experts
    else:
        out_rows, experts = rows, 0
    g = float(global_scale)
    dev = x.get_device()
    if out is None:
        pitch, size = fp4_layout(type_, out_rows, K, matrices, experts)
        out = Fp4Matrix.__new__(Fp4Matrix)
        out.type, out.rows, out.K, out.matrices = type_, out_rows, K, matrices
        out.codes = torch.empty((matrices * out_rows, pitch), dtype=torch.uint8, device=x.device)
        out.scales = torch.empty(size, dtype=torch.uint8, device=x.device)
    else:
        if (out.type, out.rows, out.K, out.matrices) != (type_, out_rows, K, matrices) or \
                (out.plan.experts if out.plan is not None else 0) != experts:
            raise PnqError("out is an operand of another type or shape")
        _same_device(x, out.codes)
    out.global_scale, out.plan = g, plan
    _call("pnq_fp4_quantize", type_, xt, x.data_ptr(), ldx, rows, K, matrices, g, None if plan is None else plan.ref,
          out.codes.data_ptr(), out.scales.data_ptr(), _stream(stream, dev))
    return out


def fp4_dequantize(m: Fp4Matrix, dtype=torch.float32, out=None, stream=None):
    """The values an operand stands for, fp32 or bf16 [matrices * rows][K] (of a plan's operand: its sorted rows,
    zeros past the rows in use). The operand's global_scale must be one float."""
    ot = _float_type(dtype if out is None else out.dtype, "out")
    if isinstance(m.global_scale, torch.Tensor):
        raise PnqError("an operand with a global scale per matrix is read back matrix by matrix")
    n = m.matrices * m.rows
    if out is None:
        out = torch.empty((n, m.K), dtype=dtype, device=m.codes.device)
    else:
        _require(out, "out", (out.dtype,), shape=(n, m.K))
        _same_device(m.codes, out)
    _call("pnq_fp4_dequantize", m.type, m.codes.data_ptr(), m.scales.data_ptr(), m.rows, m.K, m.matrices, m.global_scale,
          None if m.plan is None else m.plan.ref, ot, out.data_ptr(), _stream(stream, m.codes.get_device()))
    return out


def fp4_pack(type_: int, codes, scales, rows: int, K: int, global_scale=1.0, matrices: int = 1, stream=None) -> Fp4Matrix:
    """Row-major weights (codes uint8 [matrices * rows][K / 2], scale words uint8 [matrices * rows][K / group]) as an
    operand, once, when they are loaded. Where K is a multiple of 32 and the codes are 16-byte aligned they are kept
    as they are, not copied."""
    G = _group(type_)
    pitch, size = fp4_layout(type_, rows, K, matrices)
    n = matrices * rows
    _require(codes, "codes", (torch.uint8,), numel=n * K // 2)
    _require(scales, "scales", (torch.uint8,), numel=n * K // G)
    dev = _same_device(codes, scales)
    keep = K % 32 == 0 and codes.data_ptr() % 16 == 0
    out_codes = codes if keep else torch.empty((n, pitch), dtype=torch.uint8, device=codes.device)
    tiled = torch.empty(size, dtype=torch.uint8, device=codes.device)
    _call("pnq_fp4_pack", type_, codes.data_ptr(), scales.data_ptr(), rows, K, matrices, out_codes.data_ptr(),
          tiled.data_ptr(), _stream(stream, dev))
    return Fp4Matrix(type_, rows, K, out_codes, tiled, global_scale, matrices)


def _operands(x: Fp4Matrix, w: Fp4Matrix) -> None:
    if not isinstance(x, Fp4Matrix) or not isinstance(w, Fp4Matrix):
        raise PnqError("both operands must be Fp4Matrix")
    if x.type != w.type or x.K != w.K:
        raise PnqError(f"operands differ: type {x.type}, K = {x.K} and type {w.type}, K = {w.K}")
    if x.matrices != 1 or isinstance(x.global_scale, torch.Tensor):
        raise PnqError("the activations are one matrix with one global scale")


def _result(out, rows: int, N: int, dtype, device):
    if out is None:
        return torch.empty((rows, N), dtype=dtype, device=device)
    _require(out, "out", (torch.float32, torch.bfloat16), shape=(rows, N))
    return out


def fp4_gemm(x: Fp4Matrix, w: Fp4Matrix, dtype=torch.float32, out=None, flags: int = 0, stream=None):
    """Y[m][n] = sum_k X[m][k] W[n][k] of two operands of one type; fp32 or bf16 [M][N]."""
    _operands(x, w)
    if w.matrices != 1 or isinstance(w.global_scale, torch.Tensor) or x.plan is not None:
        raise PnqError("fp4_gemm takes one matrix each; expert layers go through fp4_gemm_experts")
    _float_type(dtype, "the result")
    out = _result(out, x.rows, w.rows, dtype, x.codes.device)
    dev = _same_device(x.codes, w.codes, out)
    _call("pnq_fp4_gemm", x.type, x.codes.data_ptr(), x.scales.data_ptr(), x.rows, w.codes.data_ptr(), w.scales.data_ptr(),
          w.rows, x.K, x.global_scale * w.global_scale, _FLOAT[out.dtype], out.data_ptr(), flags, _stream(stream, dev))
    return out


def fp4_gemm_experts(x: Fp4Matrix, w: Fp4Matrix, plan: ExpertPlan, dtype=torch.float32, out=None, flags: int = 0,
                     stream=None):
    """Every sorted row of x (made with `plan`) times its expert's matrix of w (matrices = the plan's experts): fp32 or
    bf16 [tokens * slots][N], zeros past the rows in use."""
    _operands(x, w)
    if x.plan is None or (x.plan is not plan and (x.plan.tokens, x.plan.slots, x.plan.experts) !=
                          (plan.tokens, plan.slots, plan.experts)):
        raise PnqError("x is not an operand of this plan's sorted rows")
    if w.matrices != plan.experts or w.plan is not None:
        raise PnqError(f"w has {w.matrices} matrices; the plan has {plan.experts} experts")
    _float_type(dtype, "the result")
    out = _result(out, plan.rows, w.rows, dtype, x.codes.device)
    dev = _same_device(x.codes, w.codes, out, plan.buffer)
    per = isinstance(w.global_scale, torch.Tensor)
    alpha = x.global_scale if per else x.global_scale * w.global_scale
    _call("pnq_fp4_gemm_experts", x.type, x.codes.data_ptr(), x.scales.data_ptr(), plan.ref, w.codes.data_ptr(),
          w.scales.data_ptr(), w.rows, x.K, alpha, w.global_scale.data_ptr() if per else None, _FLOAT[out.dtype],
          out.data_ptr(), flags, _stream(stream, dev))
    return out


# ---- tokens to their experts and back ----------------------------------------------------------------

def expert_sort(ids, experts: int, plan: ExpertPlan | None = None, stream=None) -> ExpertPlan:
    """The plan of ids (CUDA int32 [tokens][slots]: the expert of each choice; one outside 0 .. experts - 1 is dropped):
    stable, so equal experts keep the order of their slots."""
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise PnqError("ids must be a torch.Tensor [tokens][slots]")
    _require(ids, "ids", (torch.int32,))
    tokens, slots = ids.shape
    if not 1 <= slots <= 64 or not 1 <= experts <= 1024:
        raise PnqError(f"{slots} slots and {experts} experts; 1..64 and 1..1024 are wanted", int(b.Status.ERR_SHAPE))
    if plan is None:
        plan = ExpertPlan(tokens, slots, experts, device=ids.device)
    elif (plan.tokens, plan.slots, plan.experts) != (tokens, slots, experts):
        raise PnqError("the plan is of another shape")
    dev = _same_device(ids, plan.buffer)
    _call("pnq_expert_sort", ids.data_ptr(), plan.ref, _stream(stream, dev))
    return plan


def _rows_in(t, what: str, rows: int, D=None):
    """(element type, row length) of a contiguous CUDA [rows][D] tensor."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise PnqError(f"{what} must be a torch.Tensor [rows][D]")
    ft = _float_type(t.dtype, what)
    _require(t, what, (t.dtype,), shape=(rows, t.shape[1] if D is None else D))
    return ft, t.shape[1]


def _rows_out(out, like, rows: int, D: int):
    if out is None:
        return torch.empty((rows, D), dtype=like.dtype, device=like.device)
    _require(out, "out", (like.dtype,), shape=(rows, D))
    return out


def _weights_of(weights, plan: ExpertPlan) -> None:
    _require(weights, "weights", (torch.float32,), shape=(plan.tokens, plan.slots))


def expert_gather(x, plan: ExpertPlan, out=None, stream=None):
    """Sorted rows of x (fp32 or bf16 [tokens][D]): [tokens * slots][D], zeros past the rows in use."""
    ft, D = _rows_in(x, "x", plan.tokens)
    out = _rows_out(out, x, plan.rows, D)
    dev = _same_device(x, plan.buffer, out)
    _call("pnq_expert_gather", ft, x.data_ptr(), D, plan.ref, out.data_ptr(), _stream(stream, dev))
    return out


def expert_gather_backward(dxs, plan: ExpertPlan, out=None, stream=None):
    """Gradient of expert_gather: dx [tokens][D], each token's rows summed in fp32 in slot order."""
    ft, D = _rows_in(dxs, "dxs", plan.rows)
    out = _rows_out(out, dxs, plan.tokens, D)
    dev = _same_device(dxs, plan.buffer, out)
    _call("pnq_expert_gather_backward", ft, dxs.data_ptr(), D, plan.ref, out.data_ptr(), _stream(stream, dev))
    return out


def expert_combine(ys, plan: ExpertPlan, weights, out=None, stream=None):
    """y[t] = sum over t's slots of weights[t][j] * its row of ys ([tokens * slots][D]; weights fp32 [tokens][slots])."""
    ft, D = _rows_in(ys, "ys", plan.rows)
    _weights_of(weights, plan)
    out = _rows_out(out, ys, plan.tokens, D)
    dev = _same_device(ys, plan.buffer, weights, out)
    _call("pnq_expert_combine", ft, ys.data_ptr(), D, plan.ref, weights.data_ptr(), out.data_ptr(), _stream(stream, dev))
    return out


def expert_combine_backward(dy, ys, plan: ExpertPlan, weights, out=None, dweights=None, stream=None):
    """Gradients of expert_combine: (dys [tokens * slots][D], dweights fp32 [tokens][slots])."""
    ft, D = _rows_in(ys, "ys", plan.rows)
    if _rows_in(dy, "dy", plan.tokens, D)[0] != ft:
        raise PnqError(f"dy has dtype {dy.dtype}, ys {ys.dtype}; one type is wanted")
    _weights_of(weights, plan)
    out = _rows_out(out, ys, plan.rows, D)
    if dweights is None:
        dweights = torch.empty((plan.tokens, plan.slots), dtype=torch.float32, device=ys.device)
    else:
        _require(dweights, "dweights", (torch.float32,), shape=(plan.tokens, plan.slots))
    dev = _same_device(ys, dy, plan.buffer, weights, out, dweights)
    _call("pnq_expert_combine_backward", ft, dy.data_ptr(), ys.data_ptr(), D, plan.ref, weights.data_ptr(), out.data_ptr(),
          dweights.data_ptr(), _stream(stream, dev))
    return out, dweights
