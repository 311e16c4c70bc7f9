"""pnq: block-quantized weight GEMV (pn3t, pn4t, NVFP4 W4A16, grouped signed-integer formats)
and 4-bit microscaled products (NVFP4, MXFP4) with the expert layer around them, for sm_103a.

The compute path is the C-ABI library ``libpnq.so`` built from ``csrc/``; this
package only marshals arguments to it (see ``_binding``). Importing the package
does not load the library; the first call does, and raises if it is missing.
"""
from ._binding import (PN3T, PN4T, NVFP4, NVFP4_DIV, Q4G64_F16S, Q5G64_F16S, Q6G64_F16S, W8G32_F16S, GROUPED,
                       BLOCK_WEIGHTS, GEMV_STATIC_WEIGHTS, Status, PnqError, lib, lib_path, gemv,
                       gemv_ex_ptr, gemv_noalloc, gemv_noalloc_ptr, grouped_plane_shapes,
                       dequantize_row, validate_row, quantize_row, gemv_ptr, dequantize_row_ptr, validate_row_ptr,
                       quantize_row_ptr, quantize_nvfp4_clip, selftest_wait, gemm, gemm_scratch_bytes, device_error, nvfp4_weights, pnq_grouped_weights)

# the 4-bit operands and the expert layer work on torch tensors throughout: their module (with torch and both
# libraries) is imported at the first use of one of its names, and `import *`, which would use them all, leaves them out
_FP4_NAMES = ("MXFP4", "FP4_GROUP", "Fp4Matrix", "ExpertPlan", "fp4_lib", "fp4_layout", "fp4_quantize",
              "fp4_dequantize", "fp4_pack", "fp4_gemm", "fp4_gemm_experts", "expert_sort", "expert_gather",
              "expert_gather_backward", "expert_combine", "expert_combine_backward")


def __getattr__(name):
    if name in _FP4_NAMES:
        from . import _fp4
        globals().update({n: getattr(_fp4, n) for n in _FP4_NAMES})
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def __dir__():
    return sorted({*globals(), *_FP4_NAMES})


__all__ = ["PN3T", "PN4T", "NVFP4", "NVFP4_DIV", "Q4G64_F16S", "Q5G64_F16S", "Q6G64_F16S", "W8G32_F16S", "GROUPED",
           "BLOCK_WEIGHTS", "GEMV_STATIC_WEIGHTS", "gemv_ex_ptr", "gemv_noalloc", "gemv_noalloc_ptr",
           "grouped_plane_shapes", "Status", "PnqError", "lib", "lib_path", "gemv", "dequantize_row", "validate_row",
           "quantize_row", "quantize_nvfp4_clip", "selftest_wait", "gemm", "gemm_scratch_bytes", "gemv_ptr", "dequantize_row_ptr", "validate_row_ptr", "quantize_row_ptr", "device_error",
           "nvfp4_weights", "pnq_grouped_weights"]
