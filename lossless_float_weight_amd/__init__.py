"""Lossless exponent-Huffman codec for floating-point tensors on AMD MI355X.

The GPU path is libzn.so (HIP kernels for gfx950, C ABI in include/zn.h);
`zn` is its Python binding and `workloads` the seeded synthetic inputs.  Beside
the codec stand the microscaled operators (mx_*): the quantiser that makes its
FP8 and FP4 tensors, their way back, and the norm and product that use them.
"""
from . import workloads  # noqa: F401
from . import zn  # noqa: F401
from .zn import (BF16, FP32, FP8_E4M3, FP4X2_E2M1, Tableset, ZnError, compress,  # noqa: F401
                 compress_bound, decompress, mx_dequantize, mx_matmul, mx_matmul_scratch_bytes, mx_quantize,
                 mx_rms_norm, plan_from_container, scratch_bytes, setup, setup_transfer)
