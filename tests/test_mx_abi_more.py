"""More refusals of the microscaled operators, on the CPU."""
import os

import pytest
import torch

from lossless_float_weight_amd import zn
from test_mx_abi import ARG, CAPACITY, FP32, FP8, LIB, MATMUL, P, _with

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libzn.so not built")


def matmul2(**change):
    args = dict(MATMUL, **{k: v for k, v in change.items() if k != "flags"})
    a = list(args.values())
    return zn.lib().zn_mx_matmul2(*a[:9], change.get("flags", 0), *a[9:])


def test_flags_of_the_product():
    assert matmul2() == 0 and matmul2(flags=zn.MX_FAST_SUMS) == 0          # no rows: nothing is launched
    assert matmul2(dtype=FP32) == 0
    for bad in (dict(flags=2), dict(flags=1 << 31), dict(flags=3), dict(flags=1, dtype=FP32), dict(flags=1, dtype=FP8),
                dict(flags=1, m=1, a=None), dict(flags=1, m=1, out=P + 1), dict(flags=1, k=48)):
        assert matmul2(**bad) == ARG
    need = zn.mx_matmul_scratch_bytes(zn.FP8_E4M3, zn.FP4X2_E2M1, 48, 4096, 14336)
    size = dict(flags=1, m=48, n=4096, k=14336, stride=4096, scratch=P)
    assert need > 0 and matmul2(**size, bytes=need - 1) == CAPACITY
    assert zn.lib().zn_mx_matmul(*_with(MATMUL)) == 0


def test_products_of_more_tiles_than_a_grid_holds_need_no_scratch():
    # 2^24 tiles of 256 threads would pass a grid: the way of few rows, which lays nothing out
    for fa in (zn.FP8_E4M3, zn.FP4X2_E2M1):
        assert zn.mx_matmul_scratch_bytes(fa, zn.FP4X2_E2M1, 17, (1 << 31) - 1, 32) == 0
        for m, n in ((17, 1 << 30), (64, (1 << 30) - 63), (65, (1 << 31) - 127)):
            assert zn.mx_matmul_scratch_bytes(fa, zn.FP4X2_E2M1, m, n, 32) == 0
        for m, n in ((17, (1 << 30) - 64), (64, (1 << 30) - 64), (65, (1 << 31) - 128)):
            assert zn.mx_matmul_scratch_bytes(fa, zn.FP4X2_E2M1, m, n, 32) == (m + n) * 16


def test_a_sum_that_would_leave_the_graph_is_refused():
    x, r, w = (torch.zeros(s, dtype=torch.bfloat16) for s in ((4, 64), (4, 64), (64,)))
    g = torch.zeros(4, 64, dtype=torch.bfloat16, requires_grad=True)

    def refused(f, *a, **k):
        with pytest.raises(zn.ZnError, match="requires a gradient") as e:
            f(*a, **k)
        assert e.value.code == ARG

    def passes(f, *a, **k):                     # as far as the device, which is the CPU here
        with pytest.raises(zn.ZnError, match="not on a CUDA device"):
            f(*a, **k)

    refused(zn.mx_rms_norm, g, w, residual=r)
    refused(zn.mx_rms_norm, x, w, residual=g)
    refused(zn.mx_rms_norm, x, w, residual=g * 1)
    refused(zn.mx_rms_norm, x, w, residual=r, residual_out=g)
    c, s = torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.zeros(4, 2, dtype=torch.float8_e8m0fnu)
    refused(zn.mx_dequantize, c, s, out=g)
    refused(zn.mx_matmul, c, s, c, s, out=g)
    passes(zn.mx_rms_norm, g, w)                # h is x itself, with its graph
    passes(zn.mx_rms_norm, x, w.clone().requires_grad_(), residual=r)
    with torch.no_grad():
        passes(zn.mx_rms_norm, g, w, residual=r)
        passes(zn.mx_dequantize, c, s, out=g)
        passes(zn.mx_matmul, c, s, c, s, out=g)
    passes(zn.mx_rms_norm, g.detach(), w, residual=r)
    passes(zn.mx_quantize, g)                   # codes have no derivative


def test_torch_without_the_short_ways():
    assert zn._torch_c("_no_such_function", len) is len
    assert callable(zn._torch_c("_cuda_getDevice", None) or len)
