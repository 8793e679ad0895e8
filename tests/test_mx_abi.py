"""Refusals of the microscaled operators, all on the CPU: the C entries check
their arguments before any launch, the binding before any C call."""
import ctypes
import math
import os

import pytest
import torch

from lossless_float_weight_amd import zn

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "lossless_float_weight_amd", "libzn.so")
pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libzn.so not built")

P = 1 << 20        # an aligned address that is never read: every call here is refused or has no rows
BF16, FP32, FP8, FP4 = zn.BF16, zn.FP32, zn.FP8_E4M3, zn.FP4X2_E2M1
ARG, CAPACITY = -1, -3


def _with(base, **change):
    args = dict(base)
    args.update(change)
    return list(args.values())


QUANT = dict(dtype=BF16, x=P, stride=64, rows=0, k=64, fmt=FP8, codes=P, scales=P, stream=None)


@pytest.mark.parametrize("bad", [
    dict(dtype=FP8), dict(dtype=9), dict(fmt=BF16), dict(fmt=7), dict(k=0), dict(k=(1 << 30) + 1), dict(rows=1 << 31),
    dict(stride=(1 << 40) + 1), dict(rows=1, x=None), dict(rows=1, x=P + 1), dict(rows=1, codes=None),
    dict(rows=1, codes=P + 8), dict(rows=1, scales=None), dict(rows=1, dtype=FP32, x=P + 2)])
def test_quantize_refuses(bad):
    f = zn.lib().zn_mx_quantize
    assert f(*_with(QUANT)) == 0                    # no rows: nothing is launched
    assert f(*_with(QUANT, **bad)) == ARG


DEQUANT = dict(fmt=FP8, codes=P, scales=P, rows=0, k=64, dtype=BF16, out=P, stride=64, stream=None)


@pytest.mark.parametrize("bad", [
    dict(fmt=BF16), dict(dtype=FP4), dict(k=0), dict(k=(1 << 30) + 1), dict(rows=1 << 31), dict(rows=2, stride=63),
    dict(rows=1, codes=None), dict(rows=1, codes=P + 4), dict(rows=1, scales=None), dict(rows=1, out=None),
    dict(rows=1, out=P + 1), dict(stride=(1 << 40) + 1)])
def test_dequantize_refuses(bad):
    f = zn.lib().zn_mx_dequantize
    assert f(*_with(DEQUANT)) == 0
    assert f(*_with(DEQUANT, **bad)) == ARG


NORM = dict(dtype=BF16, x=P, stride=64, res=P, rs=64, w=P, eps=1e-5, rows=0, k=64, h=P, hs=64, fmt=FP8, codes=P,
            scales=P, stream=None)


@pytest.mark.parametrize("bad", [
    dict(dtype=FP8), dict(fmt=FP32), dict(k=0), dict(rows=1 << 31), dict(eps=-1.0), dict(eps=math.nan),
    dict(eps=math.inf), dict(res=None), dict(h=None), dict(rows=2, hs=63), dict(rs=(1 << 40) + 1),
    dict(hs=(1 << 40) + 1), dict(rows=1, x=None), dict(rows=1, w=None), dict(rows=1, w=P + 1),
    dict(rows=1, res=P + 1), dict(rows=1, h=P + 1), dict(rows=1, codes=P + 2), dict(rows=1, codes=None),
    dict(rows=1, scales=None)])
def test_norm_refuses(bad):
    f = zn.lib().zn_mx_rms_norm
    assert f(*_with(NORM)) == 0
    assert f(*_with(NORM, res=None, h=None)) == 0
    assert f(*_with(NORM, **bad)) == ARG


MATMUL = dict(fa=FP8, a=P, sa=P, fw=FP4, w=P, sw=P, m=0, n=64, k=64, dtype=BF16, out=P, stride=64, scratch=None,
              bytes=0, stream=None)


@pytest.mark.parametrize("bad", [
    dict(fa=BF16), dict(fw=FP32), dict(dtype=FP8), dict(k=0), dict(k=48), dict(k=(1 << 30) + 32), dict(m=1 << 31),
    dict(n=1 << 31), dict(m=2, stride=63), dict(stride=(1 << 40) + 1), dict(m=1, a=None), dict(m=1, a=P + 8),
    dict(m=1, sa=None), dict(m=1, w=None), dict(m=1, w=P + 8), dict(m=1, sw=None), dict(m=1, out=None),
    dict(m=1, out=P + 1)])
def test_matmul_refuses(bad):
    f = zn.lib().zn_mx_matmul
    assert f(*_with(MATMUL)) == 0
    assert f(*_with(MATMUL, m=1, n=0)) == 0
    assert f(*_with(MATMUL, **bad)) == ARG


def test_matmul_scratch_is_asked_and_checked():
    L = zn.lib()
    b = ctypes.c_uint64()
    assert L.zn_mx_matmul_scratch_bytes(FP8, FP4, 4, 64, 64, None) == ARG
    assert L.zn_mx_matmul_scratch_bytes(FP8, FP4, 4, 64, 33, ctypes.byref(b)) == ARG
    assert L.zn_mx_matmul_scratch_bytes(FP8, FP4, 0, 64, 64, ctypes.byref(b)) == 0 and b.value == 0
    for fa in (FP8, FP4):
        for fw in (FP8, FP4):
            for m, n, k in ((1, 16, 32), (48, 4096, 14336), (100, 200, 8192), (300, 1024, 14336), (8192, 28672, 4096)):
                need = zn.mx_matmul_scratch_bytes(fa, fw, m, n, k)
                assert need < 1 << 31
                if need:
                    args = dict(fa=fa, fw=fw, m=m, n=n, k=k, stride=n)
                    assert L.zn_mx_matmul(*_with(MATMUL, **args)) == ARG                       # none given
                    assert L.zn_mx_matmul(*_with(MATMUL, **args, scratch=P, bytes=need - 1)) == CAPACITY
                    assert L.zn_mx_matmul(*_with(MATMUL, **args, scratch=P + 8, bytes=need)) == ARG


def test_row_views():
    rows = zn._mx_rows
    x = torch.zeros(6, 40)
    assert rows("t", "x", x) == (6, 40, 40)
    assert rows("t", "x", x[:, :33]) == (6, 33, 40)
    assert rows("t", "x", x[::2]) == (3, 40, 80)
    assert rows("t", "x", x[0]) == (1, 40, 40)
    assert rows("t", "x", x.view(2, 3, 40)[:, :, 1:]) == (6, 39, 40)
    assert rows("t", "x", x[:1].expand(4, 40)) == (4, 40, 0)
    assert rows("t", "x", x[:0]) == (0, 40, 40)
    assert rows("t", "x", x[:, 3:4]) == (6, 1, 40)
    assert rows("t", "x", torch.zeros(0, 3, 40)[:, :, :8]) == (0, 8, 8)
    for bad in (x.t(), x[:, ::2], x.view(2, 3, 40)[:, :2], torch.zeros(())):
        with pytest.raises(zn.ZnError):
            rows("t", "x", bad)
    with pytest.raises(zn.ZnError):
        rows("t", "x", x[:1].expand(4, 40), write=True)


def _raises(f, *a, **k):
    with pytest.raises(zn.ZnError) as e:
        f(*a, **k)
    assert e.value.code == -1


def test_binding_refuses_types_and_devices():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    c8, c4 = torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.zeros(4, 32, dtype=torch.uint8)
    s = torch.zeros(4, 2, dtype=torch.float8_e8m0fnu)
    _raises(zn.mx_quantize, x)                                       # on the CPU
    _raises(zn.mx_quantize, x.half())
    _raises(zn.mx_dequantize, c8, s)                                 # on the CPU
    _raises(zn.mx_dequantize, x, s)                                  # no codes
    _raises(zn.mx_dequantize, c8, s[:, :1].contiguous())
    _raises(zn.mx_dequantize, c8, s.view(torch.uint8).to(torch.int32))
    _raises(zn.mx_dequantize, c8, s, k=32)
    _raises(zn.mx_dequantize, c8, s, k=65)
    _raises(zn.mx_dequantize, c8.t(), s)
    _raises(zn.mx_dequantize, c4[:, :24].contiguous(), s)            # half a block
    _raises(zn.mx_rms_norm, x, x[0])
    _raises(zn.mx_rms_norm, x.half(), x[0].half())
    _raises(zn.mx_matmul, c8, s, c4, s)
    _raises(zn.mx_matmul, c8, s, c4.view(2, 2, 32), s.view(2, 2, 2))
    _raises(zn.mx_matmul, c8, s, c4[:, :16].contiguous(), s[:, :1].contiguous())
    _raises(zn._mx_codes, "t", (4,), 64, zn.BF16, None, None, x.device, None)
    _raises(zn._mx_codes, "t", (4,), 0, zn.FP8_E4M3, None, None, x.device, None)
    _raises(zn._mx_codes, "t", (4,), 64, zn.FP8_E4M3, c4, None, x.device, None)
    _raises(zn._mx_codes, "t", (4,), 64, zn.FP8_E4M3, c8, s[:2], x.device, None)
    got = zn._mx_codes("t", (4,), 64, zn.FP4X2_E2M1, c4, s, x.device, None)
    assert got[0] is c4 and got[1] is s
