"""Refusals of the key-value cache's calls that take flags, and which kernel takes a call, on the CPU."""
import ctypes
import os

import pytest
import torch

from lossless_float_weight_amd import zn
from test_kv_abi import ARG, ATTEND, CAPACITY, FP32, LIB, P, _raises, cache, i32

pytestmark = pytest.mark.skipif(not os.path.exists(LIB), reason="libzn.so not built")


def attend2(flags, scratch=None, nbytes=0, **change):
    return zn.lib().zn_mx_attention2(cache(), zn._ATTENTION_ARGS.pack(*dict(ATTEND, **change).values()), flags, scratch, nbytes, None)


def test_attention_flags():
    assert attend2(0) == 0 and attend2(zn.MX_FAST_WEIGHTS) == 0             # no queries: nothing is launched
    assert attend2(0, dtype=FP32) == 0
    for flags, bad in ((2, {}), (3, {}), (1 << 31, {}), (1, dict(dtype=FP32)), (1, dict(heads=3)), (1, dict(window=4, causal=0)),
                       (1, dict(dtype=9))):
        assert attend2(flags, **bad) == ARG
    assert zn.lib().zn_mx_attention2(cache(), None, 1, None, 0, None) == ARG
    size = dict(batch=8, tokens=4096, starts=P, width=4096, ts=4096)
    assert attend2(1, P, 16, **size) == CAPACITY and attend2(1, **size) == ARG


def test_binding_refuses_fast_weights_beside_fp32():
    c = zn.mx_kv_cache(6, 2, 16, 64, device="cpu")
    q = torch.zeros(5, 4, 64)
    _raises(zn.mx_attention, q, c, i32(5, 4), i32(5), fast_weights=True, match="fast_weights is for bfloat16")
    _raises(zn.mx_attention, q.bfloat16(), c, i32(5, 4), i32(5), fast_weights=True, match="not on a CUDA device")


def kernel_of(batch, width, tokens=None, heads=4, kv_heads=2, dim=64, dtype=torch.bfloat16, page=16, **kw):
    c = zn.mx_kv_cache(1, kv_heads, page, dim, device="cpu")
    starts = None if tokens is None else i32(batch + 1)
    # (no memory behind the queries' and the table's shapes)
    q = torch.zeros(1, 1, 1, dtype=dtype).expand(batch if tokens is None else tokens, heads, dim)
    return zn.debug_attention_kernel(q, c, i32(1, 1).expand(batch, width), starts, **kw)


def test_which_kernel_takes_a_call():
    assert kernel_of(0, 8) == "none" and kernel_of(3, 8, tokens=0) == "none"
    for dtype in (torch.bfloat16, torch.float32):
        assert kernel_of(1, 64, dtype=dtype) == "short" and kernel_of(600, 8, dtype=dtype) == "short pairs"
        assert kernel_of(1, 4096, dtype=dtype) == "few rows"
        assert kernel_of(4, 65536, tokens=1000, max_new=250, dtype=dtype) == "many rows"
    L, b = zn.lib(), ctypes.c_int()
    g = zn._ATTENTION_ARGS.pack(*ATTEND.values())
    assert L.zn_debug_attention_kernel(cache(), g, None) == ARG
    assert L.zn_debug_attention_kernel(cache(), None, ctypes.byref(b)) == ARG
    assert L.zn_debug_attention_kernel(cache(), zn._ATTENTION_ARGS.pack(*dict(ATTEND, heads=3).values()), ctypes.byref(b)) == ARG


def test_a_wrong_hint_makes_no_grid_too_large():
    # 2^25 groups of 16 rows: with two waves each more than the 2^32 threads of a grid
    for dtype, dim in ((torch.bfloat16, 32), (torch.bfloat16, 64), (torch.float32, 128)):
        size = dict(tokens=1 << 29, heads=1, kv_heads=1, dim=dim, dtype=dtype)
        assert kernel_of(8192, 8, max_new=1, **size) != "short pairs"
        assert kernel_of(8192, 8, max_new=1, **dict(size, tokens=1 << 20)) == "short pairs"


def test_binding_refuses_to_cut_keys_and_values_from_a_graph():
    c = zn.mx_kv_cache(6, 2, 16, 64, device="cpu")
    x = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    g = torch.zeros(5, 2, 64, dtype=torch.bfloat16, requires_grad=True)
    _raises(zn.mx_kv_write, g, x, c, i32(5), match="k requires a gradient")
    _raises(zn.mx_kv_write, x, g * 2, c, i32(5), match="v requires a gradient")
    _raises(zn.mx_kv_write, g.detach(), x, c, i32(5), match="not on a CUDA device")
    with torch.no_grad():
        _raises(zn.mx_kv_write, g, g, c, i32(5), match="not on a CUDA device")
