"""Refusals of the key-value cache's calls, all on the CPU: the C entries check
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
Q = P + 64
BF16, FP32, FP8, FP4 = zn.BF16, zn.FP32, zn.FP8_E4M3, zn.FP4X2_E2M1
ARG, CAPACITY = -1, -3
FAR = (1 << 40) + 1

CACHE = dict(k=P, ks=P, v=P, vs=P, n_pages=8, page_size=16, kv_heads=2, head_dim=64, reserved=0, page_stride=64,
             head_stride=32, place_stride=2)
BAD_CACHES = [
    dict(page_size=8), dict(page_size=24), dict(page_size=131072), dict(n_pages=0), dict(n_pages=1 << 27),
    dict(kv_heads=0), dict(kv_heads=1025), dict(head_dim=0), dict(head_dim=48), dict(head_dim=288), dict(reserved=1),
    dict(page_stride=FAR), dict(head_stride=FAR), dict(place_stride=(1 << 20) + 1), dict(page_stride=1 << 32)]
BAD_ADDRESSES = [dict(k=0), dict(k=P + 8), dict(v=0), dict(v=P + 4), dict(ks=0), dict(vs=0)]


def cache(**change):
    return zn._CACHE_ARGS.pack(*dict(CACHE, **change).values())


EXTEND = dict(lens=P, add=P, batch=4, table=P, ts=8, width=8, free=P, cap=8, n_free=P, page=16, n_pages=8, tokens=4,
              new_lens=Q, starts=Q, slots=Q, positions=Q, n_left=Q, stream=None)


@pytest.mark.parametrize("bad", [
    dict(lens=None), dict(lens=P + 2), dict(add=None), dict(add=P + 1), dict(batch=8193), dict(table=None), dict(ts=7),
    dict(ts=FAR), dict(width=1 << 27, ts=1 << 27), dict(free=None), dict(cap=1 << 31), dict(n_free=None), dict(page=0),
    dict(page=24), dict(page=131072), dict(n_pages=1 << 27), dict(tokens=1 << 31), dict(new_lens=None),
    dict(new_lens=P), dict(starts=None), dict(slots=None), dict(positions=None), dict(n_left=None), dict(n_left=P)])
def test_extend_refuses(bad):
    assert zn.lib().zn_kv_extend(*dict(EXTEND, **bad).values()) == ARG


RELEASE = dict(lens=P, done=P, batch=4, table=P, ts=8, width=8, free=P, cap=8, n_free=P, page=16, new_lens=Q, n_left=Q,
               stream=None)


@pytest.mark.parametrize("bad", [
    dict(lens=None), dict(done=None), dict(batch=8193), dict(table=None), dict(ts=7), dict(width=1 << 27, ts=1 << 27),
    dict(free=None), dict(free=P + 2), dict(cap=1 << 31), dict(n_free=None), dict(page=3), dict(new_lens=None),
    dict(new_lens=P), dict(n_left=None), dict(n_left=P)])
def test_release_refuses(bad):
    assert zn.lib().zn_kv_release(*dict(RELEASE, **bad).values()) == ARG


WRITE = dict(dtype=BF16, k=P, kt=128, kh=64, v=P, vt=128, vh=64, slots=P, tokens=0, cache=None, stream=None)


@pytest.mark.parametrize("bad", [
    dict(dtype=FP8), dict(dtype=9), dict(tokens=1 << 31), dict(cache=None), dict(kt=FAR), dict(kh=FAR), dict(vt=FAR),
    dict(vh=FAR), dict(tokens=1, k=None), dict(tokens=1, k=P + 1), dict(tokens=1, v=None),
    dict(tokens=1, dtype=FP32, v=P + 2), dict(tokens=1, slots=None), dict(tokens=1, slots=P + 2)])
def test_write_refuses(bad):
    f = zn.lib().zn_mx_kv_write
    good = dict(WRITE, cache=cache())
    assert f(*good.values()) == 0                       # no tokens: nothing is launched
    assert f(*dict(good, **bad).values()) == ARG


READ = dict(cache=None, slots=P, tokens=0, dtype=BF16, k=P, v=P, stream=None)


@pytest.mark.parametrize("bad", [
    dict(dtype=FP4), dict(tokens=1 << 31), dict(cache=None), dict(tokens=1, k=None), dict(tokens=1, v=P + 1),
    dict(tokens=1, slots=None)])
def test_read_refuses(bad):
    f = zn.lib().zn_mx_kv_read
    good = dict(READ, cache=cache())
    assert f(*good.values()) == 0
    assert f(*dict(good, **bad).values()) == ARG


ATTEND = dict(dtype=BF16, heads=4, batch=0, tokens=0, max_new=0, q=P, qt=256, qh=64, out=Q, ot=256, oh=64, lse=0,
              table=P, lens=P, starts=0, ts=8, width=8, scale=0.125, causal=1, window=0)


def attend(scratch=None, nbytes=0, c=None, **change):
    g = zn._ATTENTION_ARGS.pack(*dict(ATTEND, **change).values())
    return zn.lib().zn_mx_attention(c or cache(), g, scratch, nbytes, None)


@pytest.mark.parametrize("bad", [
    dict(dtype=FP8), dict(heads=0), dict(heads=3), dict(batch=8193, tokens=8193), dict(tokens=1), dict(batch=1),
    dict(tokens=(1 << 27) + 1, starts=P), dict(qt=FAR), dict(qh=FAR), dict(ot=FAR), dict(oh=FAR), dict(ts=FAR),
    dict(batch=2, tokens=2, ts=7), dict(width=1 << 27, ts=1 << 27), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=math.nan), dict(scale=math.inf), dict(window=1 << 31), dict(window=4, causal=0),
    dict(batch=2, tokens=2, oh=63), dict(batch=2, tokens=2, ot=255), dict(batch=2, tokens=2, ot=64, oh=64),
    dict(batch=3, tokens=3, ot=64, oh=191), dict(batch=2, tokens=2, ot=0), dict(batch=2, tokens=2, oh=0)])
def test_attention_refuses(bad):
    assert attend() == 0
    assert attend(**bad) == ARG
    g = zn._ATTENTION_ARGS.pack(*dict(ATTEND, **bad).values())
    b = ctypes.c_uint64()
    assert zn.lib().zn_mx_attention_scratch_bytes(cache(), g, ctypes.byref(b)) == ARG


def test_attention_takes_scales_to_2_127():
    assert attend(scale=2.0 ** 127) == 0 and attend(scale=2.0 ** -149) == 0
    assert attend(scale=2.0 ** 127 * (1 + 2.0 ** -23)) == ARG


@pytest.mark.parametrize("bad", [
    dict(q=0), dict(q=P + 1), dict(dtype=FP32, q=P + 2), dict(out=0), dict(out=P + 1), dict(lse=P + 2), dict(table=0),
    dict(table=P + 2), dict(lens=0), dict(lens=P + 1), dict(starts=P + 2)])
def test_attention_refuses_addresses(bad):
    one = dict(batch=1, tokens=1, width=4)
    assert attend(scratch=P, nbytes=1 << 40, **dict(one, **bad)) == ARG


@pytest.mark.parametrize("bad", BAD_CACHES)
def test_caches_refused(bad):
    L, c = zn.lib(), cache(**bad)
    assert L.zn_mx_kv_write(*dict(WRITE, cache=c).values()) == ARG
    assert L.zn_mx_kv_read(*dict(READ, cache=c).values()) == ARG
    assert attend(c=c) == ARG


@pytest.mark.parametrize("bad", BAD_ADDRESSES)
def test_cache_addresses_refused(bad):
    L, c = zn.lib(), cache(**bad)
    assert L.zn_mx_kv_write(*dict(WRITE, cache=c).values()) == 0
    assert L.zn_mx_kv_write(*dict(WRITE, cache=c, tokens=1).values()) == ARG
    assert L.zn_mx_kv_read(*dict(READ, cache=c, tokens=1).values()) == ARG
    assert attend(c=c, batch=1, tokens=1, width=4, scratch=P, nbytes=1 << 40) == ARG


def test_results_may_lie_either_way():
    b = ctypes.c_uint64()
    for change in (dict(), dict(ot=64, oh=192), dict(ot=64, oh=FAR - 1), dict(ot=300, oh=70), dict(heads=2, batch=1, tokens=1, oh=64, ot=0)):
        g = zn._ATTENTION_ARGS.pack(*dict(ATTEND, **dict(dict(batch=3, tokens=3), **change)).values())
        assert zn.lib().zn_mx_attention_scratch_bytes(cache(), g, ctypes.byref(b)) == 0


def test_attention_scratch_is_asked_and_checked():
    L = zn.lib()
    b = ctypes.c_uint64()
    g = zn._ATTENTION_ARGS.pack(*ATTEND.values())
    assert L.zn_mx_attention_scratch_bytes(cache(), g, None) == ARG
    assert L.zn_mx_attention_scratch_bytes(cache(), None, ctypes.byref(b)) == ARG
    assert L.zn_mx_attention_scratch_bytes(None, g, ctypes.byref(b)) == ARG
    assert L.zn_mx_attention_scratch_bytes(cache(), g, ctypes.byref(b)) == 0 and b.value == 0
    for size in (dict(batch=1, tokens=1, width=4096, ts=4096), dict(batch=64, tokens=64, width=1024, ts=1024),
                 dict(batch=8, tokens=4096, starts=P, width=512, ts=512)):
        g = zn._ATTENTION_ARGS.pack(*dict(ATTEND, **size).values())
        assert L.zn_mx_attention_scratch_bytes(cache(), g, ctypes.byref(b)) == 0
        need = b.value
        assert 0 < need < 1 << 30
        assert attend(**size) == ARG                                        # none given
        assert attend(scratch=P, nbytes=need - 1, **size) == CAPACITY
        assert attend(scratch=P + 8, nbytes=need, **size) == ARG


def _raises(f, *a, match=None, **k):
    with pytest.raises(zn.ZnError, match=match) as e:
        f(*a, **k)
    assert e.value.code == ARG


ON_CPU = "not on a CUDA device"


def test_binding_refuses_caches():
    lay = lambda c: zn._kv_cache("t", c)[1]                                 # noqa: E731
    c = zn.mx_kv_cache(6, 2, 16, 96, device="cpu")
    assert lay(c) == (6, 16, 2, 96, (96, 48, 3))
    assert lay(zn.MxCache(*(t.view(torch.uint8) for t in c))) == lay(c)
    both = [torch.zeros(6, 2, 3, 16, n, dtype=torch.uint8) for n in (32, 2)]   # keys beside values in a page
    assert lay((both[0][:, 0], both[1][:, 0], both[0][:, 1], both[1][:, 1])) == (6, 16, 3, 64, (192, 32, 2))
    near = [torch.zeros(6, 16, 2, n, dtype=torch.uint8).transpose(1, 2) for n in (32, 2)]  # heads beside each other
    assert lay((near[0], near[1], near[0], near[1])) == (6, 16, 2, 64, (64, 2, 4))
    one = [torch.zeros(1, 1, 16, n, dtype=torch.uint8) for n in (16, 1)]
    assert lay((one[0], one[1], one[0], one[1])) == (1, 16, 1, 32, (1, 1, 1))
    k, ks, v, vs = c
    for bad in ((k.float(), ks, v, vs), (k, ks.view(torch.uint8).float(), v, vs), (k[:5], ks, v, vs), (k, ks[:5], v, vs),
                (k, ks, v[:, :1], vs), (k[0], ks[0], v[0], vs[0]), (k[..., :40], ks, v[..., :40], vs),
                (k[:, :, :12], ks[:, :, :12], v[:, :, :12], vs[:, :, :12]),
                (k[:, :, ::2], ks[:, :, :8], v[:, :, ::2], vs[:, :, :8]),
                (k.transpose(0, 1), ks.transpose(0, 1), v.transpose(0, 1), vs[:2].expand(2, 2, 16, 3)),
                (k[:1].expand(6, 2, 16, 48), ks[:1].expand(6, 2, 16, 3), v[:1].expand(6, 2, 16, 48),
                 vs[:1].expand(6, 2, 16, 3)),
                (k.transpose(2, 3), ks, v, vs), (near[0], both[1][:, 0, :2], near[0], near[1])):
        _raises(zn._kv_cache, "t", bad)
    for bad in ((0, 2, 16, 64), (1 << 27, 2, 16, 64), (4, 0, 16, 64), (4, 2, 8, 64), (4, 2, 24, 64), (4, 2, 16, 48),
                (4, 2, 16, 0), (4, 2, 16, 288), (4, 1025, 16, 64)):
        _raises(zn.mx_kv_cache, *bad, device="cpu")


def i32(*n):
    return torch.zeros(*n, dtype=torch.int32)


def test_binding_refuses_steps():
    good = (i32(4), i32(4), i32(4, 8), i32(16), i32(1), 16, 8, 5)
    _raises(zn.kv_extend, *good, match=ON_CPU)
    done = torch.zeros(4, dtype=torch.bool)
    _raises(zn.kv_release, i32(4), done, i32(4, 8), i32(16), i32(1), 16, match=ON_CPU)
    assert zn._kv_table("t", i32(4, 8), 4) == (8, 8) and zn._kv_table("t", i32(4, 8)[:, :5], 4) == (8, 5)
    assert zn._kv_table("t", i32(1, 8), 1) == (8, 8)
    for bad in (i32(4, 8).long(), i32(3, 8), i32(32), i32(8, 4).t(), i32(1, 8).expand(4, 8)):
        _raises(zn._kv_table, "t", bad, 4)
    for bad in (i32(4).long(), i32(5), i32(8)[::2], i32(4, 1)):
        _raises(zn._kv_ints, "t", "x", bad, (4,))
    for bad in (0, 24, 131072):
        _raises(zn._kv_page, "t", bad)


def test_binding_refuses_rows_and_queries():
    x = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    c = zn.mx_kv_cache(6, 2, 16, 64, device="cpu")
    _raises(zn.mx_kv_write, x, x, c, i32(5), match=ON_CPU)
    _raises(zn.mx_kv_write, x.half(), x, c, i32(5), match="wanted bfloat16")
    _raises(zn.mx_kv_read, c, i32(5), match=ON_CPU)
    rows = zn._kv_rows
    assert rows("t", "x", x, (5, 2, 64), x.dtype) == (128, 64)
    assert rows("t", "x", x.transpose(0, 1).contiguous().transpose(0, 1), (5, 2, 64), x.dtype) == (64, 320)
    assert rows("t", "x", x[:1].expand(5, 2, 64), (5, 2, 64), x.dtype) == (0, 64)
    for bad in (x.float(), x[:4], x[..., :32], torch.zeros(5, 64, 2, dtype=x.dtype).transpose(1, 2)):
        _raises(rows, "t", "x", bad, (5, 2, 64), x.dtype)
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    _raises(zn.mx_attention, q, c, i32(5, 4), i32(5), match=ON_CPU)
    _raises(zn.mx_attention, q.half(), c, i32(5, 4), i32(5), match="wanted bfloat16")
    g = q.clone().requires_grad_()
    _raises(zn.mx_attention, g, c, i32(5, 4), i32(5), match="requires a gradient")
    _raises(zn.mx_attention, q, c, i32(5, 4), i32(5), out=g, match="requires a gradient")
    with torch.no_grad():
        _raises(zn.mx_attention, g, c, i32(5, 4), i32(5), match=ON_CPU)
