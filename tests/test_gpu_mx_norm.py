"""The norm's second look on the GPU: signs of zeros, and rows whose product
with the weight leaves FP32's normal numbers before or after the weight.

The formula in 64 bits is compared code by code.  Where its value is no number
of the grid's middle (all cases of zeros and powers of two below) the codes are
its own, bit by bit; elsewhere `between` of the first file holds them to the
64-bit roundings, and the sign of every code to the value's.
"""
import numpy as np
import pytest
import torch

from lossless_float_weight_amd import zn
from oracle import mx
from test_gpu_mx import FMT, TYPE, between, f64, raw, rounded

pytestmark = pytest.mark.gpu

EPS = float(np.float32(1e-5))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zn.lib()


def signs(y, fmt, codes, scales):
    """Every code has its value's sign, on zeros too, except in NaN blocks."""
    c = mx.unpack(raw(codes).reshape(len(y), -1), fmt)
    live = np.repeat(raw(scales).reshape(len(y), -1) != 255, 32, 1)[:, :y.shape[1]]
    got = (c >> (7 if fmt == "fp8" else 3))[:, :y.shape[1]].astype(bool)
    assert (got == np.signbit(y))[live].all(), "signs"


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("k", [32, 96, 4096, 8224, 16416])
def test_zeros_keep_their_sign_in_blocks_in_doubt(k, t, fmt):
    # a quarter of the values is +-1: the mean of the squares is 1/4 and y +-2, a
    # maximum on a power of two, which the first look cannot tell from one below
    rng = np.random.default_rng(k)
    x = np.where(np.arange(k) % 4 == 0, 1.0, 0.0) * np.ones((3, 1))
    x = np.copysign(x, rng.choice([-1.0, 1.0], x.shape))
    xt = rounded(x, TYPE[t])
    w = rounded(np.copysign(1.0, rng.choice([-1.0, 1.0], k)), TYPE[t])
    codes, scales, _ = zn.mx_rms_norm(xt.cuda(), w.cuda(), eps=0.0, fmt=FMT[fmt])
    want, s = mx.quantize(x * 2 * f64(w), fmt)
    np.testing.assert_array_equal(raw(scales).reshape(s.shape), s)
    np.testing.assert_array_equal(raw(codes).reshape(want.shape), want)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("k", [64, 8224, 16416])
def test_values_that_round_to_zero_keep_their_sign(k, fmt):
    # rows far under sqrt(eps): y stays near x / sqrt(eps), too small for the first look
    rng = np.random.default_rng(k)
    x = rounded(rng.normal(0, 1, (6, k)) * np.exp2(rng.integers(-40, 0, (6, k)) - 105.0), torch.float32)
    x[:, ::5] = -0.0
    x[:, 1::5] = 0.0
    x[4] = -0.0
    w = rounded(np.ones(k), torch.float32)
    codes, scales, _ = zn.mx_rms_norm(x.cuda(), w.cuda(), eps=1e-5, fmt=FMT[fmt])
    y = mx.rms_norm(f64(x), f64(w), EPS)
    between(y, fmt, codes, scales)
    signs(y, fmt, codes, scales)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("k", [96, 512, 4096, 8224, 16416])
def test_weights_that_bring_tiny_values_back(k, fmt):
    # h / rms lies under FP32's normal numbers, or is zero there, and the weight makes y ordinary
    rng = np.random.default_rng(k)
    z = rng.normal(0, 1, (5, k))
    x = z * np.exp2(np.array([-50.0, -80, -100, -38, -20]))[:, None]
    x[:, 3] = 2.0 ** 100
    x[4, 3] = 2.0 ** 90
    x[:, 40:48] = -0.0
    x = rounded(x, torch.float32)
    for power in (12, 25, 60, 100):
        w = rounded((1 + 0.3 * rng.random(k)) * np.where(np.arange(k) == 3, 1.0, 2.0 ** power), torch.float32)
        codes, scales, _ = zn.mx_rms_norm(x.cuda(), w.cuda(), eps=0.0, fmt=FMT[fmt])
        y = mx.rms_norm(f64(x), f64(w), 0.0)
        between(y, fmt, codes, scales)
        signs(y, fmt, codes, scales)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("k", [64, 4096, 8224, 16416])
def test_values_past_fp32_have_finite_scales(k, fmt):
    # |y| passes 2^128: the formula's scale is finite (at most 254) and so is the block
    rng = np.random.default_rng(k)
    x = rounded(rng.normal(0, 1, (4, k)), torch.float32)
    x[1, 0] = 2.0 ** 40
    x[2] = 0.0
    x[3, k // 2] = float("inf")
    for w in (np.full(k, 2.0 ** 127), rng.normal(0, 1, k) * 2.0 ** 126):
        w = rounded(w, torch.float32)
        codes, scales, _ = zn.mx_rms_norm(x.cuda(), w.cuda(), eps=1e-5, fmt=FMT[fmt])
        y = mx.rms_norm(f64(x), f64(w), EPS)
        assert np.abs(y[0]).max() > 2.0 ** 128
        between(y, fmt, codes, scales)
        signs(y, fmt, codes, scales)
        # normal numbers past 4 are no FP32 weights any more: infinities, whose blocks are NaNs
        dead = ~np.isfinite(mx.blocks(f64(w)[None])).all(2)[0]
        assert ((raw(scales)[:3] == 255) == dead).all()
    # an infinite weight is one, and a NaN is one
    w[k // 3], w[k - 1] = float("inf"), float("nan")
    codes, scales, _ = zn.mx_rms_norm(x.cuda(), w.cuda(), eps=1e-5, fmt=FMT[fmt])
    assert (raw(scales)[:, k // 3 // 32] == 255).all() and (raw(scales)[:, -1] == 255).all()
