"""The microscaled oracle against values worked by hand, torch's own E4M3
cast, and brute force over the grid."""
import numpy as np
import pytest
import torch

from oracle import mx


def test_grids():
    g4 = mx.grid(mx.FP4)
    assert list(g4[:8]) == [0, 0.5, 1, 1.5, 2, 3, 4, 6] and list(g4[8:]) == [0, -0.5, -1, -1.5, -2, -3, -4, -6]
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64).numpy()
    np.testing.assert_array_equal(mx.grid(mx.FP8), want)


@pytest.mark.parametrize("fmt", [mx.FP8, mx.FP4])
def test_nearest_is_nearest_with_ties_to_even(fmt):
    g = mx.grid(fmt)[:127 if fmt == mx.FP8 else 8]
    mids = (g[1:] + g[:-1]) / 2
    for i, m in enumerate(mids):
        even = i if i % 2 == 0 else i + 1
        got = mx.nearest(np.array([m, m * (1 + 1e-12), m * (1 - 1e-12), -m]), fmt)
        assert list(got) == [even, i + 1, i, even + (0x80 if fmt == mx.FP8 else 8)]
    assert list(mx.nearest(np.array([0.0, -0.0, 1e9, -1e9]), fmt)) == (
        [0, 0x80, 0x7E, 0xFE] if fmt == mx.FP8 else [0, 8, 7, 15])
    rng = np.random.default_rng(1)
    v = rng.uniform(-1, 1, 2000) * g[-1]
    d = np.abs(np.abs(v)[:, None] - g[None, :])
    np.testing.assert_array_equal(np.abs(mx.grid(fmt)[mx.nearest(v, fmt)]), g[d.argmin(1)])


def test_scale_bytes_of_known_maxima():
    def s(top, fmt):
        x = np.zeros((1, 32))
        x[0, 5] = top
        return int(mx.scale_bytes(mx.blocks(x), fmt)[0, 0])
    assert s(1.0, mx.FP8) == 119 and s(-1.99, mx.FP8) == 119 and s(2.0, mx.FP8) == 120
    assert s(1.0, mx.FP4) == 125 and s(6.0, mx.FP4) == 127 and s(7.9, mx.FP4) == 127
    assert s(0.0, mx.FP8) == 0 and s(2.0 ** -140, mx.FP4) == 0 and s(2.0 ** -126, mx.FP4) == 0
    assert s(2.0 ** -124, mx.FP4) == 1 and s(2.0 ** 127, mx.FP4) == 252 and s(2.0 ** 127, mx.FP8) == 246
    assert s(np.inf, mx.FP8) == 255 and s(np.nan, mx.FP4) == 255


@pytest.mark.parametrize("fmt", [mx.FP8, mx.FP4])
@pytest.mark.parametrize("k", [1, 31, 32, 33, 95])
def test_round_trip_stays_within_half_a_step(fmt, k):
    # a block's largest step is that of its top binade: 2^(emax - fraction bits) scales
    rng = np.random.default_rng(k)
    x = rng.normal(0, 1, (7, k)) * np.exp2(rng.integers(-20, 20, (7, 1)))
    x[2] = 0
    c, s = mx.quantize(x, fmt)
    nb = -(-k // 32)
    assert c.shape == (7, nb * (32 if fmt == mx.FP8 else 16)) and s.shape == (7, nb)
    y = mx.values(c, s, fmt)
    assert (y[:, k:] == 0).all()
    scale = np.repeat(mx.scale_value(s), 32, 1)[:, :k]
    top = 448 if fmt == mx.FP8 else 6
    step = 32 if fmt == mx.FP8 else 2
    inside = np.abs(x) <= top * scale
    assert (np.abs(y[:, :k] - x)[inside] <= (step / 2 * scale)[inside]).all()
    assert (np.abs(y[:, :k])[~inside] == (top * scale)[~inside]).all()


def test_blocks_with_infinities_and_nans_read_back_as_nans():
    x = np.ones((1, 64))
    x[0, 40] = np.inf
    c, s = mx.quantize(x, mx.FP8)
    assert list(s[0]) == [119, 255] and (c[0, 32:] == 0).all()
    y = mx.values(c, s, mx.FP8)
    assert (y[0, :32] == 1).all() and np.isnan(y[0, 32:]).all()
