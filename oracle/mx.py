"""Microscaled numbers in 64 bits: the oracle of the library's quantiser, norm
and product.  Plain numpy float64, no code shared with the library.

A block of 32 values of a row has one byte s; a value is code * 2^(s - 127),
s = 255 a NaN.  Formats: E4M3 (bias 7, 3 fraction bits, largest 448, one NaN
per sign at 0x7F / 0xFF) and E2M1 (bias 1, 1 fraction bit, largest 6), the
latter two to a byte, the first in the low nibble.
"""
from __future__ import annotations

import numpy as np

FP8, FP4 = "fp8", "fp4"
BLOCK = 32
EMAX = {FP8: 8, FP4: 2}


def grid(fmt: str) -> np.ndarray:
    """Values of all codes in the order of the codes."""
    bits, bias, frac = (8, 7, 3) if fmt == FP8 else (4, 1, 1)
    out = []
    for c in range(1 << bits):
        sign = -1.0 if c >> (bits - 1) else 1.0
        e = (c >> frac) & ((1 << (bits - 1 - frac)) - 1)
        f = c & ((1 << frac) - 1)
        if fmt == FP8 and (c & 0x7F) == 0x7F:
            out.append(np.nan)
        elif e == 0:
            out.append(sign * f * 2.0 ** (1 - bias - frac))
        else:
            out.append(sign * (2.0 ** frac + f) * 2.0 ** (e - bias - frac))
    return np.array(out)


def nearest(v: np.ndarray, fmt: str) -> np.ndarray:
    """Codes of finite values, to the nearest grid point, ties to the even
    code, saturating; the sign of the value also on zeros."""
    n = 127 if fmt == FP8 else 8
    g = grid(fmt)[:n]
    a = np.minimum(np.abs(v), g[-1])
    hi = np.searchsorted(g, a).clip(0, n - 1)      # first grid point >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - g[lo], g[hi] - a                  # exact: few bits each
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(a == g[hi], hi, code)
    return (code + np.where(np.signbit(v), 0x80 if fmt == FP8 else 8, 0)).astype(np.uint8)


def blocks(x: np.ndarray) -> np.ndarray:
    """[rows, k] float64 -> [rows, blocks, 32], zeros past k."""
    rows, k = x.shape
    nb = -(-k // BLOCK)
    full = np.zeros((rows, nb * BLOCK))
    full[:, :k] = x
    return full.reshape(rows, nb, BLOCK)


def scale_value(s: np.ndarray) -> np.ndarray:
    return np.where(s == 255, np.nan, np.ldexp(1.0, s.astype(np.int64) - 127))


def scale_bytes(x: np.ndarray, fmt: str) -> np.ndarray:
    """Scale byte of every block of x [rows, blocks, 32]."""
    top = np.abs(x).max(2)
    fine = np.isfinite(top)
    _, e = np.frexp(np.where(fine & (top > 0), top, 1.0))
    s = np.clip(e - 1 + 127 - EMAX[fmt], 0, 254)
    s = np.where(top == 0, 0, s)
    return np.where(fine, s, 255).astype(np.uint8)


def pack(codes: np.ndarray, fmt: str) -> np.ndarray:
    return codes if fmt == FP8 else (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(stored: np.ndarray, fmt: str) -> np.ndarray:
    if fmt == FP8:
        return stored
    return np.stack([stored & 15, stored >> 4], -1).reshape(*stored.shape[:-1], -1)


def quantize(x: np.ndarray, fmt: str):
    """[rows, k] float64 -> (stored codes, scale bytes)."""
    b = blocks(x)
    with np.errstate(invalid="ignore"):
        s = scale_bytes(b, fmt)
    live = (s != 255)[..., None]
    v = np.where(live, b, 0.0) / np.where(live, scale_value(np.where(s == 255, 127, s))[..., None], 1.0)
    c = np.where(live, nearest(v, fmt), 0).astype(np.uint8)
    return pack(c.reshape(len(x), -1), fmt), s


def values(stored: np.ndarray, s: np.ndarray, fmt: str) -> np.ndarray:
    """Stored codes [rows, ...] and scale bytes -> float64 [rows, kp]."""
    v = grid(fmt)[unpack(stored, fmt)]
    rows = len(v)
    return (v.reshape(rows, -1, BLOCK) * scale_value(s)[..., None]).reshape(rows, -1)


def rms_norm(h: np.ndarray, w: np.ndarray, eps: float) -> np.ndarray:
    with np.errstate(all="ignore"):
        return h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w


def matmul(a: np.ndarray, w: np.ndarray) -> np.ndarray:
    with np.errstate(invalid="ignore"):
        return a @ w.T
