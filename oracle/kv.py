"""The key-value cache in 4 bits in 64 bits: the oracle of the library's block
tables, its cache rows and its attention.  Plain Python and numpy float64, one
request, token and row after the other; no code shared with the library.
"""
from __future__ import annotations

import numpy as np

from . import mx


def pages_of(n: int, page: int) -> int:
    return -(-n // page)


def release(lens, done, table, free, n_free, page):
    """(lens, free, n_free) after the pages of requests that are done came back."""
    free, stack = list(free), max(0, min(n_free, len(free)))
    out = []
    for n, d, row in zip(lens, done, table):
        n = max(0, n)
        if d:
            for p in row[:pages_of(n, page)]:
                if stack < len(free):
                    free[stack] = p
                    stack += 1
            n = 0
        out.append(n)
    return out, free, stack


def extend(lens, add, table, free, n_free, page, n_pages, tokens):
    """(lens, starts, slots, positions, n_free, table) after a step."""
    table = [list(r) for r in table]
    width = len(table[0]) if table else 0
    stack = max(0, min(n_free, len(free)))
    asked = 0               # pages that the requests so far need, served or not
    taken = 0
    starts, out = [0], []
    slots, positions = [-1] * tokens, [0] * tokens
    for row, n, a in zip(table, lens, add):
        n, a = max(0, n), max(0, a)
        begin, end = starts[-1], starts[-1] + a
        starts.append(end)
        have, want = pages_of(n, page), pages_of(n + a, page)
        fits = want <= width and end <= tokens
        need = want - have if fits else 0
        asked += need
        if not fits or (need and asked > stack):
            out.append(n)
            continue
        for i in range(have, want):
            taken += 1
            row[i] = free[stack - taken]
        for i in range(a):
            p = row[(n + i) // page]
            positions[begin + i] = n + i
            if 0 <= p < n_pages:
                slots[begin + i] = p * page + (n + i) % page
        out.append(n + a)
    return out, [min(s, 2 ** 31 - 1) for s in starts], slots, positions, stack - taken, table


def rows(x: np.ndarray):
    """[tokens, heads, dim] float64 -> the values that its rows have in 4 bits."""
    t, h, d = x.shape
    codes, s = mx.quantize(x.reshape(-1, d), mx.FP4)
    return codes.reshape(t, h, -1), s.reshape(t, h, -1)


def values(codes: np.ndarray, scales: np.ndarray) -> np.ndarray:
    """Codes [..., dim / 2] and scale bytes [..., dim / 32] as float64; bytes over 252 are NaNs."""
    s = np.where(scales > 252, 255, scales)
    d = codes.shape[-1]
    return mx.values(codes.reshape(-1, d), s.reshape(-1, d // 16), mx.FP4).reshape(*codes.shape[:-1], 2 * d)


def attention(q, k, v, table, lens, starts, page, causal=True, window=0, scale=None):
    """(out, lse, magnitude) of q [tokens, heads, dim] over k, v [pages, kv heads,
    page, dim]; magnitude is the same sum over |v|, which bounds its roundings.
    Rows that no request has are NaN with magnitude -1."""
    tokens, heads, dim = q.shape
    group = heads // k.shape[1]
    scale = 1 / np.sqrt(dim) if scale is None else scale
    out = np.full(q.shape, np.nan)
    lse = np.full(q.shape[:2], np.nan)
    size = np.full(q.shape, -1.0)
    for b, n in enumerate(lens):
        first, end = (b, b + 1) if starts is None else (starts[b], starts[b + 1])
        at = np.arange(n)
        pages = np.asarray(table[b], dtype=np.int64)[at // page] if n else np.zeros(0, np.int64)
        good = (pages >= 0) & (pages < k.shape[0])
        safe = np.where(good, pages, 0)
        for h in range(heads):
            kk, vv = (np.where(good[:, None], x[safe, h // group, at % page], np.nan) for x in (k, v))
            for t in range(first, end):
                p = n - (end - first) + t - first
                hi = p + 1 if causal else n
                lo = max(0, hi - window) if window else 0
                if hi <= lo:
                    out[t, h], lse[t, h], size[t, h] = 0, -np.inf, 0
                    continue
                with np.errstate(all="ignore"):
                    s = scale * (kk[lo:hi] @ q[t, h])
                    top = s.max()
                    w = np.exp(s - top)
                    out[t, h] = w @ vv[lo:hi] / w.sum()
                    size[t, h] = w @ np.abs(vv[lo:hi]) / w.sum()
                    lse[t, h] = top + np.log(w.sum())
    return out, lse, size
