"""What the tests of the key-value cache share: caches, their values in 64 bits, and the bound on attention."""
import numpy as np
import torch

from lossless_float_weight_amd import zn
from oracle import kv

TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def f64(t):
    return t.to(torch.float64).cpu().numpy()


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def random_cache(n_pages, heads, page, dim, seed, strides="pages", spread=2):
    """A cache full of random codes, the scales of each block its own."""
    g = torch.Generator().manual_seed(seed)
    if strides == "pages":
        c = zn.mx_kv_cache(n_pages, heads, page, dim)
    elif strides == "beside":     # keys and values of a page beside each other
        both = [torch.zeros(n_pages, 2, heads, page, n, dtype=torch.uint8, device="cuda") for n in (dim // 2, dim // 32)]
        c = zn.MxCache(both[0][:, 0], both[1][:, 0], both[0][:, 1], both[1][:, 1])
    else:                         # heads of a token beside each other, one of several layers
        four = [torch.zeros(n_pages, page, 3, heads, n, dtype=torch.uint8, device="cuda")[:, :, 1].transpose(1, 2)
                for n in (dim // 2, dim // 32) * 2]
        c = zn.MxCache(*four)
    for codes, scales in ((c.k, c.k_scales), (c.v, c.v_scales)):
        codes.copy_(torch.randint(0, 256, codes.shape, generator=g, dtype=torch.uint8))
        scales.view(torch.uint8).copy_(torch.randint(126 - spread, 127 + spread, scales.shape, generator=g, dtype=torch.uint8))
    return c


def values(c):
    """Keys and values of a cache in 64 bits: [pages, heads, page, dim] each."""
    return [kv.values(raw(a), raw(b)) for a, b in ((c.k, c.k_scales), (c.v, c.v_scales))]


def dealt(lens, page, n_pages, width, seed):
    """A table with random pages; behind a request's length pages of others."""
    rng = np.random.default_rng(seed)
    order = rng.permutation(n_pages)
    table = rng.integers(0, n_pages, (len(lens), width))
    at = 0
    for b, n in enumerate(lens):
        m = -(-n // page)
        table[b, :m] = order[at:at + m]
        at += m
    assert at <= n_pages
    return table


def check_attention(q, c, table, lens, starts, page, got, got_lse=None, causal=True, window=0, scale=None):
    """Against the oracle.  With weights w_j of relative error d the result is off by
    2 d sum w|v| / sum w; d has
      * the score: dim FP32 additions, each within 2^-23 of a partial sum of
        scale |q|.|k|, and three roundings (scale, its product with log2 e, the
        multiply-add) within 2^-24 of at most that sum and the largest score's;
      * the exponential, 2^-22, and the weight's bits: beside BF16 queries 2^-11
        (FP16, or two BF16 pieces, 2^-17), 2^-24 beside FP32;
    the sums over n keys add n 2^-23 each, joining pieces and dividing 8 roundings
    of 2^-24, and the result half a step of its type.  What FP32 cannot hold: a
    weight under 2^-126 may vanish, whole or in its last piece, the largest being at
    least 2^-8, so n 2^-118 max|v| are added for sum w|v| and as much for the sum of
    weights; an FP16 weight under 2^-14 is off by up to 2^-25 where the row's largest
    is 2^7 or more, n 2^-32 max|v| in all; the result's step is at least 2^-133; and sums past FP32's range, which
    weights up to 1 reach where n max|v| does, give infinities and NaNs."""
    k, v = values(c)
    x = f64(q)
    out, lse, size = kv.attention(x, k, v, table, lens, starts, page, causal, window, scale)
    dim = x.shape[2]
    sc = 1 / np.sqrt(dim) if scale is None else scale
    top = sc * np.abs(x).sum(2) * np.nanmax(np.abs(k))         # at least scale |q|.|k| of any key
    d = top * (dim * 2.0 ** -23 + 6 * 2.0 ** -24) + 2.0 ** -22 + (2.0 ** -11 if q.dtype == torch.bfloat16 else 2.0 ** -24)
    n = max(max(lens), 1)
    mine = (size != -1)                                        # rows that some request has
    bound = (2 * d[..., None] + 2 * n * 2.0 ** -23 + 8 * 2.0 ** -24) * size + torch.finfo(q.dtype).eps / 2 * np.abs(out)
    least = 2.0 ** -32 if q.dtype == torch.bfloat16 else 2.0 ** -118
    bound = bound + 2 * n * least * np.nanmax(np.abs(v), (0, 1, 2)) + 2.0 ** -134      # of the result's own column
    y = f64(got)
    nan = np.isnan(out)
    if n * np.nanmax(np.abs(v)) >= 2.0 ** 127:
        mine = mine & np.isfinite(y)
    assert (np.isnan(y) == nan)[mine].all(), "NaNs differ"
    ok = mine & ~nan
    assert (np.abs(y - out) <= bound)[ok].all(), np.abs((y - out) / np.maximum(bound, 1e-300))[ok].max()
    if got_lse is not None:
        z = f64(got_lse)
        rows = mine[..., 0]
        gone = rows & np.isnan(lse)
        assert np.isnan(z[gone]).all()
        rows = rows & ~np.isnan(lse)
        assert (z[rows & np.isinf(lse)] == -np.inf).all()
        rows = rows & np.isfinite(lse)
        slack = d + n * 2.0 ** -23 + 4 * 2.0 ** -24 * (1 + np.abs(np.where(rows, lse, 0)))
        assert (np.abs(z[rows] - lse[rows]) <= slack[rows]).all()
    return y
