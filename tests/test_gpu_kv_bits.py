"""The bits that attention's weights and queries keep, in sums that cancel.

Two keys count, with values 1 and -1, at positions of different tiles: A with the
score 0 (or s) and B with one lower by d.  All others have weights under 2^-700, which
are 0.  With w = 2^-d the result is (1 - w) / (1 + w), so an error of e in a weight
shows as e / 2 beside a result that may be far smaller.

Bound.  The sums have two terms that are not 0, so the additions are exact but one
each (2^-24 of at most 2); w is off by
  * its exponent's rounding, the weights' being 2^(c (s - m) - 8): half a step of a
    number under 16, 2^-21 ln 2 of w, and c (scale log2 e) and its product with the
    difference, 2 * 2^-24 d;
  * the exponential, 2^-22;
  * its own bits, 2^-17 beside BF16 queries (2^-11 where fast weights are asked for, half a
    step of FP16), 2^-24 beside FP32;
for both keys, each of which has half of the sum of weights; the division adds
2^-22, and the result half a step of its type."""
import numpy as np
import pytest
import torch

import test_gpu_kv as gpu
from kv_util import TYPE, f64, i32
from lossless_float_weight_amd import zn

LN2 = float(np.float32(np.log(2.0)))


def bound(d, want, t, bits):
    w = 2.0 ** -21 * np.log(2) + 2 * 2.0 ** -24 * d + 2.0 ** -22 + 2.0 ** -bits
    return w + 2 * 2.0 ** -24 + 2.0 ** -22 + torch.finfo(TYPE[t]).eps / 2 * np.abs(want)


def differences(n, t, seed=3):
    """n differences of scores from 2^-14 to 4."""
    g = torch.Generator().manual_seed(seed)
    return torch.exp2(torch.rand(n, generator=g, dtype=torch.float64) * 16 - 14).to(TYPE[t])


def pair_cache(n, at_a, at_b, dim, block, apart=False):
    """(k, v) codes and scales of n keys: in a block of 32 places A's key is 0, B's -1 in place 0, the others' -768 in
    place 1.  apart: A's is 1 in place 0, B's 1 in place 2."""
    k = torch.zeros(n, dim // 2, dtype=torch.uint8)
    ks = torch.full((n, dim // 32), 127, dtype=torch.uint8)
    v = torch.full((n, dim // 2), 0x77, dtype=torch.uint8)   # 6 where nothing should count
    vs = torch.full((n, dim // 32), 127, dtype=torch.uint8)
    at = 16 * block
    k[:, at] = 0xF0                                           # -6 in place 1
    ks[:, block] = 134
    k[at_a], ks[at_a], v[at_a] = 0, 127, 0x22                 # 1
    k[at_b], ks[at_b], v[at_b] = 0, 127, 0xAA                 # -1
    if apart:
        k[at_a, at], k[at_b, at + 1] = 0x02, 0x02
    else:
        k[at_b, at] = 0x0A                                    # -1 in place 0
    return k, ks, v, vs


def rounded(w, pieces):
    """w as the sum of so many BF16 numbers; 0: as FP16 times a power of two."""
    if pieces == 0:
        return (w * 2.0 ** 7).half().double() / 2.0 ** 7
    rest, out = w.clone(), torch.zeros_like(w)
    for _ in range(pieces):
        p = rest.bfloat16().double()
        out, rest = out + p, rest - p
    return out


@pytest.mark.parametrize("t,bits,enough,few", [("bf16", 17, 2, 1), ("bf16", 17, 2, 0), ("bf16", 11, 0, 1), ("fp32", 24, 3, 2)])
def test_the_bound_tells_pieces_apart(t, bits, enough, few):
    # the plain formula with weights rounded so: within the bound with enough pieces, out of it with one less
    d = differences(400, t).double()
    w = torch.exp2(-d)
    want = ((1 - w) / (1 + w)).numpy()
    off = {p: np.abs(((1 - rounded(w, p)) / (1 + w)).to(TYPE[t]).double().numpy() - want) for p in (enough, few)}
    b = bound(d.numpy(), want, t, bits)
    assert (off[enough] <= b).all() and (off[few] > b).sum() > 20


def large_pairs(n):
    """(s, s - d) for queries: s from 20 to 32 in 24 bits, and d from 2^-14 to 4 as FP32 has it."""
    s = (20 + 12 * torch.rand(n, generator=torch.Generator().manual_seed(8), dtype=torch.float64)).float()
    return s, (s.double() - differences(n, "fp32").double()).float()


def large_bound(d, want):
    """Scores of 32 on top: three pieces' products add to them exactly or within a half step each, 2 * 2^-24 * 32 a score."""
    return bound(d, want, "fp32", 24) + 2 * 2.0 ** -24 * 32 * np.log(2)


def test_the_bound_tells_pieces_of_queries_apart():
    s, less = large_pairs(400)
    d = s.double() - less.double()
    want = np.tanh(d.numpy() * np.log(2) / 2)
    off = {p: np.abs(np.tanh((rounded(s.double(), p) - rounded(less.double(), p)).numpy() * np.log(2) / 2) - want) for p in (3, 2)}
    b = large_bound(d.numpy(), want)
    assert (off[3] <= b).all() and (off[2] > b).sum() > 20


def run_pairs(t, kind, n, page, at_a, at_b, dim=32, block=0, large=False, **kw):
    """(d, result) of 160 queries over n keys, by the kernel that `kind` names."""
    rows = 160
    codes = pair_cache(n, at_a, at_b, dim, block, large)
    n_pages = -(-n // page)
    c = zn.mx_kv_cache(n_pages, 1, page, dim)
    for to, x in zip(c, codes):
        to.view(torch.uint8).view(n_pages * page, -1)[:n] = x.cuda()
    d = differences(rows, t)
    q = torch.zeros(rows, 1, dim, dtype=TYPE[t])
    q[:, 0, 32 * block] = d
    q[:, 0, 32 * block + 1] = 1
    if large:
        q[:, 0, 32 * block], q[:, 0, 32 * block + 2] = large_pairs(rows)
        d = q[:, 0, 32 * block].double() - q[:, 0, 32 * block + 2].double()
    # the kernel goes by the sizes that the host sees: one with many queries, the hint of one, the table's width
    tiles = {"short": n_pages * page // 64, "few": 3000, "many": 20480}[kind]
    width = max(n_pages, tiles * 64 // page)
    table = torch.full((1, width), -1, dtype=torch.int32)
    table[0, :n_pages] = torch.arange(n_pages)
    hint = rows if kind == "many" else 1
    args = (q.cuda(), c, table.cuda(), i32([n]), i32([0, rows]))
    assert zn.debug_attention_kernel(args[0], c, args[2], args[4], hint).startswith(kind)
    out = zn.mx_attention(*args, max_new=hint, causal=False, scale=LN2, **kw)
    return f64(d), f64(out)


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["short", "few", "many"])
@pytest.mark.parametrize("n,at_a,at_b", [(2, 0, 1), (2, 1, 0), (64, 63, 0), (200, 3, 150)])
def test_weights_keep_their_bits(n, at_a, at_b, kind, t):
    d, out = run_pairs(t, kind, n, 64, at_a, at_b)
    want = np.tanh(d * np.log(2) / 2)[:, None, None]
    b = bound(d[:, None, None], want, t, 17 if t == "bf16" else 24)
    worst = (np.abs(out - want) / b).max()
    assert worst <= 1


@pytest.mark.gpu
@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["short", "few", "many"])
@pytest.mark.parametrize("dim,block", [(64, 1), (96, 0), (96, 2), (128, 3), (160, 4), (192, 1), (224, 6), (256, 7)])
def test_weights_keep_their_bits_in_every_head_size(dim, block, kind, t):
    d, out = run_pairs(t, kind, 130, 64, 100, 20, dim, block)
    want = np.tanh(d * np.log(2) / 2)[:, None, None]
    worst = (np.abs(out - want) / bound(d[:, None, None], want, t, 17 if t == "bf16" else 24)).max()
    assert worst <= 1


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["short", "few", "many"])
@pytest.mark.parametrize("dim,block", [(32, 0), (64, 0), (96, 1), (128, 2), (160, 4), (192, 5), (224, 3), (256, 6)])
def test_queries_keep_their_bits(dim, block, kind):
    d, out = run_pairs("fp32", kind, 130, 64, 20, 100, dim, block, large=True)
    want = np.tanh(d * np.log(2) / 2)[:, None, None]
    worst = (np.abs(out - want) / large_bound(d[:, None, None], want)).max()
    assert worst <= 1


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["short", "few", "many"])
@pytest.mark.parametrize("n,at_a,at_b", [(2, 0, 1), (64, 63, 0), (200, 3, 150)])
def test_fast_weights_keep_11_bits(n, at_a, at_b, kind):
    d, out = run_pairs("bf16", kind, n, 64, at_a, at_b, fast_weights=True)
    want = np.tanh(d * np.log(2) / 2)[:, None, None]
    worst = (np.abs(out - want) / bound(d[:, None, None], want, "bf16", 11)).max()
    assert worst <= 1
    # few rows a request keep theirs, and so does a call whose rows the host takes for few
    if kind != "many":
        assert np.array_equal(out, run_pairs("bf16", kind, n, 64, at_a, at_b)[1])


@pytest.mark.gpu
@pytest.mark.parametrize("test,args", [
    *((gpu.test_attention_of_several_queries, (lens, new, m, "bf16")) for lens, new, m in (
        ([300, 0, 20], [129, 0, 1], dict(causal=False)), ([700], [700], dict(window=50)), ([65, 64, 63, 130], [2, 64, 63, 100], {}))),
    (gpu.test_attention_of_long_caches, ([9000, 4000], [20, 100], {}, "bf16")),
    *((gpu.test_attention_of_many_rows, ([700, 150, 0], [300, 150, 0], d)) for d in (32, 64, 96, 128, 160, 192, 224, 256)),
    *((gpu.test_scores_past_the_weights_precision, (lens, new, "bf16")) for lens, new in (([3000], [40]), ([300], [200]))),
    (gpu.test_what_a_query_does_not_see_has_no_effect, ("bf16",)),
    *((gpu.test_values_of_many_sizes, (k,)) for k in ("near", "less near", "far", "rising", "zeros first", "one far block",
                                                      "far where nobody looks")),
    (gpu.test_small_values_beside_large_ones_keep_their_bits, ()), (gpu.test_many_small_weights_add_up, (100,)),
    (gpu.test_nans_among_the_largest_values, ()), (gpu.test_kernels_of_many_rows_captured_and_replayed, ())],
    ids=lambda x: x.__name__[5:] if callable(x) else "-".join(str(i).replace(" ", "") for i in x) if isinstance(x, tuple) else x)
def test_fast_weights(test, args, monkeypatch):
    attention = gpu.by_sizes("many")
    monkeypatch.setattr(zn, "mx_attention", lambda *a, **kw: attention(*a, **dict(kw, fast_weights=True)))
    test(*args)


@pytest.mark.gpu
@pytest.mark.parametrize("t,bits", [("bf16", 17), ("fp32", 24), ("bf16", 11)])
@pytest.mark.parametrize("kind", ["short", "few", "many"])
@pytest.mark.parametrize("n,at_a,at_b", [(200, 199, 64), (200, 64, 199), (320, 130, 300), (256, 255, 128)])
def test_keys_far_below_leave_no_rounding(n, at_a, at_b, kind, t, bits):
    # tiles whose scores are all around -768 come first: what follows them is not rounded at their size
    d, out = run_pairs(t, kind, n, 64, at_a, at_b, **(dict(fast_weights=True) if bits == 11 else {}))
    want = np.tanh(d * np.log(2) / 2)[:, None, None]
    worst = (np.abs(out - want) / bound(d[:, None, None], want, t, bits)).max()
    assert worst <= 1
