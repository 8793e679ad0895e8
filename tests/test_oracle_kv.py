"""The 64-bit oracle of the key-value cache against worked examples and dense formulas."""
import numpy as np
import torch

from oracle import kv, mx


def test_extend_worked_example():
    # pages of 4; request 0 fills its page, 1 is new, 2 does not fit its two columns, 3 has no page left, 4 needs none
    table = [[7, -1, -1], [-1, -1, -1], [5, 6, 8], [9, -1, -1], [4, -1, -1]]
    got = kv.extend([3, 0, 12, 4, 1], [2, 5, 1, 1, 2], table, [1, 2, 3], 3, 4, 10, 11)
    assert got[0] == [5, 5, 12, 4, 3]
    assert got[1] == [0, 2, 7, 8, 9, 11]
    assert got[2] == [7 * 4 + 3, 3 * 4, 2 * 4, 2 * 4 + 1, 2 * 4 + 2, 2 * 4 + 3, 1 * 4, -1, -1, 17, 18]
    assert got[3] == [3, 4, 0, 1, 2, 3, 4, 0, 0, 1, 2]
    assert got[4] == 0
    assert got[5] == [[7, 3, -1], [2, 1, -1], [5, 6, 8], [9, -1, -1], [4, -1, -1]]


def test_release_worked_example():
    table = [[7, 1, 2], [3, 4, 5], [6, 8, 9]]
    assert kv.release([5, 9, 4], [True, False, True], table, [0, -1, -1, -1], 1, 4) == ([0, 9, 0], [0, 7, 1, 6], 4)
    assert kv.release([5, 9, 4], [False, True, True], table, [0, -1, -1], 1, 4) == ([5, 0, 0], [0, 3, 4], 3)


def test_what_is_released_can_be_taken_again():
    lens, free, left = kv.release([5, 9], [True, False], [[7, 1, 0], [3, 4, 5]], [0] * 6, 0, 4)
    got = kv.extend(lens, [0, 4], [[7, 1, 0], [3, 4, 5]], free, left, 4, 8, 4)
    assert got[0] == [0, 9] and got[4] == 2                      # three columns hold 12 tokens, 13 do not fit
    got = kv.extend(lens, [8, 3], [[7, 1, 0], [3, 4, 5]], free, left, 4, 8, 11)
    assert got[0] == [8, 12] and got[4] == 0 and got[5][0][:2] == [1, 7]


def test_attention_equals_a_dense_softmax():
    rng = np.random.default_rng(0)
    lens, starts, page, dim = [9, 0, 40, 17], [0, 3, 3, 8, 9], 16, 32
    k, v = rng.normal(size=(2, 8, 2, page, dim))
    table = [[5, 1, 0], [2, 2, 2], [3, 0, 7], [6, 4, 1]]
    q = rng.normal(size=(9, 4, dim))
    for causal, window in ((True, 0), (True, 5), (False, 0)):
        out, lse, size = kv.attention(q, k, v, table, lens, starts, page, causal, window)
        for b, n in enumerate(lens):
            m = starts[b + 1] - starts[b]
            if not m:
                continue
            x = torch.from_numpy(q[starts[b]:starts[b + 1]]).transpose(0, 1)                     # [heads, m, dim]
            kk, vv = (torch.from_numpy(a[table[b]].transpose(1, 0, 2, 3).reshape(2, -1, dim)[:, :n].repeat(2, 0).copy())
                      for a in (k, v))
            s = x @ kk.transpose(1, 2) / dim ** 0.5
            i, j = torch.arange(n - m, n).view(-1, 1), torch.arange(n)
            hide = (j > i) | ((j <= i - window) if window else (j < 0)) if causal else (j < 0).expand(m, n)
            s = s.masked_fill(hide, -torch.inf)
            # sums of at most 40 products under 4, in any order: 40 * 4 * 2^-53
            np.testing.assert_allclose(out[starts[b]:starts[b + 1]], (s.softmax(-1) @ vv).transpose(0, 1), rtol=1e-12, atol=2e-14)
            np.testing.assert_allclose(lse[starts[b]:starts[b + 1]], s.logsumexp(-1).t(), rtol=1e-12)
    assert (size >= np.abs(out) * (1 - 1e-12)).all()


def test_attention_of_queries_without_keys():
    k = v = np.ones((2, 1, 16, 32))
    out, lse, _ = kv.attention(np.ones((4, 1, 32)), k, v, [[0], [1]], [0, 2], [0, 1, 4], 16)
    assert (out[:2] == 0).all() and (out[2:] == 1).all()
    assert (lse[:2] == -np.inf).all() and np.isfinite(lse[2:]).all()


def test_values_of_scale_bytes():
    codes = np.full((1, 16), 0x22, np.uint8)
    for s, want in ((0, 2.0 ** -127), (127, 1.0), (252, 2.0 ** 125), (253, np.nan), (255, np.nan)):
        np.testing.assert_array_equal(kv.values(codes, np.array([[s]], np.uint8)), np.full((1, 32), want))
    x = np.random.default_rng(1).normal(size=(3, 2, 64))
    codes, scales = kv.rows(x)
    np.testing.assert_array_equal(kv.values(codes, scales).reshape(6, 64),
                                  mx.values(*mx.quantize(x.reshape(6, 64), mx.FP4), mx.FP4))
