"""Attention where its numbers end: queries, scores, starts and sizes at their limits, by every kernel."""
import numpy as np
import pytest
import torch

from kv_kernels import KINDS, attention_by
from kv_util import check_attention, i32
from lossless_float_weight_amd import zn
from test_gpu_kv import attend_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zn.lib()


def case_for(kind, lens=(100, 45), new=(90, 45), heads=2, kv_heads=1, dim=32, t="bf16", seed=1):
    """A call that the kernel takes: more heads for two waves a workgroup."""
    if kind == "short pairs":
        heads, kv_heads = 300 * heads // kv_heads, 300
    q, c, table, starts = attend_case(list(lens), list(new), heads, kv_heads, dim, 16, t, seed)
    return q, c, table, list(lens), starts


def call(kind, q, c, table, lens, starts, **kw):
    return attention_by(kind)(q, c, i32(table.tolist()), i32(lens), None if starts is None else i32(starts), **kw)


@pytest.mark.parametrize("kind", KINDS)
def test_queries_to_the_end_of_fp32(kind):
    # from 2^128 (1 - 2^-9) on a value rounds to infinity in BF16; with keys near 2^-126 scores are a few units
    q, c, table, lens, starts = case_for(kind, t="fp32")
    g = torch.Generator().manual_seed(5)
    far = 2.0 ** 128 * (1 - 2.0 ** -24) * (1 - 2.0 ** -8 * torch.rand(q.shape, generator=g, dtype=torch.float64))
    sign = torch.randint(0, 2, q.shape, generator=g) * 2 - 1
    q.copy_((far * sign).float())
    q[1] = torch.finfo(torch.float32).max
    c.k_scales.view(torch.uint8).fill_(1)                          # 2^-126
    out, lse = call(kind, q, c, table, lens, starts, lse=True)
    assert out.isfinite().all() and lse.isfinite().all()
    check_attention(q, c, table, lens, starts, 16, out, lse)
    c.k.zero_()                                                    # keys of 0: means of the values
    out = call(kind, q, c, table, lens, starts)
    check_attention(q, c, table, lens, starts, 16, out)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_infinite_and_nan_queries_stay_by_themselves(kind, t):
    q, c, table, lens, starts = case_for(kind, t=t)
    want = call(kind, q, c, table, lens, starts)
    q[2, 1, 5], q[97, 0, 0], q[40, 1, 31] = float("nan"), float("inf"), -float("inf")
    gone = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    gone[2, 1] = gone[97, 0] = gone[40, 1] = True
    out = call(kind, q, c, table, lens, starts)
    assert torch.equal(out[~gone], want[~gone]) and out[gone].isnan().all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [float("inf"), 3e38])
def test_scores_of_minus_infinity_alone_are_nan(kind, t, value):
    # every key is negative where the query is infinite, or so large that the product passes FP32's range
    q, c, table, lens, starts = case_for(kind, t=t)
    want, want_lse = call(kind, q, c, table, lens, starts, lse=True)
    c.k[..., 0] = 0xFF                                             # -6, -6
    c.k_scales.view(torch.uint8)[..., 0] = 130
    want, want_lse = call(kind, q, c, table, lens, starts, lse=True)
    gone = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    for row, head in ((0, 0), (3, 1), (89, 0), (90, 1), (134, 0)):
        q[row, head, :2] = value
        gone[row, head] = True
    out, lse = call(kind, q, c, table, lens, starts, lse=True)
    assert out[gone].isnan().all() and lse[gone].isnan().all()
    assert torch.equal(out[~gone], want[~gone]) and torch.equal(lse[~gone], want_lse[~gone])
    # a key that is not: it has all the weight
    keep = table[0][5 // 16], 5 % 16
    c.k[keep[0], :, keep[1], 0] = 0
    out, lse = call(kind, q, c, table, lens, starts, lse=True)
    rows = torch.tensor([3, 89], device="cuda") if value < 1e39 else torch.tensor([], dtype=torch.long, device="cuda")
    for row in rows.tolist():
        head = 1 if row == 3 else 0
        v = zn.mx_kv_read(c, i32([int(keep[0]) * 16 + keep[1]]), dtype=torch.float32)[1][0]
        assert torch.equal(out[row, head].float(), v[head * v.shape[0] // q.shape[1]].to(q.dtype).float())
        assert lse[row, head].isfinite()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_queries_that_see_nothing_stay_zeros(kind, t):
    # more queries than keys, an empty request, and a piece or a wave whose tiles a row does not see
    q, c, table, lens, starts = case_for(kind, lens=(70, 0, 300), new=(90, 40, 60), t=t)
    # (a window leaves few tiles, which the other kernels take)
    masks = {"few rows": (dict(window=2100),), "many rows": ()}.get(kind, (dict(window=3),))
    for kw in (dict(), *masks, dict(causal=False)):
        out, lse = call(kind, q, c, table, lens, starts, lse=True, **kw)
        nothing = torch.zeros(q.shape[0], dtype=torch.bool, device="cuda")
        nothing[90:130] = True
        nothing[:20] = kw.get("causal", True)
        assert (out[nothing] == 0).all() and (lse[nothing] == -torch.inf).all()
        assert lse[~nothing].isfinite().all()
        check_attention(q, c, table, lens, starts, 16, out, lse, **kw)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_starts_out_of_order_leave_rows_or_answer_them(kind, t):
    # requests that all name the same rows and keys, each followed by one that ends before it starts: far more groups of
    # rows than the sizes let the host expect, so that workgroups run out, of pieces among others
    n, lens, heads, kv_heads, page = (512, 3000, 16, 8, 64) if kind == "many rows" else (64, 200, 4, 2, 64)
    if kind == "short pairs":
        heads, kv_heads = 600, 300
    times = 7 if t == "fp32" else 12
    q, c, table, _ = attend_case([lens], [n], heads, kv_heads, 32, page, t, 3)
    all_lens, starts = [lens] * (2 * times), [0, n] * times + [0]
    scratch = torch.full((1 << 24,), 1e30, device="cuda").view(torch.uint8)      # no piece has such numbers
    out, lse = torch.full_like(q, 7.0), torch.full(q.shape[:2], 7.0, device="cuda")
    call(kind, q, c, np.repeat(table, 2 * times, 0), all_lens, starts, out=out, lse=lse, scratch=scratch)
    left = (out == 7).all(-1) & (lse == 7)
    want, want_lse = zn.mx_attention(q, c, i32(table.tolist()), i32([lens]), i32([0, n]), lse=True)
    got, got_lse = torch.where(left[..., None], want, out), torch.where(left, want_lse, lse)
    check_attention(q, c, table, [lens], [0, n], page, got, got_lse)
