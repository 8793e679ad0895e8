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
