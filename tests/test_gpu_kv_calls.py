"""Calls of the key-value cache as a program mixes them with its own work: results that autograd may use, refusals."""
import numpy as np
import pytest
import torch

from kv_kernels import KINDS, attention_by, widened
from kv_util import check_attention, dealt, f64, i32, random_cache, values
from lossless_float_weight_amd import zn
from oracle import kv
from test_gpu_kv import attend_case, plain_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zn.lib()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("given", [False, True])
def test_rows_read_back_are_a_programs_own(dtype, given):
    c = random_cache(4, 3, 16, 64, 1)
    slots = i32([3, 60, -1, 17])
    kw = dict(out=tuple(torch.empty(4, 3, 64, dtype=dtype, device="cuda") for _ in range(2))) if given else {}
    k, v = zn.mx_kv_read(c, slots, dtype=dtype, **kw)
    old_k, old_v = k.clone(), v.clone()
    w = torch.full((64,), 2.0, dtype=dtype, device="cuda", requires_grad=True)
    k.mul_(w)                                                     # changed in place, with a gradient
    k.sum().backward()
    assert torch.equal(k.detach(), old_k * 2) and torch.equal(v, old_v) and not v.requires_grad
    # the sum over rows of what w multiplied: 12 values in whole 16ths (codes in halves, scales from 1/8), exact in FP32
    assert torch.equal(w.grad.float(), old_k.float().sum((0, 1)).to(dtype).float())
