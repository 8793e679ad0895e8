"""Calls of the key-value cache as a program mixes them with its own work: results that autograd may use, refusals."""
import numpy as np
import pytest
import torch

from kv_util import f64, i32, random_cache
from lossless_float_weight_amd import zn
from oracle import kv
from test_gpu_kv import plain_rows

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


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_tokens_that_share_a_slot_touch_no_other(t):
    c, d = (random_cache(40, 2, 16, 64, 7) for _ in range(2))
    tokens = 600
    k, v = plain_rows(tokens, 2, 64, t, 1).cuda(), plain_rows(tokens, 2, 64, t, 2).cuda()
    slots = np.random.default_rng(0).permutation(640)[:tokens]
    shared = np.arange(tokens) % 3 == 0                           # far from each other: in several workgroups
    zn.mx_kv_write(k, v, d, i32(np.where(shared, -1, slots).tolist()))
    slots[shared] = slots[0]
    zn.mx_kv_write(k, v, c, i32(slots.tolist()))
    page, place = int(slots[0]) // 16, int(slots[0]) % 16
    for i, x in ((0, k), (2, v)):
        codes, scales = kv.rows(f64(x[torch.from_numpy(shared).cuda()]))
        left, mine = c[i][page, :, place].cpu().numpy(), c[i + 1].view(torch.uint8)[page, :, place].cpu().numpy()
        # four bytes at a time of one of the tokens, and a scale of one of them
        for h in range(2):
            assert all((codes[:, h, at:at + 4] == left[h, at:at + 4]).all(1).any() for at in range(0, 32, 4))
            assert all((scales[:, h, b] == mine[h, b]).any() for b in range(2))
        for a, b in ((c[i], d[i]), (c[i + 1], d[i + 1])):
            a, b = a.view(torch.uint8).clone(), b.view(torch.uint8).clone()
            a[page, :, place], b[page, :, place] = 0, 0
            assert torch.equal(a, b)


def test_a_table_without_columns():
    # nothing fits but what asks for nothing
    none = torch.zeros(3, 0, dtype=torch.int32, device="cuda")
    step = zn.kv_extend(i32([0, 0, 0]), i32([2, 0, 1]), none, i32([4, 5]), i32([2]), 16, 8, 5)
    assert step.lens.tolist() == [0, 0, 0] and step.starts.tolist() == [0, 2, 2, 3] and step.n_free.tolist() == [2]
    assert step.slots.tolist() == [-1] * 5 and step.positions.tolist() == [0] * 5
    lens, n = zn.kv_release(i32([7, 0, 3]), torch.ones(3, dtype=torch.bool, device="cuda"), none, i32([4, 5]), i32([2]), 16)
    assert lens.tolist() == [0, 0, 0] and n.tolist() == [2]
