"""The key-value cache on the GPU: block tables and slots against the oracle
(equal), rows written and read (equal, bit for bit), attention within the bound
of kv_util.check_attention."""
import numpy as np
import pytest
import torch

from kv_util import TYPE, check_attention, dealt, f64, i32, random_cache, raw, values
from lossless_float_weight_amd import zn
from oracle import kv, mx

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zn.lib()


# ------------------------------------------------------------------ tables --
def step_case(batch, page, seed, spare=1.0, longest=200, new=40):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest, batch)
    add = np.where(rng.random(batch) < 0.2, 0, rng.integers(1, new + 1, batch))
    width = -(-longest // page) + max(1, new // page)
    need = int((-(-(lens + add) // page) + -lens // page).sum())
    used = int((-(-lens // page)).sum())
    n_pages = used + max(1, int(spare * need))
    order = rng.permutation(n_pages)
    table = rng.integers(-3, n_pages + 3, (batch, width))
    at = 0
    for b in range(batch):
        m = min(width, -(-int(lens[b]) // page))
        table[b, :m] = order[at:at + m]
        at += m
    return lens, add, table, order[at:], n_pages


def same_step(lens, add, table, free, n_free, page, n_pages, tokens):
    want = kv.extend([int(x) for x in lens], [int(x) for x in add], table.tolist(), [int(x) for x in free], n_free, page,
                     n_pages, tokens)
    t = i32(table.tolist()) if table.size else torch.zeros(table.shape, dtype=torch.int32, device="cuda")
    got = zn.kv_extend(i32(lens.tolist()), i32(add.tolist()), t, i32([int(x) for x in free]), i32([n_free]), page, n_pages, tokens)
    for name, g, w in zip(("lens", "starts", "slots", "positions", "n_free"), got, (*want[:4], [want[4]])):
        assert g.tolist() == list(w), name
    assert t.tolist() == want[5]
    return got


@pytest.mark.parametrize("batch,page,spare", [(1, 16, 1.0), (1, 1, 1.0), (3, 4, 0.5), (64, 64, 1.0), (65, 16, 0.7),
                                              (257, 32, 0.9), (600, 2, 1.0), (1030, 16, 0.3)])
def test_extend_equals_oracle(batch, page, spare):
    lens, add, table, free, n_pages = step_case(batch, page, batch + page, spare)
    total = int(add.sum())
    for tokens in (total, total + 37, max(0, total - 5), 0):
        same_step(lens, add, table, free, len(free), page, n_pages, tokens)


def test_extend_of_the_most_requests_and_of_none():
    lens, add, table, free, n_pages = step_case(8192, 16, 9, longest=40, new=3)
    same_step(lens, add, table, free, len(free), 16, n_pages, int(add.sum()))
    none = np.zeros(0, np.int64)
    same_step(none, none, np.zeros((0, 4), np.int64), np.arange(5), 5, 16, 8, 3)
    same_step(none, none, np.zeros((0, 0), np.int64), none, 0, 16, 0, 0)


def test_extend_checks_what_the_device_holds():
    lens, add, table, free, n_pages = step_case(40, 16, 5)
    total = int(add.sum())
    odd = lens.copy()
    odd[::7] = -5
    odd[3] = 10 ** 9                                             # longer than its table
    more = add.copy()
    more[1::9] = -1
    more[5] = 2 ** 31 - 1                                        # starts pass 32 bits after two of them
    more[6] = 2 ** 31 - 1
    same_step(odd, add, table, free, len(free), 16, n_pages, total)
    same_step(odd, more, table, free, len(free), 16, n_pages, total)
    same_step(lens, add, table, free, -4, 16, n_pages, total)    # a stack below empty
    same_step(lens, add, table, free, 10 ** 9, 16, n_pages, total)
    bad = free.copy()
    bad[::3] = n_pages + 7
    bad[1::3] = -2
    wrong = table.copy()
    wrong[::2, 0] = -1
    same_step(lens, add, wrong, bad, len(free), 16, n_pages, total)
    same_step(lens, add, table, free, len(free), 16, 0, total)   # no pages at all


@pytest.mark.parametrize("batch,page", [(1, 16), (5, 1), (64, 64), (300, 16), (2000, 8)])
def test_release_equals_oracle(batch, page):
    lens, _, table, free, n_pages = step_case(batch, page, batch)
    rng = np.random.default_rng(batch)
    lens = np.where(rng.random(batch) < 0.05, -3, lens)
    if batch > 4:
        lens[2] = 10 ** 9
    for share in (0.0, 0.3, 1.0):
        done = rng.random(batch) < share
        for cap in (n_pages + 10 * table.shape[1], len(free) + 3):
            stack = np.concatenate([free, np.full(cap - len(free), -1)])
            want = kv.release([int(x) for x in lens], done.tolist(), table.tolist(), stack.tolist(), len(free), page)
            f, t = i32(stack.tolist()), i32(table.tolist())
            got = zn.kv_release(i32(lens.tolist()), torch.tensor(done).cuda(), t, f, i32([len(free)]), page)
            assert got[0].tolist() == want[0] and f.tolist() == want[1] and got[1].tolist() == [want[2]]
            assert t.tolist() == table.tolist()


def test_tables_given_outputs_and_strided_tables():
    lens, add, table, free, n_pages = step_case(20, 16, 3)
    total = int(add.sum())
    want = kv.extend(lens.tolist(), add.tolist(), table.tolist(), free.tolist(), len(free), 16, n_pages, total)
    wide = torch.full((20, table.shape[1] + 3), 99, dtype=torch.int32, device="cuda")
    t = wide[:, 1:1 + table.shape[1]]
    t.copy_(i32(table.tolist()))
    out = zn.KvStep(*(torch.full((n,), 5, dtype=torch.int32, device="cuda") for n in (20, 21, total, total, 1)))
    got = zn.kv_extend(i32(lens.tolist()), i32(add.tolist()), t, i32(free.tolist()), i32([len(free)]), 16, n_pages, total,
                       out=out)
    assert all(a is b for a, b in zip(got, out)) and got.slots.tolist() == want[2] and t.tolist() == want[5]
    assert (wide[:, 0] == 99).all() and (wide[:, -2:] == 99).all()
    n = i32([len(free)])
    with pytest.raises(zn.ZnError):
        zn.kv_extend(i32(lens.tolist()), i32(add.tolist()), t, i32(free.tolist()), n, 16, n_pages, total, out=out._replace(n_free=n))
    with pytest.raises(zn.ZnError):
        zn.kv_extend(i32(lens.tolist()), i32(add.tolist()), t, i32(free.tolist()), n, 16, n_pages, total + 1, out=out)
    with pytest.raises(zn.ZnError):
        zn.kv_release(out.lens, torch.zeros(20, dtype=torch.bool, device="cuda"), t, i32(free.tolist()), n, 16, out=(out.lens, out.n_free))


# -------------------------------------------------------------------- rows --
def plain_rows(tokens, heads, dim, t, seed):
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 1, (tokens, heads, dim)) * np.exp2(rng.integers(-9, 9, (tokens, heads, 1)))
    x = np.where(rng.random(x.shape) < 0.05, 0.0, x)
    return torch.from_numpy(x).to(TYPE[t])


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens,heads,dim,page,strides", [
    (1, 1, 32, 16, "pages"), (3, 8, 128, 64, "pages"), (100, 5, 96, 16, "beside"), (33, 3, 256, 32, "tokens"),
    (260, 2, 160, 128, "pages"), (17, 1, 64, 16, "tokens")])
def test_write_and_read(tokens, heads, dim, page, strides, t):
    n_pages = tokens // page + 3
    c = random_cache(n_pages, heads, page, dim, 7, strides)
    before = [raw(x).copy() for x in c]
    k, v = plain_rows(tokens, heads, dim, t, 1), plain_rows(tokens, heads, dim, t, 2)
    if tokens > 2:
        k[1, 0, 3], v[2, -1, dim - 1] = float("inf"), float("nan")
    rng = np.random.default_rng(3)
    slots = rng.permutation(n_pages * page)[:tokens]
    if tokens > 10:
        slots[::9] = -1
        slots[4] = n_pages * page
        slots[5] = 2 ** 31 - 1
        slots[6] = -2 ** 31
    zn.mx_kv_write(k.cuda(), v.cuda(), c, i32(slots.tolist()))
    live = (slots >= 0) & (slots < n_pages * page)
    for x, at in ((k, 0), (v, 2)):
        codes, scales = kv.rows(f64(x))
        for want, now, old in ((codes, raw(c[at]), before[at]), (scales, raw(c[at + 1]), before[at + 1])):
            old = old.reshape(now.shape)
            old[slots[live] // page, :, slots[live] % page] = want[live]
            np.testing.assert_array_equal(now, old)
    for dtype in TYPE.values():
        got = zn.mx_kv_read(c, i32(slots.tolist()), dtype=dtype)
        for y, x in zip(got, (k, v)):
            want = np.where(live[:, None, None], kv.values(*kv.rows(f64(x))), 0.0)
            np.testing.assert_array_equal(f64(y), want)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_write_takes_strides(t):
    c, d = (random_cache(4, 3, 16, 64, 1) for _ in range(2))
    x = plain_rows(20, 3, 3 * 64 + 1, t, 4).cuda()               # q, k and v of a projection in one row
    k, v = x[:, :, 1:65], x[:, :, 129:193]
    slots = i32(list(range(5, 25)))
    zn.mx_kv_write(k, v, c, slots)
    zn.mx_kv_write(k.contiguous(), v.contiguous(), d, slots)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(c, d))
    turned = k.transpose(0, 1).contiguous().transpose(0, 1)
    zn.mx_kv_write(turned, v[:1].expand(20, 3, 64), d, slots)
    assert torch.equal(c.k, d.k) and torch.equal(d.v.view(-1, 32)[5], c.v.view(-1, 32)[5])
    got = zn.mx_kv_read(d, slots)[1]
    assert torch.equal(got, got[:1].expand_as(got))


def test_pages_are_rows_of_the_other_operators():
    c = random_cache(3, 2, 16, 64, 2)
    x = plain_rows(16, 2, 64, "bf16", 5).cuda()
    zn.mx_kv_write(x, x, c, i32(list(range(16, 32))))
    codes, scales = zn.mx_quantize(x.transpose(0, 1).contiguous(), zn.FP4X2_E2M1)
    assert torch.equal(c.k[1], codes) and torch.equal(c.k_scales[1].view(torch.uint8), scales.view(torch.uint8))
    assert torch.equal(zn.mx_dequantize(c.v[1], c.v_scales[1]), zn.mx_kv_read(c, i32(list(range(16, 32))))[1].transpose(0, 1))
    ts = zn.setup([c.k])                                          # and tensors of an FP4 plan
    assert torch.equal(zn.decompress(ts, zn.compress(ts, [c.k]))[0].view(c.k.shape), c.k)


# --------------------------------------------------------------- attention --
def attend_case(lens, new, heads, kv_heads, dim, page, t, seed, strides="pages", pad=0, spread=2):
    """(q, cache, table, starts); new None: one query a request and no starts."""
    width = max(1, -(-max(lens) // page) + 1)
    n_pages = sum(-(-n // page) for n in lens) + 2
    c = random_cache(n_pages, kv_heads, page, dim, seed, strides, spread)
    table = dealt(lens, page, n_pages, width, seed)
    starts = None if new is None else np.concatenate([[0], np.cumsum(new)]).tolist()
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((len(lens) if starts is None else starts[-1]) + pad, heads, dim, generator=g).to(TYPE[t])
    return q.cuda(), c, table, starts


def run_attention(lens, new, heads, kv_heads, dim, page, t, seed, strides="pages", **kw):
    print("case:", lens, new, heads, kv_heads, dim, page, t, kw, flush=True)
    q, c, table, starts = attend_case(lens, new, heads, kv_heads, dim, page, t, seed, strides)
    hint = {} if new is None else {"max_new": max(new)}
    out, lse = zn.mx_attention(q, c, i32(table.tolist()), i32(lens), None if starts is None else i32(starts), lse=True,
                               **hint, **kw)
    check_attention(q, c, table, lens, starts, page, out, lse, **kw)
    return q, c, table, starts, out, lse


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
def test_attention_of_every_head_size(dim, t):
    run_attention([70, 1, 0, 333], None, 4, 2, dim, 16, t, dim)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (5, 5), (3, 1), (14, 2), (16, 1), (40, 2), (33, 1), (128, 1)])
def test_attention_of_every_group(heads, kv_heads, t):
    run_attention([5, 130], None, heads, kv_heads, 64, 32, t, heads)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 63, 64, 65, 127, 255, 256, 257, 1000])
def test_attention_of_every_length(n):
    run_attention([n, 0, n + 1], None, 4, 1, 128, 64, "bf16", n)


@pytest.mark.parametrize("page", [16, 32, 128, 1024])
@pytest.mark.parametrize("strides", ["pages", "beside", "tokens"])
def test_attention_of_pages_and_orders(page, strides):
    run_attention([200, 77], [3, 1], 4, 2, 96, page, "bf16", page, strides)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,new", [([40, 90, 7], [40, 5, 7]), ([300, 0, 20], [129, 0, 1]), ([3, 200], [9, 33]),
                                      ([700], [700]), ([65, 64, 63, 130], [2, 64, 63, 100])])
@pytest.mark.parametrize("mask", [dict(), dict(window=1), dict(window=50), dict(window=5000), dict(causal=False)])
def test_attention_of_several_queries(lens, new, mask, t):
    run_attention(lens, new, 6, 2, 64, 16, t, sum(lens), **mask)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,new,mask", [([9000, 300], None, dict()), ([5000, 1, 2500], [4, 1, 2], dict()),
                                           ([9000, 4000], None, dict(window=3000)), ([6000], [5], dict(causal=False)),
                                           ([4100], [300], dict())])
def test_attention_of_long_caches(lens, new, mask, t):
    run_attention(lens, new, 4, 1, 64, 64, t, 3, **mask)


@pytest.mark.parametrize("dim", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("lens,new", [([700, 150, 0], [300, 150, 0]), ([257, 5, 900], [257, 5, 256])])
def test_attention_of_many_rows(lens, new, dim):
    # 512 rows a request on average and more
    run_attention(lens, new, 8, 2, dim, 32, "bf16", dim)
    run_attention(lens, new, 4, 1, dim, 16, "bf16", dim, window=100)


@pytest.mark.parametrize("batch", [64, 65, 300, 700])
def test_attention_of_many_requests(batch):
    rng = np.random.default_rng(batch)
    lens = rng.integers(0, 90, batch).tolist()
    lens[0] = 1500
    run_attention(lens, None, 2, 1, 32, 16, "bf16", batch)
    run_attention(lens, rng.integers(0, 4, batch).tolist(), 2, 1, 32, 16, "bf16", batch)


def test_equal_weights_give_means():
    # queries of zeros: each result is the mean of the values seen, small whole numbers summed exactly
    for lens, new, page, mask in (([100, 37], [100, 3], 16, dict()), ([500, 64], [70, 64], 64, dict(window=33)),
                                  ([2000], [2], 32, dict(causal=False)), ([5000], [1], 64, dict())):
        q, c, table, starts = attend_case(lens, new, 2, 1, 64, page, "fp32", 1)
        c.v_scales.view(torch.uint8).fill_(128)                   # whole numbers up to 12
        out, lse = zn.mx_attention(torch.zeros_like(q), c, i32(table.tolist()), i32(lens), i32(starts), lse=True, **mask)
        want, l2, _ = kv.attention(np.zeros(q.shape), *values(c), table, lens, starts, page, **mask)
        # one division and one product: two roundings
        assert (np.abs(f64(out) - want) <= 2.0 ** -22 * np.abs(want)).all()
        assert (np.abs(f64(lse) - l2) <= 2.0 ** -21 * np.maximum(1, np.abs(l2))).all()


def test_scores_far_apart():
    # one key far above the others, late and early; scores to +-1e4 and beyond FP32's range of weights
    for at in (0, 300, 699):
        q, c, table, starts = attend_case([700], None, 4, 1, 64, 64, "bf16", at)
        q.mul_(100)
        c.k_scales.view(torch.uint8).fill_(127)
        page, place = table[0][at // 64], at % 64
        c.k_scales.view(torch.uint8)[page, :, place] = 134
        out, lse = zn.mx_attention(q, c, i32(table.tolist()), i32([700]), lse=True)
        check_attention(q, c, table, [700], None, 64, out, lse)
        out = zn.mx_attention(q, c, i32(table.tolist()), i32([700]), scale=1e-3)
        check_attention(q, c, table, [700], None, 64, out, scale=1e-3)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,new", [([300], None), ([3000], None), ([300], [200]), ([3000], [40])])
def test_scores_past_the_weights_precision(lens, new, t):
    # scores to 2^60, whose last bits are worth far more than a weight's exponent: one key has all the weight
    q, c, table, starts = attend_case(lens, new, 2, 1, 64, 64, t, 3)
    c.k_scales.view(torch.uint8).copy_(torch.randint(60, 187, c.k_scales.shape))
    out, lse = zn.mx_attention(q, c, i32(table.tolist()), i32(lens), None if new is None else i32(starts), lse=True)
    assert not out.isnan().any() and not lse.isnan().any()
    k, v = values(c)
    rows = [(b, t) for b, n in enumerate(lens) for t in range(1 if new is None else new[b])]
    at = np.arange(lens[0])
    pages = np.array(table[0])[at // 64]
    kk, vv, x = k[pages, 0, at % 64], v[pages, 0, at % 64], f64(q)
    for r, (b, i) in enumerate(rows):
        seen = lens[0] - len(rows) + i + 1
        for h in range(2):
            s = kk[:seen] @ x[r, h] / 8
            order = np.argsort(s)
            if seen == 1 or s[order[-1]] - s[order[-2]] > 2.0 ** -18 * s[order[-1]] + 200:
                assert np.array_equal(f64(out)[r, h], vv[order[-1]].astype(np.float32)), (r, h)
                assert abs(f64(lse)[r, h] - s[order[-1]]) <= 2.0 ** -16 * abs(s[order[-1]]) + 2.0 ** -20


def test_rows_behind_the_last_request_stay():
    q, c, table, starts = attend_case([30, 50], [3, 4], 4, 2, 64, 16, "bf16", 3, pad=9)
    for n in (9, 0):
        qq = q[:7 + n]
        out = torch.full_like(qq, 7.0)
        lse = torch.full(qq.shape[:2], 7.0, device="cuda")
        got = zn.mx_attention(qq, c, i32(table.tolist()), i32([30, 50]), i32(starts), out=out, lse=lse)
        assert got[0] is out and got[1] is lse
        assert (out[7:] == 7).all() and (lse[7:] == 7).all()
        check_attention(qq, c, table, [30, 50], starts, 16, out, lse)


def test_attention_takes_strides():
    q, c, table, starts = attend_case([30, 50], [3, 4], 4, 2, 64, 16, "bf16", 3)
    want = zn.mx_attention(q, c, i32(table.tolist()), i32([30, 50]), i32(starts))
    wide = torch.zeros(7, 9, 67, dtype=q.dtype, device="cuda")
    wide[:, 2:6, 3:] = q
    place = torch.full((4, 8, 65), 7.0, dtype=q.dtype, device="cuda")
    out = place.transpose(0, 1)[:7, :, 1:]
    t = torch.full((2, table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    t[:, 2:2 + table.shape[1]] = i32(table.tolist())
    zn.mx_attention(wide[:, 2:6, 3:], c, t[:, 2:2 + table.shape[1]], i32([30, 50]), i32(starts), out=out)
    assert torch.equal(out, want) and (place[:, :, 0] == 7).all() and (place[:, 7] == 7).all()
    one = q[:1, :1].expand(7, 4, 64)
    assert torch.equal(zn.mx_attention(one, c, t[:, 2:2 + table.shape[1]], i32([30, 50]), i32(starts)),
                       zn.mx_attention(one.contiguous(), c, i32(table.tolist()), i32([30, 50]), i32(starts)))
    with pytest.raises(zn.ZnError):
        zn.mx_attention(q, c, i32(table.tolist()), i32([30, 50]), i32(starts), out=q[:1, :1].expand(7, 4, 64))


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_what_a_query_does_not_see_has_no_effect(t):
    lens, new = [100, 45, 200], [70, 2, 1]
    for mask in (dict(), dict(window=20)):
        q, c, table, starts = attend_case(lens, new, 4, 2, 64, 16, t, 8)
        tb = i32(table.tolist())
        want = zn.mx_attention(q, c, tb, i32(lens), i32(starts), **mask)
        # NaNs behind every length, in pages of the table that no token reaches, and in pages of nobody
        seen = torch.zeros(c.k.shape[0], 16, dtype=torch.bool, device="cuda")
        for row, n in zip(table, lens):
            for p in range(n):
                seen[row[p // 16], p % 16] = True
        for s in (c.k_scales, c.v_scales):
            s.view(torch.uint8).masked_fill_(~seen[:, None, :, None], 255)
        assert torch.equal(zn.mx_attention(q, c, tb, i32(lens), i32(starts), **mask), want)
        # NaNs at one key: the queries that see it are NaN, where the block is, the others are as they were
        for s, key in ((c.v_scales, 60), (c.v_scales, 31), (c.k_scales, 64)):
            u = s.view(torch.uint8)
            old = u.clone()
            u[table[0][key // 16], 1, key % 16, 1] = 255
            out = zn.mx_attention(q, c, tb, i32(lens), i32(starts), **mask)
            pos = torch.arange(30, 100, device="cuda")
            hit = (pos >= key) & ((pos < key + mask["window"]) if mask else (pos >= 0))
            hit = torch.cat([hit, torch.zeros(3, dtype=torch.bool, device="cuda")])
            nan = torch.zeros_like(out, dtype=torch.bool)
            nan[hit, 2:, 0 if s is c.k_scales else 32:] = True
            assert torch.equal(out.isnan(), nan) and torch.equal(out[~nan], want[~nan])
            u.copy_(old)


@pytest.mark.parametrize("kind", ["near", "less near", "far", "rising", "zeros first", "one far block", "far where nobody looks"])
def test_values_of_many_sizes(kind):
    # values whose scales leave FP16's reach of the first tile's are taken another way
    lens, new = [300, 90], [200, 90]
    q, c, table, starts = attend_case(lens, new, 4, 2, 64, 16, "bf16", 9)
    vs, rng = c.v_scales.view(torch.uint8), np.random.default_rng(2)
    where = torch.zeros(c.v.shape[0], 16, dtype=torch.long, device="cuda")     # the position of each place
    for row, n in zip(table, lens):
        for p in range(n):
            where[row[p // 16], p % 16] = p
    pos = where[:, None, :, None].expand(vs.shape)
    if kind == "near":        # as far as it reaches: 12 above and 13 below the first tile's largest
        vs.copy_(torch.where(pos < 64, 127, torch.from_numpy(rng.integers(114, 140, vs.shape)).cuda()))
    elif kind == "less near":
        vs.copy_(torch.where(pos < 64, 127, torch.from_numpy(rng.integers(104, 140, vs.shape)).cuda()))
    elif kind == "far":
        vs.copy_(torch.from_numpy(rng.integers(60, 200, vs.shape)))
    elif kind == "rising":
        vs.copy_(100 + pos // 8)
    elif kind == "zeros first":
        c.v.mul_(where[:, None, :, None] >= 64)
        vs.copy_(torch.where(pos < 64, 0, 150))
    elif kind == "one far block":
        vs[table[0][250 // 16], 1, 250 % 16, 1] = 90
    else:                     # pages that no request's length reaches, and a key of zeros
        used = torch.zeros(c.v.shape[0], 16, dtype=torch.bool, device="cuda")
        for row, n in zip(table, lens):
            for p in range(n):
                used[row[p // 16], p % 16] = True
        vs.masked_fill_(~used[:, None, :, None], 200)
        c.v[table[0][200 // 16], :, 200 % 16] = 0x80 | 0x08
        vs[table[0][200 // 16], :, 200 % 16] = 0
    for mask in (dict(), dict(window=70), dict(causal=False)):
        out, lse = zn.mx_attention(q, c, i32(table.tolist()), i32(lens), i32(starts), lse=True, **mask)
        check_attention(q, c, table, lens, starts, 16, out, lse, **mask)


def test_small_values_beside_large_ones_keep_their_bits():
    lens, new = [150], [100]
    q, c, table, starts = attend_case(lens, new, 4, 1, 64, 16, "bf16", 9)
    vs = c.v_scales.view(torch.uint8)
    vs.fill_(127)
    args = (q, c, i32(table.tolist()), i32(lens), i32(starts))
    want = zn.mx_attention(*args)
    for byte in (104, 110, 113, 114, 120, 139, 140):
        vs[..., 1] = byte
        out = zn.mx_attention(*args)
        check_attention(q, c, table, lens, starts, 16, out)
        if 114 <= byte <= 139:    # 2^-13 to 2^12 of the other block: powers of two, exact
            assert torch.equal(out[..., :32], want[..., :32])
            assert torch.equal(out[..., 32:].float() * 2.0 ** (127 - byte), want[..., 32:].float())


@pytest.mark.parametrize("new", [1, 40])
def test_many_small_weights_add_up(new):
    # one key with a weight of 1 and a value of 0, 300 with weights of 2^-23 and values of 6
    q, c, table, starts = attend_case([301], [new], 1, 1, 32, 64, "bf16", 9)
    q.zero_()
    q[:, :, 0] = 23.0
    c.k.zero_()
    c.k_scales.view(torch.uint8).fill_(127)
    c.k[table[0][0], 0, 0, 0] = 2                                  # 1.0
    c.v.fill_(0x77)
    c.v_scales.view(torch.uint8).fill_(127)
    c.v[table[0][0], 0, 0] = 0
    out = zn.mx_attention(q, c, i32(table.tolist()), i32([301]), i32(starts), scale=float(np.log(2.0)), causal=False)
    want = 300 * 6 * 2.0 ** -23 / (1 + 300 * 2.0 ** -23)
    # each weight within 2^-11 of itself and 2^-32, the scale's rounding 23 * 2^-24, the result's half a step
    assert (np.abs(f64(out) - want) <= want * (2.0 ** -11 + 2.0 ** -9 + 2.0 ** -16 + 2.0 ** -8)).all()


def test_offsets_past_32_bits():
    heads, page, dim, n_pages = 8, 64, 128, 150000                 # 4.9 GB of codes each
    c = zn.mx_kv_cache(n_pages, heads, page, dim)
    small = zn.mx_kv_cache(8, heads, page, dim)
    high = [149999, 140001, 75000, 131073, 3, 149000]
    lens = [300, 70]
    table = i32([high[:5], [high[5], 0, 0, 0, 0]])
    near = i32([[0, 1, 2, 3, 4], [5, 6, 6, 6, 6]])
    rng = np.random.default_rng(0)
    k, v = (torch.from_numpy(rng.normal(0, 1, (370, heads, dim))).bfloat16().cuda() for _ in range(2))
    def slots(t):
        t = t.tolist()
        return i32([t[b][p // page] * page + p % page for b, n in enumerate(lens) for p in range(n)])
    table[1, 1] = 99999
    near[1, 1] = 6
    for cache, t in ((c, table), (small, near)):
        zn.mx_kv_write(k, v, cache, slots(t))
    for a, b in zip(zn.mx_kv_read(c, slots(table)), zn.mx_kv_read(small, slots(near))):
        assert torch.equal(a, b)
    for new in ([1, 1], [60, 20], [300, 70]):
        starts = i32([0, new[0], sum(new)])
        q = torch.randn(sum(new), 16, dim, device="cuda").bfloat16()
        for hint in (1, 300):
            assert torch.equal(zn.mx_attention(q, c, table, i32(lens), starts, max_new=hint),
                               zn.mx_attention(q, small, near, i32(lens), starts, max_new=hint))


def test_the_largest_page():
    run_attention([70000, 5], None, 2, 1, 32, 65536, "bf16", 3)
    run_attention([66000], [20], 2, 1, 32, 65536, "bf16", 4)


def test_nans_among_the_largest_values():
    # a NaN's byte lies within reach of the largest scales
    lens, new = [100], [80]
    q, c, table, starts = attend_case(lens, new, 4, 1, 64, 16, "bf16", 9)
    vs = c.v_scales.view(torch.uint8)
    vs.fill_(240)
    want = zn.mx_attention(q, c, i32(table.tolist()), i32(lens), i32(starts))
    for byte in (253, 254, 255):
        vs[table[0][50 // 16], 0, 50 % 16, 1] = byte
        out = zn.mx_attention(q, c, i32(table.tolist()), i32(lens), i32(starts))
        nan = torch.zeros_like(out, dtype=torch.bool)
        nan[30:, :, 32:] = True                                # queries at 20 .. 99
        assert torch.equal(out.isnan(), nan) and torch.equal(out[~nan], want[~nan])


def test_values_of_many_sizes_in_pieces():
    lens, new = [5000], [20]
    q, c, table, starts = attend_case(lens, new, 4, 2, 64, 64, "bf16", 9)
    c.v_scales.view(torch.uint8)[table[0][70], 0, 5, 0] = 60       # one piece the other way, the others not
    out, lse = zn.mx_attention(q, c, i32(table.tolist()), i32(lens), i32(starts), lse=True)
    check_attention(q, c, table, lens, starts, 64, out, lse)


def test_scale_bytes_at_the_ends():
    q, c, table, starts = attend_case([90], None, 2, 1, 64, 16, "bf16", 4)
    vs = c.v_scales.view(torch.uint8)
    for byte in (0, 1, 100, 200, 240, 250, 252):
        vs.fill_(byte)
        out = zn.mx_attention(q, c, i32(table.tolist()), i32([90]))
        # byte 0 gives values from 2^-128 and results under 2^-126, whose step is 2^-133; byte 1 results up to
        # 6 * 2^-126, whose half steps reach 2^-132: half a step of the value or 2^-134, whichever is more
        check_attention(q, c, table, [90], None, 16, out)
    vs.fill_(253)
    assert zn.mx_attention(q, c, i32(table.tolist()), i32([90])).isnan().all()


def test_queries_that_are_not_finite_stay_by_themselves():
    q, c, table, starts = attend_case([90, 40], [9, 5], 4, 1, 64, 16, "bf16", 4)
    want = zn.mx_attention(q, c, i32(table.tolist()), i32([90, 40]), i32(starts))
    q[2, 1, 5], q[11, 3, 0] = float("nan"), float("inf")
    out = zn.mx_attention(q, c, i32(table.tolist()), i32([90, 40]), i32(starts))
    assert out[2, 1].isnan().all() and out[11, 3].isnan().all()
    same = torch.ones(14, 4, dtype=torch.bool)
    same[2, 1] = same[11, 3] = False
    assert torch.equal(out[same], want[same])


def test_attention_checks_what_the_device_holds():
    lens = [100, 45, 200]
    q, c, table, _ = attend_case(lens, None, 4, 2, 64, 16, "bf16", 8)
    want = zn.mx_attention(q, c, i32(table.tolist()), i32(lens))
    # a page outside the cache: whoever sees it gets NaNs
    for page in (-1, c.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        bad = table.copy()
        bad[1, 2] = page
        bad[0, 7:] = page                                        # behind the length: not looked at
        out, lse = zn.mx_attention(q, c, i32(bad.tolist()), i32(lens), lse=True)
        assert out[1].isnan().all() and lse[1].isnan().all()
        assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])
    # lengths past the table, and below 0
    out, lse = zn.mx_attention(q, c, i32(table.tolist()), i32([table.shape[1] * 16 + 1, -7, 200]), lse=True)
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert (out[1] == 0).all() and (lse[1] == -torch.inf).all()
    # (the order of a request's sums goes by all lengths: the same result, not the same bits)
    check_attention(q[2:], c, table[2:], lens[2:], None, 16, out[2:], lse[2:])
    out = zn.mx_attention(q, c, i32(table.tolist()), i32([2 ** 31 - 1, -2 ** 31, 200]))
    assert out[0].isnan().all() and (out[1] == 0).all()
    check_attention(q[2:], c, table[2:], lens[2:], None, 16, out[2:])
    # a table without columns
    out = zn.mx_attention(q, c, torch.zeros(3, 0, dtype=torch.int32, device="cuda"), i32([0, 0, 0]))
    assert (out == 0).all()
    # starts outside the queries, and a request that ends before it starts
    out = torch.full_like(q, 7.0)
    zn.mx_attention(q, c, i32(table.tolist()), i32(lens), i32([-5, 1, 1, 9]), out=out)
    check_attention(q, c, table, lens, [0, 1, 1, 3], 16, out)
    zn.mx_attention(q, c, i32(table.tolist()), i32(lens), i32([2, -1, 3, 1]), out=out)
    torch.cuda.synchronize()


def test_no_queries():
    q, c, table, _ = attend_case([10], None, 4, 2, 64, 16, "bf16", 8)
    got = zn.mx_attention(q[:0], c, i32(table[:0].tolist()).view(0, 1), i32([]))
    assert got.shape == (0, 4, 64)
    out = torch.full_like(q, 7.0)
    zn.mx_attention(q, c, i32(table.tolist()), i32([10]), i32([0, 0]), out=out)
    assert (out == 7).all()


def test_the_hint_has_no_effect_but_on_sums():
    lens, new = [300, 90, 33], [40, 1, 33]
    q, c, table, starts = attend_case(lens, new, 4, 2, 128, 64, "bf16", 8)
    for hint in (0, 1, 7, 40, 74, 10 ** 6):
        out, lse = zn.mx_attention(q, c, i32(table.tolist()), i32(lens), i32(starts), max_new=hint, lse=True)
        check_attention(q, c, table, lens, starts, 64, out, lse)


def test_the_same_bits_again():
    q, c, table, starts = attend_case([9000, 300, 4000], None, 8, 2, 128, 64, "bf16", 8)
    args = (q, c, i32(table.tolist()), i32([9000, 300, 4000]))
    first = zn.mx_attention(*args)
    for _ in range(5):
        assert torch.equal(zn.mx_attention(*args), first)


def test_another_stream():
    q, c, table, starts = attend_case([900, 300], None, 8, 2, 128, 64, "bf16", 8)
    tb, ln = i32(table.tolist()), i32([900, 300])
    want = zn.mx_attention(q, c, tb, ln)
    k = torch.randn(5, 2, 128, device="cuda").bfloat16()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = zn.mx_attention(q, c, tb, ln, stream=s)
    d = zn.mx_kv_cache(4, 2, 16, 128)
    s.wait_stream(torch.cuda.current_stream())
    step = zn.kv_extend(i32([3]), i32([5]), i32([[0, 0]]), i32([1, 2, 3]), i32([3]), 16, 4, 5, stream=s)
    s.wait_stream(torch.cuda.current_stream())
    zn.mx_kv_write(k, k, d, step.slots, stream=s)
    back = zn.mx_kv_read(d, step.slots, stream=s)
    gone = zn.kv_release(step.lens, torch.ones(1, dtype=torch.bool, device="cuda"), i32([[0, 0]]), i32([1, 2, 3]), step.n_free, 16,
                         stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(out, want) and step.slots.tolist() == [3, 4, 5, 6, 7] and gone[0].tolist() == [0]
    np.testing.assert_array_equal(f64(back[0]), kv.values(*kv.rows(f64(k))))


# ------------------------------------------------------------ run together --
@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_a_serving_loop(t):
    """Prompts, steps of single tokens and of drafts, requests that end and others that take their place."""
    heads, kv_heads, dim, page, batch, width = 6, 2, 64, 16, 5, 8
    n_pages = 24
    rng = np.random.default_rng(0)
    c = random_cache(n_pages, kv_heads, page, dim, 1)
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(n_pages, dtype=torch.int32, device="cuda")
    n_free, lens = i32([n_pages]), i32([0] * batch)
    held = [np.zeros((0, 2, kv_heads, dim)) for _ in range(batch)]   # what each request's tokens hold
    plan = [([30, 0, 17, 64, 5], []), ([1] * 5, []), ([3, 2, 5, 1, 4], [3]), ([1, 40, 1, 50, 1], []), ([1] * 5, [0, 2]),
            ([90, 1, 33, 1, 100], []), ([1, 1, 1, 1, 1], [])]
    for add, done in plan:
        flags = torch.tensor([b in done for b in range(batch)], device="cuda")
        lens, n_free = zn.kv_release(lens, flags, table, free, n_free, page)
        for b in done:
            held[b] = held[b][:0]
        total = sum(add)
        step = zn.kv_extend(lens, i32(add), table, free, n_free, page, n_pages, total)
        k, v, q = (torch.from_numpy(rng.normal(0, 1, (total, h, dim))).to(TYPE[t]).cuda() for h in (kv_heads, kv_heads, heads))
        zn.mx_kv_write(k, v, c, step.slots)
        out = zn.mx_attention(q, c, table, step.lens, step.starts, max_new=max(add))
        lens, n_free = step.lens, step.n_free
        stored = np.stack([kv.values(*kv.rows(f64(x))) for x in (k, v)], 1)
        starts = np.concatenate([[0], np.cumsum(add)])
        now = lens.tolist()
        for b in range(batch):
            if now[b] != len(held[b]):
                assert now[b] == len(held[b]) + add[b]
                held[b] = np.concatenate([held[b], stored[starts[b]:starts[b + 1]]])
        tb = table.tolist()
        used = [p for b in range(batch) for p in tb[b][:-(-now[b] // page)]]
        assert len(set(used)) == len(used) and sorted(used + free.tolist()[:n_free.item()]) == list(range(n_pages))
        kk, vv = values(c)
        for b in range(batch):
            at = np.arange(now[b])
            pages = np.array(tb[b], dtype=np.int64)[at // page]
            np.testing.assert_array_equal(kk[pages, :, at % page], held[b][:, 0])
            np.testing.assert_array_equal(vv[pages, :, at % page], held[b][:, 1])
        check_attention(q, c, np.array(tb), now, starts.tolist(), page, out)
    assert -1 in step.slots.tolist() or len(used) <= n_pages


def test_a_captured_step_replayed():
    """Table, write and attention of a decoding step in one graph; lengths move on by a copy inside it."""
    heads, kv_heads, dim, page, batch, n_pages = 8, 2, 64, 16, 6, 64
    def make():
        c = random_cache(n_pages, kv_heads, page, dim, 1)
        return c, torch.full((batch, 10), -1, dtype=torch.int32, device="cuda"), torch.arange(n_pages, dtype=torch.int32, device="cuda"), i32([n_pages]), i32([0] * batch)
    rng = np.random.default_rng(1)
    prompt = torch.from_numpy(rng.normal(0, 1, (60, kv_heads, dim))).bfloat16().cuda()
    new = torch.empty(batch, kv_heads, dim, dtype=torch.bfloat16, device="cuda")
    q = torch.empty(batch, heads, dim, dtype=torch.bfloat16, device="cuda")
    one = i32([1] * batch)
    def prefill(c, table, free, n_free, lens):
        step = zn.kv_extend(lens, i32([10, 20, 0, 15, 14, 1]), table, free, n_free, page, n_pages, 60)
        zn.mx_kv_write(prompt, prompt, c, step.slots)
        lens.copy_(step.lens)
        n_free.copy_(step.n_free)
    def step(c, table, free, n_free, lens):
        s = zn.kv_extend(lens, one, table, free, n_free, page, n_pages, batch)
        zn.mx_kv_write(new, new, c, s.slots)
        out = zn.mx_attention(q, c, table, s.lens)
        lens.copy_(s.lens)
        n_free.copy_(s.n_free)
        return out
    eager, captured = make(), make()
    prefill(*eager)
    prefill(*captured)
    new.copy_(prompt[:batch])
    q.normal_()
    saved = [x.clone() for x in (*captured[0], *captured[1:])]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*captured)
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((*captured[0], *captured[1:]), saved):
        x.copy_(y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step(*captured)
    for i in range(25):
        new.copy_(torch.from_numpy(rng.normal(0, 1, (batch, kv_heads, dim))))
        q.normal_()
        want = step(*eager)
        g.replay()
        if i % 3 == 0:
            torch.cuda.synchronize()
        assert torch.equal(got, want), i
        assert all(torch.equal(a, b) for a, b in zip(captured[1:], eager[1:]))


@pytest.mark.parametrize("lens,new,spread", [([600, 40], None, 2), ([7000, 900], None, 2), ([500, 300], [90, 300], 2),
                                             ([6000], [33], 2), ([500, 300], [90, 300], 60)])
def test_every_kernel_captured_and_replayed(lens, new, spread):
    q, c, table, starts = attend_case(lens, new, 8, 2, 128, 64, "bf16", 1, spread=spread)
    args = [q, c, i32(table.tolist()), i32(lens)] + ([i32(starts)] if new else [])
    g = torch.cuda.CUDAGraph()
    zn.mx_attention(*args, lse=True)
    with torch.cuda.graph(g):
        out, lse = zn.mx_attention(*args, lse=True)
    for i in range(6):
        q.normal_()
        if i == 3:
            args[3].sub_(7)                                        # lengths are looked at by every replay
        want = zn.mx_attention(*args, lse=True)
        out.zero_()
        g.replay()
        if i % 2:
            torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_the_most_requests_captured():
    lens, add, table, free, n_pages = step_case(8192, 16, 9, longest=40, new=3)
    total = int(add.sum())
    a = (i32(lens.tolist()), i32(add.tolist()), i32(table.tolist()), i32(free.tolist()), i32([len(free)]), 16, n_pages, total)
    want = zn.kv_extend(*a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = zn.kv_extend(*a)
        gone = zn.kv_release(got.lens, torch.ones(8192, dtype=torch.bool, device="cuda"), a[2], a[3].clone(), got.n_free, 16)
    for _ in range(3):
        for x in got:
            x.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and not gone[0].any()


def test_two_graphs_at_once():
    made = []
    for seed in (1, 2):
        q, c, table, _ = attend_case([7000, 900], None, 8, 2, 128, 64, "bf16", seed)
        args = (q, c, i32(table.tolist()), i32([7000, 900]))
        want = zn.mx_attention(*args)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = zn.mx_attention(*args)
        made.append((g, got, want, torch.cuda.Stream(), args))   # a graph's inputs live as long as it
    for _ in range(6):
        for g, got, want, s, _ in made:
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                got.zero_()
                g.replay()
        torch.cuda.synchronize()
        for g, got, want, s, _ in made:
            assert torch.equal(got, want)


# ------------------------------------------------- the kernels by their sizes --
# Which kernel takes a call goes by the sizes that the host sees, the table's width and the hint among them: wide tables
# send the cases above to kernels that their lengths would not choose.
def by_sizes(kind):
    attention = zn.mx_attention

    def call(q, c, table, lens, starts=None, max_new=0, **kw):
        kv_heads, page = c.k.shape[1:3]
        if kind == "few":        # waves of 16 rows that share out all tiles: a cache past 32 tiles, one query a request
            tiles, max_new = 40, 1
        else:                    # workgroups for 128 rows: many queries a request, 20480 tiles and more
            tiles, max_new = 20480 // kv_heads + 1, q.shape[0]
            if starts is None:
                starts = torch.arange(q.shape[0] + 1, dtype=torch.int32, device="cuda")
        width = max(-(-tiles * 64 // page), table.shape[1])
        wide = torch.full((table.shape[0], width), -1, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = table
        return attention(q, c, wide, lens, starts, max_new=max_new, **kw)
    return call


@pytest.mark.parametrize("kind", ["few", "many"])
@pytest.mark.parametrize("test,args", [
    *((test_attention_of_several_queries, ([300, 0, 20], [129, 0, 1], m, t)) for m in (dict(), dict(causal=False)) for t in TYPE),
    *((test_attention_of_several_queries, (lens, new, {}, t)) for lens, new in (([3, 200], [9, 33]), ([700], [700]),
                                                                             ([65, 64, 63, 130], [2, 64, 63, 100])) for t in TYPE),
    *((test_attention_of_long_caches, (lens, new, {}, t)) for lens, new in (([5000, 1, 2500], [4, 1, 2]), ([4100], [300]),
                                                                         ([9000, 4000], [20, 100])) for t in TYPE),
    *((test_attention_of_many_rows, ([700, 150, 0], [300, 150, 0], d)) for d in (32, 64, 96, 128, 256)),
    (test_attention_of_many_requests, (300,)), (test_attention_of_pages_and_orders, (128, "beside")),
    (test_attention_of_pages_and_orders, (16, "tokens")), (test_equal_weights_give_means, ()),
    *((test_scores_past_the_weights_precision, ([3000], [40], t)) for t in TYPE),
    *((test_what_a_query_does_not_see_has_no_effect, (t,)) for t in TYPE),
    *((test_values_of_many_sizes, (k,)) for k in ("near", "less near", "far", "rising", "zeros first", "one far block",
                                                  "far where nobody looks")),
    (test_small_values_beside_large_ones_keep_their_bits, ()), (test_many_small_weights_add_up, (40,)),
    (test_nans_among_the_largest_values, ()), (test_values_of_many_sizes_in_pieces, ()),
    (test_queries_that_are_not_finite_stay_by_themselves, ()), (test_rows_behind_the_last_request_stay, ()),
    *((test_a_serving_loop, (t,)) for t in TYPE)],
    ids=lambda x: x.__name__[5:] if callable(x) else "-".join(str(i).replace(" ", "") for i in x) if isinstance(x, tuple) else x)
def test_by_other_sizes(test, args, kind, monkeypatch):
    monkeypatch.setattr(zn, "mx_attention", by_sizes(kind))
    test(*args)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
def test_attention_of_every_head_size_and_kernel(dim, t, monkeypatch):
    for kind in ("few", "many"):
        monkeypatch.setattr(zn, "mx_attention", by_sizes(kind))
        run_attention([70, 0, 333], [40, 0, 33], 4, 2, dim, 16, t, dim)
        run_attention([3000], [40], 4, 2, dim, 64, t, dim)
        monkeypatch.undo()


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,new,kv_heads,window", [([300, 40, 0], [300, 40, 0], 64, 1), ([300, 40, 0], [300, 40, 0], 64, 50),
                                                      ([300, 40, 9], [299, 40, 1], 64, 5000), ([6000], [40], 96, 3000),
                                                      ([70, 500], [64, 40], 200, 130)])
def test_windows_of_many_heads(lens, new, kv_heads, window, t):
    q, c, table, starts = attend_case(lens, new, 2 * kv_heads, kv_heads, 32, 16, t, window)
    for hint in (1, max(new)):
        out, lse = zn.mx_attention(q, c, i32(table.tolist()), i32(lens), i32(starts), max_new=hint, window=window, lse=True)
        check_attention(q, c, table, lens, starts, 16, out, lse, window=window)


def test_kernels_of_many_rows_captured_and_replayed():
    for lens, new in (([500, 300], [90, 300]), ([6000, 40], [50, 40])):
        q, c, table, starts = attend_case(lens, new, 8, 2, 128, 64, "bf16", 1, spread=60)
        wide = torch.full((2, 11000), -1, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = i32(table.tolist())
        args = [q, c, wide, i32(lens), i32(starts)]
        zn.mx_attention(*args, lse=True)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out, lse = zn.mx_attention(*args, lse=True)
        for i in range(6):
            q.normal_()
            if i == 3:
                args[3].sub_(7)
            want = zn.mx_attention(*args, lse=True)
            out.zero_()
            g.replay()
            if i % 2:
                torch.cuda.synchronize()
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("new", [1, 40])
def test_the_largest_and_smallest_scales(new):
    # one key whose score is 1 among scores of 0, and weights that are all alike
    q, c, table, _ = attend_case([100], [new], 2, 1, 32, 16, "bf16", 9)
    q.zero_()
    q[:, :, 0] = 1.0
    c.k.zero_()
    c.k_scales.view(torch.uint8).fill_(127)
    c.k[table[0][3], 0, 2, 0] = 2                                  # 1.0, at 50
    v = torch.from_numpy(values(c)[1])
    seen = torch.stack([v[table[0][p // 16], 0, p % 16] for p in range(100)])
    for kind in ("few", "many"):
        args = (q, c, i32(table.tolist()), i32([100]), i32([0, new]))
        for attend in (zn.mx_attention, by_sizes(kind)):
            assert torch.equal(attend(*args, scale=2.0 ** 127, causal=False).cpu(), seen[50].bfloat16().expand(new, 2, 32))
            out = attend(*args, scale=2.0 ** -149, causal=False).cpu().double()
            # weights alike: sums of 100 within 100 2^-24 of the sum of sizes, a half step of the mean
            mean, size = seen.mean(0), seen.abs().mean(0)
            assert ((out - mean).abs() <= size * 100 * 2.0 ** -23 + mean.abs() * 2.0 ** -8 + 2.0 ** -24 * size).all()


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("dim", [32, 64, 96, 128, 160, 192, 224, 256])
def test_short_caches_of_many_heads(dim, t):
    # more groups of rows than workgroups of many waves run at a time, caches of eight tiles at most
    run_attention([300, 0, 77], None, 800, 400, dim, 16, t, dim)
    run_attention([300, 40, 0], [40, 40, 0], 192, 96, dim, 16, t, dim)
    run_attention([129, 500], [7, 20], 384, 96, dim, 64, t, dim, window=60)


def test_short_caches_of_many_heads_see_their_own():
    lens = [100, 45, 200]
    q, c, table, _ = attend_case(lens, None, 800, 400, 64, 16, "bf16", 8)
    tb = i32(table.tolist())
    want = zn.mx_attention(q, c, tb, i32(lens))
    vs = c.v_scales.view(torch.uint8)
    vs[table[0][60 // 16], 399, 60 % 16, 1] = 255                  # seen by one request's last heads
    vs[table[1][45 // 16], :, 45 % 16] = 255                       # behind a length
    out = zn.mx_attention(q, c, tb, i32(lens))
    nan = torch.zeros_like(out, dtype=torch.bool)
    nan[0, 798:, 32:] = True
    assert torch.equal(out.isnan(), nan) and torch.equal(out[~nan], want[~nan])
    bad = table.copy()
    bad[1, 2] = -1
    out = zn.mx_attention(q, c, i32(bad.tolist()), i32([100, 45, 10 ** 9]))
    assert out[1:].isnan().all() and torch.equal(out[0].isnan(), nan[0])
    now = i32(lens)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = zn.mx_attention(q, c, tb, now)
    for i in range(4):
        q.normal_()
        now.copy_(i32([100 - i, 45 + i, 200 - 50 * i]))
        want = zn.mx_attention(q, c, tb, now)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.isnan(), want.isnan()) and torch.equal(out.nan_to_num(), want.nan_to_num())
