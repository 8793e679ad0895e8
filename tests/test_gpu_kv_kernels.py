"""Every kernel of attention over every layout, page size, offset, mask and bad array; each case asks that its sizes
reach the kernel that it is for."""
import numpy as np
import pytest
import torch

from kv_kernels import KINDS, attention_by, widened
from kv_util import check_attention, f64, i32, random_cache, values
from lossless_float_weight_amd import zn
from oracle import kv
from test_gpu_kv import attend_case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zn.lib()


# lens, new, query heads and key heads that reach each kernel (two waves a workgroup want many groups of rows)
SHAPES = {"short": ([300, 45], [90, 45], 4, 2), "short pairs": ([300, 45], [9, 45], 300, 150),
          "few rows": ([300, 45, 2100], [90, 45, 3], 4, 2), "many rows": ([300, 45, 2100], [90, 45, 3], 4, 2)}


def make(kind, dim, page, t, seed, strides="pages", pad=0):
    lens, new, heads, kv_heads = SHAPES[kind]
    q, c, table, starts = attend_case(lens, new, heads, kv_heads, dim, page, t, seed, strides, pad)
    return q, c, i32(table.tolist()), lens, starts


def same(a, b):
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(), b.nan_to_num())


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("kind,strides,page", [
    (k, s, p) for k in KINDS for s, p in (("beside", 16), ("beside", 128), ("tokens", 32), ("tokens", 16), ("pages", 512))
    if k != "short pairs" or p < 512])                             # (such a page is more than two waves take)
def test_orders_and_pages(kind, strides, page, t):
    q, c, table, lens, starts = make(kind, 96, page, t, page, strides)
    for mask in (dict(), dict(causal=False)):
        out, lse = attention_by(kind)(q, c, table, i32(lens), i32(starts), lse=True, **mask)
        check_attention(q, c, table.cpu().numpy(), lens, starts, page, out, lse, **mask)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("kind,window", [("short", 1), ("short", 70), ("short pairs", 33), ("few rows", 2100), ("few rows", 2500)])
def test_windows(kind, window, t):
    q, c, table, lens, starts = make(kind, 64, 16, t, window)
    out, lse = attention_by(kind)(q, c, table, i32(lens), i32(starts), lse=True, window=window)
    check_attention(q, c, table.cpu().numpy(), lens, starts, 16, out, lse, window=window)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("window", [1, 100, 5000])
def test_windows_of_many_rows(window, t):
    # windows leave few tiles: this kernel takes them where heads are many
    q, c, table, starts = attend_case([700, 90, 400], [640, 90, 3], 128, 64, 32, 16, t, window)
    table = widened(i32(table.tolist()), 800)
    assert zn.debug_attention_kernel(q, c, table, i32(starts), 640, window) == "many rows"
    out, lse = zn.mx_attention(q, c, table, i32([700, 90, 400]), i32(starts), max_new=640, window=window, lse=True)
    check_attention(q, c, table.cpu().numpy(), [700, 90, 400], starts, 16, out, lse, window=window)


@pytest.mark.parametrize("kind", KINDS)
def test_rows_behind_the_last_request_stay(kind):
    q, c, table, lens, starts = make(kind, 64, 16, "bf16", 3, pad=9)
    n = starts[-1]
    for more, first in ((9, 0), (0, 0), (9, 7)):
        at = [s + first for s in starts]                          # rows before the first request stay too
        qq = q[:n + more] if not first else torch.cat([q[n:n + first], q[:n + 2]])
        out, lse = torch.full_like(qq, 7.0), torch.full(qq.shape[:2], 7.0, device="cuda")
        got = attention_by(kind)(qq, c, table, i32(lens), i32(at), out=out, lse=lse)
        assert got[0] is out and got[1] is lse
        for rows in (slice(0, first), slice(at[-1], None)):
            assert (out[rows] == 7).all() and (lse[rows] == 7).all()
        check_attention(qq, c, table.cpu().numpy(), lens, at, 16, out, lse)


@pytest.mark.parametrize("kind", KINDS)
def test_queries_and_results_of_any_stride(kind):
    q, c, table, lens, starts = make(kind, 64, 16, "bf16", 3)
    n, heads, _ = q.shape
    want = attention_by(kind)(q, c, table, i32(lens), i32(starts))
    wide = torch.zeros(n, heads + 3, 67, dtype=q.dtype, device="cuda")
    wide[:, 2:2 + heads, 3:] = q
    place = torch.full((heads + 2, n + 1, 65), 7.0, dtype=q.dtype, device="cuda")
    out = place.transpose(0, 1)[:n, :heads, 1:]
    attention_by(kind)(wide[:, 2:2 + heads, 3:], c, table, i32(lens), i32(starts), out=out)
    assert torch.equal(out, want)
    assert (place[:, :, 0] == 7).all() and (place[heads:] == 7).all() and (place[:, n:] == 7).all()


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", KINDS)
def test_bad_pages_and_lengths(kind, t):
    q, c, table, lens, starts = make(kind, 64, 16, t, 8)
    attend = attention_by(kind)
    want, want_lse = attend(q, c, table, i32(lens), i32(starts), lse=True)
    first = slice(0, starts[1])
    for page in (-1, c.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        bad = table.clone()
        bad[0, 230 // 16] = page                                  # seen from the position 224 on
        bad[1, 3:] = page                                         # behind the length: not looked at
        out, lse = attend(q, c, bad, i32(lens), i32(starts), lse=True)
        pos = torch.arange(lens[0] - starts[1], lens[0], device="cuda")
        gone = torch.cat([pos >= 224, torch.zeros(q.shape[0] - starts[1], dtype=torch.bool, device="cuda")])
        assert out[gone].isnan().all() and lse[gone].isnan().all()
        assert torch.equal(out[~gone], want[~gone]) and torch.equal(lse[~gone], want_lse[~gone])
    for n in (2 ** 31 - 1, 10 ** 6 * 16 + 1):
        out, lse = attend(q, c, table, i32([n] + lens[1:]), i32(starts), lse=True)
        assert out[first].isnan().all() and lse[first].isnan().all()
        check_attention(q[starts[1]:], c, table.cpu().numpy()[1:], lens[1:], [s - starts[1] for s in starts[1:]], 16, out[starts[1]:],
                        lse[starts[1]:])
    out, lse = attend(q, c, table, i32([-7] + lens[1:]), i32(starts), lse=True)
    assert (out[first] == 0).all() and (lse[first] == -torch.inf).all()
    # starts outside the queries are clamped
    far = [-5, *starts[1:-1], 2 ** 31 - 1]
    out = torch.full_like(q, 7.0)
    attend(q, c, table, i32(lens), i32(far), out=out)
    assert torch.equal(out, want)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", KINDS)
def test_what_a_query_does_not_see_has_no_effect(kind, t):
    q, c, table, lens, starts = make(kind, 64, 16, t, 8)
    attend = attention_by(kind)
    want, want_lse = attend(q, c, table, i32(lens), i32(starts), lse=True)
    tb = table.cpu().numpy()
    seen = torch.zeros(c.k.shape[0], 16, dtype=torch.bool)
    for row, n in zip(tb, lens):
        at = np.arange(n)
        seen[row[at // 16], at % 16] = True
    for s in (c.k_scales, c.v_scales):
        s.view(torch.uint8).masked_fill_(~seen.cuda()[:, None, :, None], 255)
    out, lse = attend(q, c, table, i32(lens), i32(starts), lse=True)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # a NaN at one key: whoever sees it, where it is
    last = c.k.shape[1] - 1
    group = q.shape[1] // c.k.shape[1]
    for s, key in ((c.v_scales, 250), (c.k_scales, 250)):
        u = s.view(torch.uint8)
        old = u.clone()
        u[tb[0][key // 16], last, key % 16, 1] = 254
        out = attend(q, c, table, i32(lens), i32(starts))
        pos = torch.arange(lens[0] - starts[1], lens[0], device="cuda")
        nan = torch.zeros_like(out, dtype=torch.bool)
        nan[:starts[1], last * group:, 0 if s is c.k_scales else 32:] = (pos >= key)[:, None, None]
        assert torch.equal(out.isnan(), nan) and torch.equal(out[~nan], want[~nan])
        u.copy_(old)


@pytest.mark.parametrize("fast", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_captured_and_replayed(kind, fast):
    q, c, table, lens, starts = make(kind, 128, 16, "bf16", 1)
    attend, now, at = attention_by(kind), i32(lens), i32(starts)
    attend(q, c, table, now, at, lse=True, fast_weights=fast)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, lse = attend(q, c, table, now, at, lse=True, fast_weights=fast)
    for i in range(6):
        q.normal_()
        if i == 3:
            now.sub_(7)
        if i == 4:
            table[0, 1].fill_(-1)
        want = attend(q, c, table, now, at, lse=True, fast_weights=fast)
        out.zero_()
        g.replay()
        if i % 2:
            torch.cuda.synchronize()
        assert same(out, want[0]) and same(lse, want[1])


@pytest.mark.parametrize("kind", KINDS)
def test_two_streams_at_once(kind):
    made = []
    for seed in (1, 2):
        q, c, table, lens, starts = make(kind, 128, 16, "bf16", seed)
        args = (q, c, table, i32(lens), i32(starts))
        made.append((args, attention_by(kind)(*args), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(4):
        got = [attention_by(kind)(*args, stream=s) for args, _, s in made]
        torch.cuda.synchronize()
        for x, (_, want, _) in zip(got, made):
            assert torch.equal(x, want)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
def test_the_largest_page(t):
    page = 65536
    c = random_cache(3, 2, page, 32, 3)
    g = torch.Generator().manual_seed(1)

    def check(kind, lens, new, table, **mask):
        starts = np.concatenate([[0], np.cumsum(new)]).tolist()
        q = torch.randn(starts[-1], 4, 32, generator=g).to(torch.bfloat16 if t == "bf16" else torch.float32).cuda()
        out, lse = attention_by(kind)(q, c, i32(table), i32(lens), i32(starts), lse=True, **mask)
        check_attention(q, c, np.array(table), lens, starts, page, out, lse, **mask)

    check("many rows", [66000, 5], [60, 5], [[2, 0], [1, -1]])
    check("few rows", [66000, 5], [2, 1], [[1, 2], [0, -1]])
    # (a page is more tiles than the others take, but for a window)
    check("short", [66000, 65536, 65537], [3, 2, 1], [[1, 2], [0, -1], [2, 0]], window=300)
    many = np.random.default_rng(0).integers(1, 2 * page, 450).tolist()
    check("short pairs", many, [1] * 450, [[b % 3, (b + 1) % 3] for b in range(450)], window=200)


def test_offsets_past_32_bits():
    heads, page, dim, n_pages = 8, 64, 128, 150000                 # 4.9 GB of codes each
    c, small = zn.mx_kv_cache(n_pages, heads, page, dim), zn.mx_kv_cache(48, heads, page, dim)
    rng = np.random.default_rng(0)
    high = np.concatenate([[n_pages - 1, 131073, 140001, 3], rng.permutation(np.arange(132000, n_pages - 1))[:44]])
    slots = torch.arange(48 * page, dtype=torch.int32, device="cuda")
    far = i32(high.tolist())[(slots // page).long()] * page + slots % page
    for x in range(2):
        k, v = (torch.from_numpy(rng.normal(0, 1, (48 * page, heads, dim))).bfloat16().cuda() for _ in range(2))
        for cache, at in ((c, far), (small, slots)):
            zn.mx_kv_write(k, v, cache, at)
        for a, b in zip(zn.mx_kv_read(c, far), zn.mx_kv_read(small, slots)):
            assert torch.equal(a, b)
    near = np.arange(48).reshape(8, 6)
    for kind, batch, new in (("short", 8, 3), ("short pairs", 100, 1), ("few rows", 8, 3), ("many rows", 8, 40)):
        lens = rng.integers(41, 6 * page, batch).tolist()
        lens[0] = 6 * page
        t = near[np.arange(batch) % 8]
        starts = i32((np.arange(batch + 1) * new).tolist())
        for dtype in (torch.bfloat16, torch.float32):
            q = torch.randn(batch * new, 16, dim, device="cuda").to(dtype)
            got = attention_by(kind)(q, c, i32(high[t].tolist()), i32(lens), starts)
            want = attention_by(kind)(q, small, i32(t.tolist()), i32(lens), starts)
            assert torch.equal(got, want), (kind, dtype)


def test_fast_weights_taken_again_in_a_piece():
    # one piece of many has values out of the first tile's reach and goes the other way, the others do not
    lens, new = [5000], [40]
    q, c, table, starts = attend_case(lens, new, 4, 2, 64, 64, "bf16", 9)
    c.v_scales.view(torch.uint8)[table[0][70], 0, 5, 0] = 60
    out, lse = attention_by("many rows")(q, c, i32(table.tolist()), i32(lens), i32(starts), lse=True, fast_weights=True)
    check_attention(q, c, table, lens, starts, 64, out, lse)


def test_a_loop_in_which_requests_are_refused():
    """Steps with more tokens than pages: some request is refused in one step and served in a later one, when others end."""
    heads, kv_heads, dim, page, batch, width, n_pages = 4, 2, 64, 16, 4, 6, 10
    rng = np.random.default_rng(0)
    c = random_cache(n_pages, kv_heads, page, dim, 1)
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    free, n_free, lens = torch.arange(n_pages, dtype=torch.int32, device="cuda"), i32([n_pages]), i32([0] * batch)
    held = [np.zeros((0, 2, kv_heads, dim)) for _ in range(batch)]
    refused = served_later = 0
    waits = set()
    for add, done in (([40, 30, 64, 20], []), ([10, 5, 1, 20], []), ([1, 1, 1, 20], [0]), ([90, 3, 30, 1], []), ([97, 1, 1, 1], [2])):
        lens, n_free = zn.kv_release(lens, torch.tensor([b in done for b in range(batch)], device="cuda"), table, free, n_free, page)
        for b in done:
            held[b] = held[b][:0]
        total = sum(add)
        before = [int(x) for x in lens.tolist()]
        want = kv.extend(before, add, table.tolist(), free.tolist(), n_free.item(), page, n_pages, total)
        step = zn.kv_extend(lens, i32(add), table, free, n_free, page, n_pages, total)
        assert step.lens.tolist() == want[0] and step.slots.tolist() == want[2] and table.tolist() == want[5]
        k, v, q = (torch.from_numpy(rng.normal(0, 1, (total, h, dim))).bfloat16().cuda() for h in (kv_heads, kv_heads, heads))
        zn.mx_kv_write(k, v, c, step.slots)
        out = zn.mx_attention(q, c, table, step.lens, step.starts, max_new=max(add))
        lens, n_free = step.lens, step.n_free
        stored = np.stack([kv.values(*kv.rows(f64(x))) for x in (k, v)], 1)
        at = np.concatenate([[0], np.cumsum(add)])
        for b in range(batch):
            if want[0][b] == before[b]:
                refused += 1
                waits.add(b)
                assert (step.slots[at[b]:at[b + 1]] == -1).all()
                continue
            served_later += b in waits
            waits.discard(b)
            held[b] = np.concatenate([held[b], stored[at[b]:at[b + 1]]])
        kk, vv = values(c)
        tb = table.cpu().numpy()
        for b in range(batch):                                      # a refused request's tokens are left as they were
            i = np.arange(want[0][b])
            for x, j in ((kk, 0), (vv, 1)):
                np.testing.assert_array_equal(x[tb[b][i // page], :, i % page], held[b][:, j])
        check_attention(q, c, tb, want[0], at.tolist(), page, out)
    assert refused >= 2 and served_later >= 1


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["few rows", "many rows"])
def test_the_most_heads(kind, t):
    # 1024 key heads leave one to four waves, or pieces of work, for each
    lens, new = [200, 0, 70, 33], [40, 0, 70, 2]
    q, c, table, starts = attend_case(lens, new, 1024, 1024, 32, 16, t, 5)
    out, lse = attention_by(kind)(q, c, i32(table.tolist()), i32(lens), i32(starts), lse=True)
    for h in (slice(0, 3), slice(127, 130), slice(510, 514), slice(769, 771), slice(1021, 1024)):
        part = zn.MxCache(*(x[:, h] for x in c))
        check_attention(q[:, h], part, table, lens, starts, 16, out[:, h], lse[:, h])


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["short pairs", "few rows", "many rows"])
def test_the_most_requests(kind, t):
    rng = np.random.default_rng(2)
    lens = rng.integers(0, 60, 8192).tolist()
    new = rng.integers(0, 3, 8192).tolist()
    if kind != "short pairs":
        lens[17], lens[8191] = 3000, 2500
    if kind == "many rows":
        new[17], new[8000] = 200, 33
    pool = 400                                                     # pages that requests share
    c = random_cache(pool, 1, 16, 32, 4)
    width = -(-max(lens) // 16)
    table = rng.integers(0, pool, (8192, width))
    starts = np.concatenate([[0], np.cumsum(new)])
    q = torch.randn(int(starts[-1]), 2, 32, generator=torch.Generator().manual_seed(1)).to(
        torch.bfloat16 if t == "bf16" else torch.float32).cuda()
    out, lse = attention_by(kind)(q, c, i32(table.tolist()), i32(lens), i32(starts.tolist()), lse=True)
    check_attention(q, c, table, lens, starts.tolist(), 16, out, lse)
