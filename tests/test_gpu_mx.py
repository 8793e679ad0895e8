"""The microscaled operators on the GPU against the 64-bit oracle.

What is exact is compared bit by bit: the quantiser, reading back, the stored
sum of the norm, and products whose terms and sums are small whole numbers.
The rest is held to bounds derived here:
  * norm: codes and scales are those of the formula in 64 bits, up to its own
    roundings (sums of another order, under 2^-40 relative for these rows), and
    rounding is monotone: the code lies between those of y (1 - 2^-40) and
    y (1 + 2^-40) under the scale that was chosen, and that scale between theirs;
  * product: every FP32 addition of the K terms and partial sums rounds (or
    cuts) by at most 2^-23 of a partial sum, which is at most the sum of the
    terms' magnitudes S: K 2^-23 S, and the output's rounding, half a step.
"""
import numpy as np
import pytest
import torch

from lossless_float_weight_amd import zn
from oracle import mx

pytestmark = pytest.mark.gpu

FMT = {"fp8": zn.FP8_E4M3, "fp4": zn.FP4X2_E2M1}
TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    zn.lib()


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def f64(t):
    return t.to(torch.float64).cpu().numpy()


def cuda(a, t):
    """float64 numpy values that `t` holds exactly, on the GPU."""
    x = torch.from_numpy(np.ascontiguousarray(a))
    y = x.to(t)
    assert torch.equal(y.double().nan_to_num(0.5), x.nan_to_num(0.5))
    return y.cuda()


def rounded(a, t):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float64)).to(torch.float32).to(t)


def sample(rows, k, t, seed):
    """Rows of many sizes with zeros of both signs, exact ties, tiny and huge values."""
    rng = np.random.default_rng(seed)
    x = rng.normal(0, 1, (rows, k)) * np.exp2(rng.integers(-12, 12, (rows, 1)))
    pick = rng.random((rows, k))
    x = np.where(pick < 0.1, np.round(x * 4) / 4, x)
    x = np.where(pick > 0.97, 0.0, x)
    x = np.where(pick > 0.985, -0.0, x)
    x = np.where((pick > 0.5) & (pick < 0.502), x * 2.0 ** -120, x)
    x = np.where((pick > 0.6) & (pick < 0.602), x * 2.0 ** 100, x)
    if rows > 2:
        x[1] = 0.0
    return rounded(x, TYPE[t])


def same_quantized(x, fmt, codes, scales):
    want, s = mx.quantize(f64(x).reshape(-1, x.shape[-1]), fmt)
    np.testing.assert_array_equal(raw(scales).reshape(s.shape), s)
    np.testing.assert_array_equal(raw(codes).reshape(want.shape), want)


SHAPES = [(1, 1), (1, 32), (3, 33), (5, 100), (2, 4096), (64, 64), (17, 2883), (9, 16392), (300, 8)]


# ---------------------------------------------------------------- quantise --
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_quantize_equals_oracle(shape, t, fmt):
    x = sample(*shape, t, 11)
    codes, scales = zn.mx_quantize(x.cuda(), FMT[fmt])
    assert codes.dtype == (torch.float8_e4m3fn if fmt == "fp8" else torch.uint8)
    same_quantized(x, fmt, codes, scales)


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("order", ["sorted", "shuffled"])
def test_quantize_every_bf16_pattern(fmt, order):
    bits = np.arange(65536, dtype=np.uint16)
    if order == "shuffled":
        bits = np.random.default_rng(3).permutation(bits)
    x = torch.from_numpy(bits.astype(np.int32)).to(torch.int16).view(torch.bfloat16).view(64, 1024)
    for t in ("bf16", "fp32"):
        y = x.to(TYPE[t])
        same_quantized(y, fmt, *zn.mx_quantize(y.cuda(), FMT[fmt]))


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_quantize_ties_of_every_binade_and_their_neighbours(fmt):
    # midpoints of the grid and the next FP32 values on both sides, under block
    # maxima that fix the scale at several powers of two, subnormal ones too
    g = mx.grid(fmt)[:127 if fmt == "fp8" else 8]
    mids = ((g[1:] + g[:-1]) / 2).astype(np.float32)
    v = np.concatenate([mids, np.nextafter(mids, np.float32(0)), np.nextafter(mids, np.float32(np.inf)), g.astype(np.float32)])
    v = np.concatenate([v, -v])
    v = np.concatenate([v, np.zeros(-len(v) % 31, np.float32)]).reshape(-1, 31)
    top = np.full((len(v), 1), g[-1], np.float32)
    x = np.concatenate([top, v], 1).astype(np.float64)
    e = np.arange(-130, 119, 3)
    x = (x[None] * np.exp2(e)[:, None, None]).reshape(-1, 32)
    x = torch.from_numpy(x).to(torch.float32)
    same_quantized(x, fmt, *zn.mx_quantize(x.cuda(), FMT[fmt]))


def test_quantize_non_finite_blocks():
    x = sample(6, 160, "fp32", 5)
    x[0, 3], x[2, 64], x[3, 159], x[5, :] = float("inf"), float("nan"), float("-inf"), float("nan")
    for fmt in FMT:
        for y in (x, x.bfloat16()):
            codes, scales = zn.mx_quantize(y.cuda(), FMT[fmt])
            same_quantized(y, fmt, codes, scales)
            back = zn.mx_dequantize(codes, scales)
            assert bool(back[5].isnan().all()) and bool(back[0, :32].isnan().all()) and not bool(back[0, 32:].isnan().any())


def test_quantize_row_views():
    x = sample(24, 200, "bf16", 7).cuda()
    views = [x[:, :100], x[:, 1:102], x[::3], x[:, 8:136], x[5], x[:1].expand(7, 200), x.view(2, 12, 200),
             x.view(-1)[1:4097].view(2, 2048), x[:, 7:8], x[:0], x.view(4, 6, 200)[:, :, 40:72]]
    for v in views:
        for fmt in FMT:
            codes, scales = zn.mx_quantize(v, FMT[fmt])
            assert codes.shape[:-1] == v.shape[:-1] and scales.shape[:-1] == v.shape[:-1]
            if v.numel():
                same_quantized(v, fmt, codes, scales)
    y = x.float()
    same_quantized(y[:, 3:99], "fp8", *zn.mx_quantize(y[:, 3:99], zn.FP8_E4M3))


def test_quantize_into_given_buffers_leaves_the_rest():
    x = sample(3, 40, "fp32", 9)
    codes = torch.full((5, 64), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((5, 2), 0x55, dtype=torch.uint8, device="cuda")
    got = zn.mx_quantize(x.cuda(), zn.FP8_E4M3, codes=codes[1:4].view(torch.float8_e4m3fn), scales=scales[1:4])
    same_quantized(x, "fp8", *got)
    for b in (codes, scales):
        assert bool((b[0] == 0x55).all()) and bool((b[4] == 0x55).all())


def test_quantize_past_two_to_the_31_elements():
    # offsets of elements pass 2^31, of bytes 2^32; the first and the last rows are checked
    rows, k = 131073, 16416
    x = torch.zeros(rows, k, dtype=torch.bfloat16, device="cuda")
    ends = sample(8, k, "bf16", 13)
    x[:4], x[-4:] = ends[:4].cuda(), ends[4:].cuda()
    codes, scales = zn.mx_quantize(x, zn.FP4X2_E2M1)
    for part, e in ((slice(0, 4), ends[:4]), (slice(rows - 4, rows), ends[4:])):
        same_quantized(e, "fp4", codes[part], scales[part])
    back = zn.mx_dequantize(codes, scales, dtype=torch.bfloat16)
    want = mx.values(raw(codes[-4:]), raw(scales[-4:]), "fp4")
    np.testing.assert_array_equal(f64(back[-4:]), f64(rounded(want, torch.bfloat16)))
    assert not bool(scales.view(torch.uint8)[4:-4].any())


# -------------------------------------------------------------------- read --
def read_back(want, t):
    """float64 -> the type by one rounding (float64 -> BF16 here goes through FP32, which holds every value exactly)."""
    with np.errstate(over="ignore"):
        w = torch.from_numpy(want.astype(np.float32))
    return w.to(TYPE[t]).to(torch.float64).numpy()


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
def test_dequantize_every_code_under_every_scale(fmt, t):
    n = 256 if fmt == "fp8" else 16
    codes = mx.pack(np.tile(np.arange(n, dtype=np.uint8), (256, 32 // 16 if fmt == "fp4" else 1)), fmt)
    nb = 1 if fmt == "fp4" else 8
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], nb, 1)
    c = torch.from_numpy(codes).cuda()
    c = c.view(torch.float8_e4m3fn) if fmt == "fp8" else c
    got = zn.mx_dequantize(c, torch.from_numpy(s).cuda(), dtype=TYPE[t])
    np.testing.assert_array_equal(f64(got), read_back(mx.values(codes, s, fmt), t))


@pytest.mark.parametrize("shape", SHAPES)
def test_dequantize_lengths_and_outputs(shape):
    rows, k = shape
    x = sample(rows, k, "bf16", 15)
    for fmt in FMT:
        codes, scales = zn.mx_quantize(x.cuda(), FMT[fmt])
        want = mx.values(raw(codes), raw(scales), fmt)
        for t in TYPE:
            got = zn.mx_dequantize(codes, scales, k=k, dtype=TYPE[t])
            np.testing.assert_array_equal(f64(got), read_back(want[:, :k], t))
            wide = torch.full((rows + 2, k + 5), 7.0, dtype=TYPE[t], device="cuda")
            zn.mx_dequantize(codes, scales, k=k, out=wide[1:-1, 2:2 + k])
            np.testing.assert_array_equal(f64(wide[1:-1, 2:2 + k]), read_back(want[:, :k], t))
            wide[1:-1, 2:2 + k] = 7.0
            assert bool((wide == 7.0).all())


# -------------------------------------------------------------------- norm --
def between(y, fmt, codes, scales):
    """Codes and scales of y within the bounds of the module's text."""
    d = 2.0 ** -40
    s = raw(scales).reshape(len(y), -1)
    b = mx.blocks(y)
    with np.errstate(invalid="ignore", over="ignore"):
        lo, hi = mx.scale_bytes(b * (1 - d), fmt), mx.scale_bytes(b * (1 + d), fmt)
    assert ((lo <= s) & (s <= hi)).all(), "scale"
    c = mx.unpack(raw(codes).reshape(len(y), -1), fmt)
    dead = s == 255
    v = mx.grid(fmt)[c].reshape(b.shape)
    assert (v[dead] == 0).all()
    unit = mx.scale_value(np.where(dead, 127, s))[..., None]
    q = np.where(dead[..., None], 0.0, b) / unit
    ends = [mx.grid(fmt)[mx.nearest(q * f, fmt)] for f in (1 - d, 1 + d)]
    assert ((np.minimum(*ends) <= v) & (v <= np.maximum(*ends)))[~dead].all(), "codes"


NORM_SHAPES = [(1, 1), (3, 31), (5, 33), (70, 512), (3, 513), (9, 1024), (2, 1032), (3, 2048), (2, 2056), (1, 4096),
               (5, 4100), (3, 8192), (2, 8200), (2, 16384), (2, 16392), (3, 40001), (5000, 40)]


@pytest.mark.parametrize("add", [True, False])
@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", NORM_SHAPES)
def test_norm(shape, t, add):
    rows, k = shape
    rng = np.random.default_rng(k)
    x = rounded(rng.normal(0, 1, shape) * np.exp2(rng.integers(-6, 6, (rows, 1))), TYPE[t])
    r = rounded(rng.normal(0, 1, shape), TYPE[t])
    w = rounded(1 + 0.3 * rng.normal(0, 1, k), TYPE[t])
    h = (x.float() + r.float()).to(TYPE[t]) if add else x
    y = mx.rms_norm(f64(h), f64(w), float(np.float32(1e-5)))
    for fmt in FMT:
        codes, scales, got = zn.mx_rms_norm(x.cuda(), w.cuda(), residual=r.cuda() if add else None, eps=1e-5, fmt=FMT[fmt])
        assert torch.equal(got.cpu(), h)
        between(y, fmt, codes, scales)


@pytest.mark.parametrize("t", ["bf16", "fp32"])
@pytest.mark.parametrize("k", [96, 4096, 20000])
def test_norm_in_place_and_views(t, k):
    rng = np.random.default_rng(k)
    big = rounded(rng.normal(0, 1, (12, k + 24)), TYPE[t]).cuda()
    r = rounded(rng.normal(0, 1, (6, k)), TYPE[t]).cuda()
    w = rounded(rng.normal(1, 0.1, k), TYPE[t]).cuda()
    for x in (big[::2, 8:8 + k], big[::2, 3:3 + k], big[:6, :k]):
        c, s, h = zn.mx_rms_norm(x, w, residual=r)
        between(mx.rms_norm(f64(h), f64(w), float(np.float32(1e-5))), "fp8", c, s)
        for into in ("x", "residual"):
            a, b = big.clone(), r.clone()
            xa = torch.as_strided(a, x.shape, x.stride(), x.storage_offset())
            c2, s2, h2 = zn.mx_rms_norm(xa, w, residual=b, residual_out=xa if into == "x" else b)
            assert torch.equal(h2, h) and np.array_equal(raw(c2), raw(c)) and np.array_equal(raw(s2), raw(s))
            if into == "x":
                xa.copy_(x)
            assert torch.equal(a, big)          # nothing beside the rows was written


@pytest.mark.parametrize("k", [64, 4096, 33000])
def test_norm_extreme_rows(k):
    rng = np.random.default_rng(k)
    z = rng.normal(0, 1, (8, k))
    x = np.stack([z[0] * 2.0 ** 100, z[1] * 2.0 ** -120, np.full(k, 3.0 * 2.0 ** 126), np.zeros(k), z[4], z[5], z[6] * 2.0 ** -70, z[7]])
    x = rounded(x, torch.float32)
    w = rounded(np.ones(k), torch.float32)
    for t in TYPE:
        xt = x.to(TYPE[t])
        for eps in (0.0, 1e-5):
            c, s, _ = zn.mx_rms_norm(xt.cuda(), w.to(TYPE[t]).cuda(), eps=eps)
            y = mx.rms_norm(f64(xt), np.ones(k), float(np.float32(eps)))
            between(y, "fp8", c, s)              # a row of zeros under eps 0 is NaN throughout
            assert (raw(s)[3] == (255 if eps == 0 else 0)).all()
    # an infinity makes its own block NaN and the rest zero; a NaN the whole row
    xt = x.clone()
    xt[4, k // 2], xt[5, 0] = float("inf"), float("nan")
    c, s, _ = zn.mx_rms_norm(xt.cuda(), w.cuda())
    back = zn.mx_dequantize(c, s, dtype=torch.float32).cpu()
    blk = k // 2 // 32
    assert bool(back[4, 32 * blk:32 * blk + 32].isnan().all()) and bool(back[5].isnan().all())
    back[4, 32 * blk:32 * blk + 32] = 0
    assert bool((back[4] == 0).all()) and not bool(back[6:].isnan().any())


# ----------------------------------------------------------------- product --
def whole(rows, k, fmt, seed):
    """Codes of small whole numbers and scales 2^-1 .. 2^1: sums stay exact in FP32."""
    rng = np.random.default_rng(seed)
    g = mx.grid(fmt)
    ok = [c for c in range(len(g)) if g[c] in (-4, -3, -2, -1, 0, 1, 2, 3, 4)]
    c = mx.pack(rng.choice(np.array(ok, np.uint8), (rows, k)), fmt)
    s = rng.integers(126, 129, (rows, k // 32)).astype(np.uint8)
    return c, s


def up(c, fmt):
    t = torch.from_numpy(c).cuda()
    return t.view(torch.float8_e4m3fn) if fmt == "fp8" else t


PRODUCTS = [(1, 1, 32), (1, 16, 128), (1, 100, 96), (2, 17, 160), (15, 33, 352), (16, 64, 512), (17, 300, 2016),
            (33, 31, 1056), (48, 130, 4096), (64, 128, 1024), (65, 1000, 224), (100, 257, 3104), (128, 128, 128),
            (129, 255, 640), (200, 513, 1120), (256, 256, 256), (257, 300, 2016), (513, 770, 416), (1000, 1030, 1184),
            (1025, 2300, 160), (2049, 1700, 384), (3600, 3650, 288), (4096, 3800, 512), (4300, 4090, 160)]


@pytest.mark.parametrize("fmts", ["fp8 fp8", "fp8 fp4", "fp4 fp8", "fp4 fp4"])
@pytest.mark.parametrize("size", PRODUCTS)
def test_product_of_whole_numbers_is_exact(size, fmts):
    # every term is a multiple of 1/4 and at most 64, so sums of up to 4096
    # terms are whole multiples of 1/4 below 2^20: exact in FP32 in any order
    (m, n, k), (fa, fw) = size, fmts.split()
    (a, sa), (w, sw) = whole(m, k, fa, m + k), whole(n, k, fw, n + k + 1)
    want = mx.matmul(mx.values(a, sa, fa), mx.values(w, sw, fw))
    assert np.abs(want).max() < 2 ** 18
    args = (up(a, fa), torch.from_numpy(sa).cuda(), up(w, fw), torch.from_numpy(sw).cuda())
    np.testing.assert_array_equal(f64(zn.mx_matmul(*args, dtype=torch.float32)), want)
    got = zn.mx_matmul(*args)
    np.testing.assert_array_equal(f64(got), f64(rounded(want, torch.bfloat16)))
    # rows apart, and nothing written beside them
    for t in TYPE:
        wide = torch.full((m + 2, n + 3), 7.0, dtype=TYPE[t], device="cuda")
        zn.mx_matmul(*args, out=wide[1:-1, 1:n + 1])
        np.testing.assert_array_equal(f64(wide[1:-1, 1:n + 1]), f64(rounded(want, TYPE[t])))
        wide[1:-1, 1:n + 1] = 7.0
        assert bool((wide == 7.0).all())


@pytest.mark.parametrize("fmts", ["fp8 fp8", "fp8 fp4", "fp4 fp8", "fp4 fp4"])
@pytest.mark.parametrize("size", [(1, 64, 4096), (7, 96, 14336), (40, 200, 14336), (80, 160, 4128), (300, 520, 4096)])
def test_product_of_random_numbers(size, fmts):
    (m, n, k), (fa, fw) = size, fmts.split()
    rng = np.random.default_rng(k + m)
    a, sa = mx.quantize(rng.normal(0, 1, (m, k)) * np.exp2(rng.integers(-3, 3, (m, 1))), fa)
    w, sw = mx.quantize(rng.normal(0, 0.02, (n, k)), fw)
    va, vw = mx.values(a, sa, fa), mx.values(w, sw, fw)
    want, size_ = mx.matmul(va, vw), mx.matmul(np.abs(va), np.abs(vw))
    args = (up(a, fa), torch.from_numpy(sa).cuda(), up(w, fw), torch.from_numpy(sw).cuda())
    bound = k * 2.0 ** -23 * size_
    assert (np.abs(f64(zn.mx_matmul(*args, dtype=torch.float32)) - want) <= bound + 2.0 ** -24 * np.abs(want)).all()
    assert (np.abs(f64(zn.mx_matmul(*args)) - want) <= bound + 2.0 ** -8 * (np.abs(want) + bound)).all()


@pytest.mark.parametrize("fmts", ["fp8 fp8", "fp8 fp4", "fp4 fp8"])
@pytest.mark.parametrize("size", [(1, 80), (40, 80), (300, 80), (1030, 2050), (2600, 2570)])
def test_product_fp32_keeps_what_lies_far_below_a_neighbour(size, fmts):
    # every eighth product is 256, the others 2^-8, 16 bits below: the sum of 256
    # of them, 8192.875, and every partial sum have at most 22 bits
    (m, n), (fa, fw) = size, fmts.split()
    k = 256
    far = np.where(np.arange(k) % 8 == 0, 0x78, 0x02).astype(np.uint8)
    one8, one4 = np.full(k, 0x38, np.uint8), np.full(k // 2, 0x22, np.uint8)
    a = np.tile(far if fa == "fp8" else one4, (m, 1))
    w = np.tile((one8 if fa == "fp8" else far) if fw == "fp8" else one4, (n, 1))
    sa, sw = (torch.full((r, k // 32), 127, dtype=torch.uint8, device="cuda") for r in (m, n))
    got = zn.mx_matmul(up(a, fa), sa, up(w, fw), sw, dtype=torch.float32)
    assert bool((got == 8192.875).all())


@pytest.mark.parametrize("size", [(3, 40, 224), (300, 300, 224)])
def test_product_scales_of_all_sizes(size):
    # one nonzero block a row: products of the extreme scales, which leave FP32's range at both ends
    m, n, k = size
    a = np.zeros((m, k), np.uint8)
    w = np.zeros((n, k), np.uint8)
    a[:, 64:96], w[:, 64:96] = 0x38, 0x38           # ones
    sa = np.full((m, k // 32), 127, np.uint8)
    sw = np.full((n, k // 32), 127, np.uint8)
    sa[:, 2] = np.linspace(0, 254, m).astype(np.uint8)
    sw[:, 2] = np.linspace(0, 254, n).astype(np.uint8)
    got = f64(zn.mx_matmul(up(a, "fp8"), torch.from_numpy(sa).cuda(), up(w, "fp8"), torch.from_numpy(sw).cuda(), dtype=torch.float32))
    want = mx.matmul(mx.values(a, sa, "fp8"), mx.values(w, sw, "fp8"))
    normal = (np.abs(want) >= 2.0 ** -126) & (np.abs(want) < 2.0 ** 128)
    np.testing.assert_array_equal(got[normal], want[normal])
    assert np.isinf(got[want >= 2.0 ** 128]).all()
    assert (got[want < 2.0 ** -126] <= 2.0 ** -126).all()


@pytest.mark.parametrize("fmts", ["fp8 fp8", "fp8 fp4", "fp4 fp8", "fp4 fp4"])
@pytest.mark.parametrize("size", [(1, 40, 224), (20, 40, 224), (300, 280, 1184)])
def test_product_nans_stay_in_their_rows(size, fmts):
    (m, n, k), (fa, fw) = size, fmts.split()
    (a, sa), (w, sw) = whole(m, k, fa, 1), whole(n, k, fw, 2)
    want = mx.matmul(mx.values(a, sa, fa), mx.values(w, sw, fw))
    sa[m // 2, -1] = 255
    sw[n - 1, 0] = 255
    if fw == "fp8":
        w[3, k - 1] = 0x7F
    got = f64(zn.mx_matmul(up(a, fa), torch.from_numpy(sa).cuda(), up(w, fw), torch.from_numpy(sw).cuda(), dtype=torch.float32))
    bad = np.zeros((m, n), bool)
    bad[m // 2], bad[:, n - 1] = True, True
    if fw == "fp8":
        bad[:, 3] = True
    assert np.isnan(got[bad]).all()
    np.testing.assert_array_equal(got[~bad], want[~bad])


@pytest.mark.parametrize("m", [3, 40, 300])
def test_product_scales_at_any_address(m):
    # k a multiple of 512 (scale rows of 16 bytes) and not, scale bytes one past an aligned address
    for k in (512, 96):
        (a, sa), (w, sw) = whole(m, k, "fp8", 3), whole(50, k, "fp4", 4)
        off = []
        for s in (sa, sw):
            b = torch.zeros(s.size + 1, dtype=torch.uint8, device="cuda")
            b[1:] = torch.from_numpy(s.reshape(-1)).cuda()
            off.append(b[1:].view(s.shape))
        got = zn.mx_matmul(up(a, "fp8"), off[0], up(w, "fp4"), off[1], dtype=torch.float32)
        np.testing.assert_array_equal(f64(got), mx.matmul(mx.values(a, sa, "fp8"), mx.values(w, sw, "fp4")))


def test_product_takes_the_scratch_it_asks_for():
    m, n, k = 40, 300, 8224           # pieces of k and scale rows of 257 bytes
    need = zn.mx_matmul_scratch_bytes(zn.FP8_E4M3, zn.FP4X2_E2M1, m, n, k)
    assert need > 0
    (a, sa), (w, sw) = whole(m, k, "fp8", 3), whole(n, k, "fp4", 4)
    args = (up(a, "fp8"), torch.from_numpy(sa).cuda(), up(w, "fp4"), torch.from_numpy(sw).cuda())
    buf = torch.full((need + 64,), 0x55, dtype=torch.uint8, device="cuda")
    got = zn.mx_matmul(*args, dtype=torch.float32, scratch=buf[:need])
    np.testing.assert_array_equal(f64(got), mx.matmul(mx.values(a, sa, "fp8"), mx.values(w, sw, "fp4")))
    assert bool((buf[need:] == 0x55).all())
    with pytest.raises(zn.ZnError):
        zn.mx_matmul(*args, scratch=buf[:need - 1])


@pytest.mark.parametrize("m", [1, 20])
def test_product_of_very_long_rows(m):
    # rows past what a tile addresses; ones by ones, a sum of at most 24 bits
    k, n = (1 << 21) + 32, 17
    a = torch.full((m, k), 0x38, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    w = torch.full((n, k // 2), 0x22, dtype=torch.uint8, device="cuda")
    sa, sw = (torch.full((r, k // 32), 127, dtype=torch.uint8, device="cuda") for r in (m, n))
    assert bool((zn.mx_matmul(a, sa, w, sw, dtype=torch.float32) == k).all())


def test_product_shapes_and_empty_sides():
    a, sa = whole(6, 64, "fp8", 1)
    w, sw = whole(10, 64, "fp4", 2)
    A, SA, W, SW = up(a, "fp8"), torch.from_numpy(sa).cuda(), up(w, "fp4"), torch.from_numpy(sw).cuda()
    want = mx.matmul(mx.values(a, sa, "fp8"), mx.values(w, sw, "fp4"))
    got = zn.mx_matmul(A.view(2, 3, 64), SA.view(2, 3, 2), W, SW, dtype=torch.float32)
    assert got.shape == (2, 3, 10)
    np.testing.assert_array_equal(f64(got).reshape(6, 10), want)
    got = zn.mx_matmul(A[1], SA[1].view(torch.float8_e8m0fnu), W, SW.view(torch.float8_e8m0fnu), dtype=torch.float32)
    np.testing.assert_array_equal(f64(got), want[1])
    assert zn.mx_matmul(A[:0], SA[:0], W, SW).shape == (0, 10)
    assert zn.mx_matmul(A, SA, W[:0], SW[:0]).shape == (6, 0)
    with pytest.raises(zn.ZnError):
        zn.mx_matmul(A, SA, W, SW, out=torch.empty(6, 11, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(zn.ZnError):
        zn.mx_matmul(A, SA, W, SW, out=torch.empty(6, 10, dtype=torch.float16, device="cuda"))
    with pytest.raises(zn.ZnError):
        zn.mx_matmul(A, SA, W.cpu(), SW)


# --------------------------------------------------- streams, graphs, chain --
def _setting(m, n, k, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(m, k, device="cuda", generator=g).bfloat16()
    r = torch.randn(m, k, device="cuda", generator=g).bfloat16()
    nw = (1 + 0.1 * torch.randn(k, device="cuda", generator=g)).bfloat16()
    w = (0.02 * torch.randn(n, k, device="cuda", generator=g)).bfloat16()
    return x, r, nw, w


@pytest.mark.parametrize("size", [(1, 512, 4096), (40, 384, 8192), (300, 640, 4096)])
def test_on_another_stream(size):
    m, n, k = size
    x, r, nw, w = _setting(m, n, k)
    q = zn.mx_quantize(w, zn.FP4X2_E2M1)
    c, s, h = zn.mx_rms_norm(x, nw, residual=r)
    want = zn.mx_matmul(c, s, *q)
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for i in range(6):
        st = side[i % 2]
        q2 = zn.mx_quantize(w, zn.FP4X2_E2M1, stream=st)
        c2, s2, h2 = zn.mx_rms_norm(x, nw, residual=r, stream=st)
        got.append((zn.mx_matmul(c2, s2, *q2, stream=st), h2, zn.mx_dequantize(*q2, stream=st)))
    torch.cuda.synchronize()
    for o, h2, back in got:
        assert torch.equal(o, want) and torch.equal(h2, h) and torch.equal(back, zn.mx_dequantize(*q))


@pytest.mark.parametrize("size", [(1, 512, 4096), (40, 384, 8192), (300, 640, 4096)])
def test_captured_and_replayed(size):
    m, n, k = size
    x, r, nw, w = _setting(m, n, k)
    q = zn.mx_quantize(w, zn.FP4X2_E2M1)
    zn.mx_matmul(*zn.mx_rms_norm(x, nw, residual=r)[:2], *q)
    graphs = []
    for _ in range(2):                       # two graphs, each with scratch of its own
        xs, rs = x.clone(), r.clone()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c, s, _h = zn.mx_rms_norm(xs, nw, residual=rs, residual_out=rs)
            o = zn.mx_matmul(c, s, *q)
        graphs.append((g, xs, rs, o))
    for step in range(4):
        for i, (g, xs, rs, o) in enumerate(graphs):
            nx, nr, _, _ = _setting(m, n, k, seed=10 * step + i)
            xs.copy_(nx)
            rs.copy_(nr)
            g.replay()
        torch.cuda.synchronize()
        for i, (g, xs, rs, o) in enumerate(graphs):
            nx, nr, _, _ = _setting(m, n, k, seed=10 * step + i)
            c, s, h = zn.mx_rms_norm(nx, nw, residual=nr)
            assert torch.equal(rs, h) and torch.equal(o, zn.mx_matmul(c, s, *q))


def test_results_do_not_depend_on_the_run():
    for m, n, k in ((1, 300, 14336), (50, 300, 14336), (300, 300, 4096)):
        x, r, nw, w = _setting(m, n, k)
        q = zn.mx_quantize(w, zn.FP4X2_E2M1)
        c, s, _ = zn.mx_rms_norm(x, nw, residual=r)
        first = zn.mx_matmul(c, s, *q, dtype=torch.float32)
        for _ in range(5):
            assert torch.equal(first, zn.mx_matmul(c, s, *q, dtype=torch.float32))


@pytest.mark.parametrize("fmt", ["fp8", "fp4"])
@pytest.mark.parametrize("m", [1, 21, 300])
def test_from_stored_weights_to_the_product(fmt, m):
    # a layer's weights are quantised, compressed by the codec, restored, and
    # multiplied by the normed residual stream
    n, k = 392, 4096
    x, r, nw, w = _setting(m, n, k, seed=3)
    codes, scales = zn.mx_quantize(w, FMT[fmt])
    ts = zn.setup([codes], chunk_bytes=65536)
    restored = zn.decompress(ts, zn.compress(ts, [codes]))[0].view(codes.shape)
    assert np.array_equal(raw(restored), raw(codes)) and restored.dtype == codes.dtype
    c, s, h = zn.mx_rms_norm(x, nw, residual=r)
    out = zn.mx_matmul(c, s, restored, scales, dtype=torch.float32)
    assert torch.equal(h, (x.float() + r.float()).bfloat16())
    y = mx.values(raw(c), raw(s), "fp8")
    v = mx.values(raw(codes), raw(scales), fmt)
    want, mag = mx.matmul(y, v), mx.matmul(np.abs(y), np.abs(v))
    assert (np.abs(f64(out) - want) <= k * 2.0 ** -23 * mag + 2.0 ** -24 * np.abs(want)).all()
    # and the whole against the unquantised layer: each side is off by at most
    # half a step of its grid, 2^-4 or 2^-2 of a value or of the block's top binade
    exact = mx.rms_norm(f64(h), f64(nw), 1e-5)
    wv = f64(w)
    ea = np.abs(y - exact)
    ew = np.abs(v - wv)
    slack = ea @ np.abs(wv).T + np.abs(y) @ ew.T
    assert (np.abs(want - exact @ wv.T) <= slack * (1 + 1e-9) + 1e-12).all()
    assert np.linalg.norm(want - exact @ wv.T) < 0.25 * np.linalg.norm(exact @ wv.T)
