"""Microscaled numbers, measured: quantisation and reading back, the norm that makes 8-bit activations, the product.

Blocks of 32 consecutive values of a row share one E8M0 scale byte (2^(byte - 127), 255 a NaN); the values are
FP8 E4M3 (torch.float8_e4m3fn) or FP4 E2M1 pairs (uint8, the first value in the low nibble).  Rows are filled up
to whole blocks with zero codes.  The scale is 2^(floor(log2 max|x|) - emax), emax 8 for E4M3 and 2 for E2M1,
and the values are rounded to nearest even, saturating.

With `own` false `run` computes the plain forms from elementary torch operations; with `own` true it calls the
library.  Sizes are those of the 8B-shaped block of the package's workloads (hidden 4096, kv 1024, ffn 14336)
and odd neighbours.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 32
EMAX = {"fp8": 8, "fp4": 2}
TOP = {"fp8": 448.0, "fp4": 6.0}
# the smallest normal exponent and the fraction bits: the spacing of the grid at 2^e is 2^(max(e, LOW) - BITS)
LOW = {"fp8": -6, "fp4": 0}
BITS = {"fp8": 3, "fp4": 1}
TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------- cases --
def listed():
    return [
        # one token's activations before a product: latency
        {"name": "quantize_fp8_token", "op": "quantize", "fmt": "fp8", "type": "bf16", "rows": 1, "k": 4096},
        # a batch of FP32 rows whose length is no whole number of blocks
        {"name": "quantize_fp8_ragged", "op": "quantize", "fmt": "fp8", "type": "fp32", "rows": 1531, "k": 2883},
        # the value projection of a BF16 block turned into 4 bits and read back
        {"name": "quantize_fp4_kv", "op": "quantize", "fmt": "fp4", "type": "bf16", "rows": 1024, "k": 4096},
        # the stacked gate and up projections of a block, 117 million weights
        {"name": "quantize_fp4_ffn", "op": "quantize", "fmt": "fp4", "type": "bf16", "rows": 28672, "k": 4096},
        # one token of the residual stream: latency
        {"name": "norm_token", "op": "norm", "type": "bf16", "rows": 1, "k": 4096, "residual": True},
        # an FP32 stream without an addition, odd length
        {"name": "norm_ragged", "op": "norm", "type": "fp32", "rows": 613, "k": 5003, "residual": False},
        # a prompt batch
        {"name": "norm_prompt", "op": "norm", "type": "bf16", "rows": 8192, "k": 4096, "residual": True},
        # one token through the gate projection: bound by the weights' bytes
        {"name": "matmul_token", "op": "matmul", "a": "fp8", "w": "fp4", "m": 1, "n": 14336, "k": 4096, "type": "bf16"},
        # a decoding batch through the down projection
        {"name": "matmul_batch", "op": "matmul", "a": "fp8", "w": "fp4", "m": 48, "n": 4096, "k": 14336, "type": "bf16"},
        # odd sizes on every side, a last step of three blocks, 8-bit weights, FP32 sums kept
        {"name": "matmul_ragged", "op": "matmul", "a": "fp8", "w": "fp8", "m": 1021, "n": 2051, "k": 2016, "type": "fp32"},
        # both sides in 4 bits
        {"name": "matmul_fp4", "op": "matmul", "a": "fp4", "w": "fp4", "m": 4096, "n": 14336, "k": 4096, "type": "bf16"},
        # a prompt batch through the stacked gate and up projections: bound by the matrix units
        {"name": "matmul_prompt", "op": "matmul", "a": "fp8", "w": "fp4", "m": 8192, "n": 28672, "k": 4096, "type": "bf16"},
    ]


def _spread(rng, low, high):
    """A whole number in [low, high], even over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["quantize", "norm", "matmul"])
    if op == "matmul":
        k = BLOCK * _spread(rng, 4, 448)
        n = _spread(rng, 16, 28672)
        m = _spread(rng, 1, 8192)
        return {"op": op, "a": rng.choice(["fp8", "fp4"]), "w": rng.choice(["fp4", "fp8"]), "m": m,
                "n": min(n, 8192 * 28672 * 4096 // (m * k)), "k": k, "type": rng.choice(["bf16", "bf16", "fp32"])}
    k = _spread(rng, 64, 16384)
    if op == "norm":
        rows = min(_spread(rng, 1, 16384), 8192 * 4096 // k)
        return {"op": op, "type": rng.choice(["bf16", "fp32"]), "rows": rows, "k": k,
                "residual": rng.random() < 0.7}
    rows = min(_spread(rng, 1, 32768), 28672 * 2048 // k)
    return {"op": op, "fmt": rng.choice(["fp8", "fp4"]), "type": rng.choice(["bf16", "fp32"]), "rows": rows, "k": k}


def _blocks(k):
    return -(-k // BLOCK)


def work(case):
    if case["op"] == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        size = {"fp8": k, "fp4": k // 2}
        out = m * n * (2 if case["type"] == "bf16" else 4)
        return {"bytes": m * (size[case["a"]] + k // BLOCK) + n * (size[case["w"]] + k // BLOCK) + out,
                "flops": 2 * m * n * k}
    rows, k, nb = case["rows"], case["k"], _blocks(case["k"])
    item = 2 if case["type"] == "bf16" else 4
    if case["op"] == "norm":
        # x (and the residual) in, the sum out where there is one, codes, scales and the weight
        return {"bytes": rows * k * item * (3 if case["residual"] else 1) + rows * nb * (BLOCK + 1) + k * item,
                "flops": 6 * rows * k}
    if case["fmt"] == "fp8":
        return {"bytes": rows * k * item + rows * nb * (BLOCK + 1), "flops": 4 * rows * k}
    # 4 bits: x in, codes and scales made, and the values that they stand for out
    return {"bytes": rows * k * item + rows * nb * (BLOCK // 2 + 1) + rows * k * 2, "flops": 6 * rows * k}


# -------------------------------------------------------------- plain forms --
def _scale_of(byte):
    """2^(byte - 127) in FP32 from the bits: byte 0 is the subnormal 2^-127, 255 a NaN."""
    b = byte.to(torch.int32)
    bits = torch.where(b == 0, torch.full_like(b, 0x00400000), b << 23)
    return torch.where(b == 255, torch.full_like(b, 0x7FC00000), bits).view(torch.float32)


def _quantize(x, fmt):
    """FP32 rows -> the values' grid points [rows, blocks, 32] in FP32 and the scale bytes [rows, blocks]."""
    rows, k = x.shape
    nb = _blocks(k)
    if nb * BLOCK != k:
        x = torch.cat([x, x.new_zeros(rows, nb * BLOCK - k)], 1)
    x = x.view(rows, nb, BLOCK)
    top = x.abs().amax(2)
    fine = torch.isfinite(top)
    exponent = torch.frexp(torch.where(fine, top, torch.ones_like(top)))[1] - 1
    byte = (exponent + (127 - EMAX[fmt])).clamp(0, 254)
    byte = torch.where(top == 0, torch.zeros_like(byte), byte)
    inverse = ((254 - byte).to(torch.int32) << 23).view(torch.float32)
    v = x * inverse.unsqueeze(2)
    e = (torch.frexp(v)[1] - 1).clamp(LOW[fmt], EMAX[fmt]) - BITS[fmt]
    step = ((e.to(torch.int32) + 127) << 23).view(torch.float32)
    q = (torch.round(v / step) * step).clamp(-TOP[fmt], TOP[fmt])
    q = torch.where(fine.unsqueeze(2), q, torch.zeros_like(q))
    byte = torch.where(fine, byte, torch.full_like(byte, 255))
    return q, byte.to(torch.uint8)


def _codes(q, fmt):
    """Grid points as the stored codes: E4M3 bytes, or E2M1 nibbles two to a byte."""
    rows = q.shape[0]
    q = q.reshape(rows, -1)
    if fmt == "fp8":
        return q.to(torch.float8_e4m3fn)
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a * 0.5 + 4)).to(torch.uint8)
    code = code | (torch.signbit(q).to(torch.uint8) << 3)
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _values(codes, scales, fmt):
    """Codes and scales as FP32 rows."""
    rows = codes.shape[0]
    if fmt == "fp8":
        v = codes.to(torch.float32)
    else:
        grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
        v = grid[torch.stack([codes & 15, codes >> 4], 2).to(torch.int32).view(rows, -1)]
    s = _scale_of(scales.view(torch.uint8))
    return (v.view(rows, -1, BLOCK) * s.unsqueeze(2)).view(rows, -1)


# ------------------------------------------------------------------ prepare --
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _activations(rows, k, g):
    """N(0, 1) with a few channels far larger than the rest, as residual streams have them."""
    loud = 1 + 15 * (torch.rand(k, device="cuda", generator=g) < 0.01).float()
    return torch.randn(rows, k, device="cuda", generator=g) * loud


def _weights(rows, k, g):
    """N(0, 0.02), each row with a size of its own."""
    size = 0.02 * torch.exp(0.2 * torch.randn(rows, 1, device="cuda", generator=g))
    return torch.randn(rows, k, device="cuda", generator=g) * size


def _stored(x, fmt):
    q, byte = _quantize(x, fmt)
    return _codes(q, fmt), byte.view(torch.float8_e8m0fnu)


def prepare(case, seed):
    g = _generator(seed)
    state = dict(case)
    if case["op"] == "matmul":
        a = _activations(case["m"], case["k"], g).to(torch.bfloat16).float()
        state["a_codes"], state["a_scales"] = _stored(a, case["a"])
        w = _weights(case["n"], case["k"], g).to(torch.bfloat16).float()
        state["w_codes"], state["w_scales"] = _stored(w, case["w"])
        return state
    t = TORCH[case["type"]]
    make = _activations if case["op"] == "norm" or case["fmt"] == "fp8" else _weights
    state["x"] = make(case["rows"], case["k"], g).to(t)
    if case["op"] == "norm":
        state["weight"] = (1 + 0.05 * torch.randn(case["k"], device="cuda", generator=g)).to(t)
        state["r"] = _activations(case["rows"], case["k"], g).to(t) if case["residual"] else None
    return state


# ---------------------------------------------------------------------- run --
def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "matmul":
        a = _values(state["a_codes"], state["a_scales"], state["a"])
        w = _values(state["w_codes"], state["w_scales"], state["w"])
        return torch.matmul(a, w.t()).to(TORCH[state["type"]])
    if op == "norm":
        h = state["x"]
        if state["r"] is not None:
            h = (h.float() + state["r"].float()).to(h.dtype)
        y = h.float()
        y = y * torch.rsqrt(y.square().mean(1, keepdim=True) + EPS) * state["weight"].float()
        q, byte = _quantize(y, "fp8")
        out = [_codes(q, "fp8"), byte.view(torch.float8_e8m0fnu)]
        return out + [h] if state["r"] is not None else out
    q, byte = _quantize(state["x"].float(), state["fmt"])
    scales = byte.view(torch.float8_e8m0fnu)
    if state["fmt"] == "fp8":
        return [_codes(q, "fp8"), scales]
    codes = _codes(q, "fp4")
    return [_values(codes, scales, "fp4")[:, :state["k"]].to(torch.bfloat16), scales]


def _run_own(state):
    from lossless_float_weight_amd import zn
    op = state["op"]
    if op == "matmul":
        return zn.mx_matmul(state["a_codes"], state["a_scales"], state["w_codes"], state["w_scales"],
                            dtype=TORCH[state["type"]])
    if op == "norm":
        codes, scales, h = zn.mx_rms_norm(state["x"], state["weight"], residual=state["r"], eps=EPS)
        return [codes, scales, h] if state["r"] is not None else [codes, scales]
    if state["fmt"] == "fp8":
        codes, scales = zn.mx_quantize(state["x"], zn.FP8_E4M3)
        return [codes, scales]
    codes, scales = zn.mx_quantize(state["x"], zn.FP4X2_E2M1)
    # what the 4 bits stand for, as a user reads it back
    return [zn.mx_dequantize(codes, scales, k=state["k"], dtype=torch.bfloat16), scales]


# -------------------------------------------------------------------- exact --
def _grid64(fmt):
    """The format's non-negative values in the order of their codes, from sign, exponent and fraction."""
    bias, bits, count = (7, 3, 127) if fmt == "fp8" else (1, 1, 8)
    got = []
    for code in range(count):
        e, f = code >> bits, code & ((1 << bits) - 1)
        got.append(math.ldexp(f, 1 - bias - bits) if e == 0 else math.ldexp((1 << bits) + f, e - bias - bits))
    return torch.tensor(got, dtype=torch.float64, device="cuda")


def _quantize64(x, fmt):
    """Rounded values [rows, blocks * 32] without their scale, and the scales [rows, blocks], in 64 bits."""
    rows, k = x.shape
    nb = _blocks(k)
    full = torch.zeros(rows, nb * BLOCK, dtype=torch.float64, device=x.device)
    full[:, :k] = x
    full = full.view(rows, nb, BLOCK)
    top = full.abs().amax(2)
    # the largest power of two at or under the block's maximum, by search and not by a logarithm
    powers = torch.tensor([math.ldexp(1.0, e) for e in range(-127, 128)], dtype=torch.float64, device=x.device)
    at = torch.bucketize(top, powers, right=True) - 1
    scale = powers[(at - EMAX[fmt]).clamp(min=0)]
    grid = _grid64(fmt)
    middle = (grid[1:] + grid[:-1]) / 2
    for r in range(0, rows, 4096):  # rows at a time, for the memory of the search
        v = full[r:r + 4096] / scale[r:r + 4096].unsqueeze(2)
        a = v.abs()
        i = torch.bucketize(a, middle)
        tie = (i < len(middle)) & (a == middle[i.clamp(max=len(middle) - 1)])
        i = i + (tie & (i % 2 == 1)).to(i.dtype)
        full[r:r + 4096] = torch.copysign(grid[i], v)
    return full.view(rows, -1), scale


def _values64(codes, scales, fmt):
    rows = codes.shape[0]
    grid = _grid64(fmt)
    c = codes.view(torch.uint8).long()
    if fmt == "fp8":
        v = torch.cat([grid, grid.new_zeros(1), -grid, grid.new_zeros(1)])[c]
    else:
        v = torch.cat([grid, -grid])[torch.stack([c % 16, c // 16], 2).view(rows, -1)]
    s = torch.pow(2.0, scales.view(torch.uint8).double() - 127)
    return (v.view(rows, -1, BLOCK) * s.unsqueeze(2)).view(rows, -1)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "matmul":
        a = _values64(state["a_codes"], state["a_scales"], case["a"])
        w = _values64(state["w_codes"], state["w_scales"], case["w"])
        return torch.matmul(a, w.t())
    if case["op"] == "norm":
        h = state["x"].double()
        if state["r"] is not None:
            h = (h + state["r"].double()).to(state["x"].dtype).double()
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS) * state["weight"].double()
        v, scale = _quantize64(y, "fp8")
        return [v, scale] + ([h] if state["r"] is not None else [])
    v, scale = _quantize64(state["x"].double(), case["fmt"])
    if case["fmt"] == "fp8":
        return [v, scale]
    return [(v.view(case["rows"], -1, BLOCK) * scale.unsqueeze(2)).view(case["rows"], -1)[:, :case["k"]], scale]
