"""Cases for the block-scaled FP4 operators and the quantising stages of a feed-forward block.

Four operators: block-scaled FP4 quantisation, the block-scaled FP4 product, root-mean-square norm with the residual's
addition and a quantised output, and the gated activation with a quantised output.

Two 4-bit formats.  "nvfp4": blocks of 16 along the row with an E4M3 scale each and one fp32 scale per row.  "mxfp4":
blocks of 32 with a power-of-two scale each.  The block scales of a [rows, cols] matrix lie in tiles of 128 rows by 4
scales, 512 bytes each, tiles of one row band side by side: scale (r, c) of a tile at (r % 32) * 16 + (r // 32) * 4 + c;
places outside the matrix hold a zero byte.
"""
import math

import torch

own = False

DEVICE = "cuda"
BLOCK = {"nvfp4": 16, "mxfp4": 32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoded token's hidden state, quantised in front of a 4-bit product
        dict(name="quantize nvfp4 1x4096", op="quantize", format="nvfp4", rows=1, cols=4096, dist="outliers"),
        # a fused QKV weight matrix, quantised once when a model is loaded
        dict(name="quantize mxfp4 12288x4096", op="quantize", format="mxfp4", rows=12288, cols=4096, dist="weights"),
        # the up projection of a single decoded token: the weights stream
        dict(name="product nvfp4 1x11008x4096", op="product", format="nvfp4", m=1, n=11008, k=4096),
        # the same projection for a decode batch
        dict(name="product mxfp4 64x11008x4096", op="product", format="mxfp4", m=64, n=11008, k=4096),
        # the down projection of a medium batch: a long sum, few outputs
        dict(name="product nvfp4 256x4096x14336", op="product", format="nvfp4", m=256, n=4096, k=14336),
        # a ragged prompt and dimensions that fill no tile
        dict(name="product mxfp4 1000x4104x4160", op="product", format="mxfp4", m=1000, n=4104, k=4160),
        # prefill of the fused QKV projection
        dict(name="product nvfp4 4096x12288x4096", op="product", format="nvfp4", m=4096, n=12288, k=4096),
        # the norm in front of a block for one decoded token
        dict(name="norm e4m3 1x4096", op="norm", format="e4m3", rows=1, cols=4096, residual=True),
        # a ragged batch of wider rows, into the 4-bit product; the first block of a model has no residual yet
        dict(name="norm nvfp4 1000x8192", op="norm", format="nvfp4", rows=1000, cols=8192, residual=False),
        # prefill
        dict(name="norm e4m3 4096x4096", op="norm", format="e4m3", rows=4096, cols=4096, residual=True),
        # the activation between the two products of a decode batch
        dict(name="gate e4m3 64x11008", op="gate", format="e4m3", rows=64, cols=11008),
        # and of a prefill
        dict(name="gate mxfp4 4096x14336", op="gate", format="mxfp4", rows=4096, cols=14336),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "product", "product", "norm", "gate"))
    if op == "product":
        m, n, k = _log(rng, 1, 4096), 8 * _log(rng, 8, 1536), 64 * _log(rng, 1, 224)
        while m * n * k > 4096 * 12288 * 4096:
            m = max(1, m // 2)
        return dict(op=op, format=rng.choice(("nvfp4", "mxfp4")), m=m, n=n, k=k)
    cols = 32 * _log(rng, 2, 512)
    rows = _log(rng, 1, 12288)
    while rows * cols > 4096 * 12288:
        rows = max(1, rows // 2)
    if op == "quantize":
        return dict(op=op, format=rng.choice(("nvfp4", "mxfp4")), rows=rows, cols=cols, dist=rng.choice(("outliers", "weights")))
    fmt = rng.choice(("e4m3", "nvfp4", "mxfp4"))
    if op == "norm":
        return dict(op=op, format=fmt, rows=rows, cols=cols, residual=rng.random() < 0.7)
    return dict(op=op, format=fmt, rows=rows, cols=cols)


# ------------------------------------------------------------------ inputs
def _hidden(rows, cols, g):
    """Hidden states: normal, 1% of the columns 20 times as large, as in the residual stream of a language model."""
    x = torch.randn(rows, cols, device=DEVICE, generator=g)
    big = torch.rand(cols, device=DEVICE, generator=g) < 0.01
    return (x * (1 + 19 * big)).to(torch.bfloat16)


def _weights(rows, cols, g):
    """Weights: Student-t with three degrees of freedom times 0.02, heavy tails included."""
    w = torch.randn(rows, cols, device=DEVICE, generator=g)
    chi = torch.randn(rows, cols, device=DEVICE, generator=g).square()
    chi += torch.randn(rows, cols, device=DEVICE, generator=g).square()
    chi += torch.randn(rows, cols, device=DEVICE, generator=g).square()
    return (0.02 * w / (chi / 3).sqrt().clamp_min(1e-3)).to(torch.bfloat16)


def _pack(codes):
    """FP4 values (on the grid) to 4-bit codes, two a byte, the even element in the low half."""
    a = codes.abs()
    mag = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    c = mag + 8 * torch.signbit(codes).to(torch.uint8)
    return c[:, 0::2] + 16 * c[:, 1::2]


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    op, s = case["op"], dict(op=case["op"], format=case["format"])
    if op == "quantize":
        make = _hidden if case["dist"] == "outliers" else _weights
        return dict(s, x=make(case["rows"], case["cols"], g))
    if op == "norm":
        rows, cols = case["rows"], case["cols"]
        s.update(x=_hidden(rows, cols, g), eps=1e-5, residual=None)
        if case["residual"]:
            s["residual"] = _hidden(rows, cols, g)
        s["weight"] = (1 + 0.2 * torch.randn(cols, device=DEVICE, generator=g)).to(torch.bfloat16)
        return s
    if op == "gate":
        # the output of a gate/up product: the gate's columns, then the up projection's
        return dict(s, x=(1.5 * torch.randn(case["rows"], 2 * case["cols"], device=DEVICE, generator=g)).to(torch.bfloat16))
    for name, rows, make in (("x", case["m"], _hidden), ("w", case["n"], _weights)):
        codes, blocks, scales = _quantize_plain(make(rows, case["k"], g).float(), case["format"])
        s[name], s[name + "_blocks"] = _pack(codes.float()), blocks.view(torch.uint8)
        s[name + "_scales"] = scales
    return s


# ------------------------------------------------------------------ plain forms (32 bits)
def _e4m3(v):
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _e2m1(v):
    """The nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code, with v's sign."""
    a = v.abs().clamp_max(6.0)
    step = 0.5 + 0.5 * (a >= 2) + (a >= 4)
    return torch.copysign(torch.round(a / step) * step, v)


def _tiles(b):
    """Block scales [rows, n] as bytes in tiles of 128 rows by 4 scales."""
    rows, n = b.shape
    r4, n4 = -(-rows // 128), -(-n // 4)
    full = torch.zeros(128 * r4, 4 * n4, dtype=torch.uint8, device=b.device)
    full[:rows, :n] = b
    return full.view(r4, 4, 32, n4, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def _rows(t, rows, n):
    """The inverse of _tiles."""
    r4, n4 = -(-rows // 128), -(-n // 4)
    return t.view(r4, n4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(128 * r4, 4 * n4)[:rows, :n]


def _quantize_plain(x, fmt):
    """x fp32 [rows, cols]: FP4 values in 8 bits, the block scales' tiles, the row scales (nvfp4)."""
    rows, cols = x.shape
    blocks = x.view(rows, cols // BLOCK[fmt], BLOCK[fmt])
    top = blocks.abs().amax(-1)
    if fmt == "nvfp4":
        # one rounding in each quotient: products of bf16 values and these constants are exact, so ties stay ties
        row = top.amax(1, keepdim=True)
        floor = row.clamp_min(2688 * 2.0 ** -100)
        scales = torch.where(row == 0, torch.ones_like(row), floor / torch.full_like(row, 2688.0))
        sf = _e4m3(448 * top / floor)
        d = sf.float() * floor
        d = d.unsqueeze(-1)
        codes = _e2m1(torch.where(d == 0, torch.zeros_like(blocks), 2688 * blocks / d))
        out = _tiles(sf.view(torch.uint8)).view(torch.float8_e4m3fn)
        return codes.reshape(rows, cols).to(torch.float8_e4m3fn), out, scales.view(rows)
    _, e = torch.frexp(top)  # top = m 2^e, m in [0.5, 1)
    byte = torch.where(top == 0, torch.zeros_like(e), (e - 1 - 2 + 127).clamp_min(0))
    byte = byte.to(torch.uint8)
    codes = _e2m1(blocks / byte.view(torch.float8_e8m0fnu).float().unsqueeze(-1))  # by a power of two: exact
    return codes.reshape(rows, cols).to(torch.float8_e4m3fn), _tiles(byte).view(torch.float8_e8m0fnu), None


def _output_plain(y, fmt):
    """y fp32 quantised: E4M3 codes and a scale per row, or FP4."""
    if fmt != "e4m3":
        return _quantize_plain(y, fmt)
    top = y.abs().amax(1, keepdim=True)
    s = (top / torch.full_like(top, 448.0)).clamp_min(2.0 ** -126)
    s = torch.where(top == 0, torch.ones_like(top), s)
    return _e4m3(y / s), s.view(-1)


def _values_plain(q, blocks, fmt):
    """FP4 codes and block scales as fp32 values, without the row scales."""
    rows, cols = q.shape[0], 2 * q.shape[1]
    c = torch.stack((q & 15, q >> 4), -1).reshape(rows, cols)
    mag, neg = (c & 7).float(), 1 - 2 * (c >> 3).float()
    v = neg * torch.where(mag < 4, 0.5 * mag, torch.where(mag < 6, mag - 2, 2 * mag - 8))
    b = _rows(blocks, rows, cols // BLOCK[fmt])
    sf = b.contiguous().view(torch.float8_e4m3fn if fmt == "nvfp4" else torch.float8_e8m0fnu).float()
    return (v.view(rows, -1, BLOCK[fmt]) * sf.unsqueeze(-1)).view(rows, cols)


def run(state):
    op, fmt = state["op"], state["format"]
    if own:
        return _run_own(state, op, fmt)
    if op == "quantize":
        return _quantize_plain(state["x"].float(), fmt)
    if op == "product":
        x = _values_plain(state["x"], state["x_blocks"], fmt)
        w = _values_plain(state["w"], state["w_blocks"], fmt)
        y = x @ w.t()
        if state["x_scales"] is not None:
            y = y * (state["x_scales"].unsqueeze(1) * state["w_scales"].unsqueeze(0))
        return y.to(torch.bfloat16)
    if op == "norm":
        h = state["x"]
        if state["residual"] is not None:
            h = (h.float() + state["residual"].float()).to(torch.bfloat16)
        f = h.float()
        y = f * torch.rsqrt(f.square().mean(1, keepdim=True) + state["eps"]) * state["weight"].float()
        return (_output_plain(y, fmt), h) if state["residual"] is not None else (_output_plain(y, fmt),)
    cols = state["x"].shape[1] // 2
    gate, up = state["x"][:, :cols].float(), state["x"][:, cols:].float()
    return _output_plain(gate / (1 + torch.exp(-gate)) * up, fmt)


# ------------------------------------------------------------------ the library's calls
def _seen(out, fmt):
    """Codes and scales as the values that they stand for."""
    if fmt == "e4m3":
        return out[0].view(torch.float8_e4m3fn), out[1]
    import structured_sparse_fp8_b200 as sp
    q, blocks, scales = out
    kind = torch.float8_e4m3fn if fmt == "nvfp4" else torch.float8_e8m0fnu
    return sp.fp4_unpack_e4m3(q).view(torch.float8_e4m3fn), blocks.view(kind), scales


def _run_own(state, op, fmt):
    import structured_sparse_fp8_b200 as sp
    if op == "quantize":
        return _seen(sp.fp4_quantize_microscaled(state["x"], fmt), fmt)
    if op == "product":
        return sp.fp4_gemm_microscaled(state["x"], state["x_blocks"], state["x_scales"],
                                       state["w"], state["w_blocks"], state["w_scales"], fmt)
    if op == "norm":
        if fmt == "e4m3":
            q, scales, h = sp.fp8_rmsnorm_quantize_pertoken(state["x"], state["weight"], state["eps"], residual=state["residual"])
            out = (q, scales)
        else:
            q, blocks, scales, h = sp.fp4_rmsnorm_quantize_microscaled(state["x"], state["weight"], state["eps"], fmt,
                                                                       residual=state["residual"])
            out = (q, blocks, scales)
        return (_seen(out, fmt), h) if state["residual"] is not None else (_seen(out, fmt),)
    if fmt == "e4m3":
        return _seen(sp.fp8_silu_mul_quantize_pertoken(state["x"]), fmt)
    return _seen(sp.fp4_silu_mul_quantize_microscaled(state["x"], fmt), fmt)


# ------------------------------------------------------------------ work
def work(case):
    op, fmt = case["op"], case["format"]
    if op == "product":
        m, n, k = case["m"], case["n"], case["k"]
        rows = (m + n) * (k // 2 + k // BLOCK[fmt] + (4 if fmt == "nvfp4" else 0))
        return {"bytes": rows + 2 * m * n, "flops": 2 * m * n * k}
    elems = case["rows"] * case["cols"]
    out = elems + 4 * case["rows"] if fmt == "e4m3" else elems + elems // BLOCK[fmt] + (4 * case["rows"] if fmt == "nvfp4" else 0)
    if op == "quantize":
        return {"bytes": 2 * elems + out, "flops": 3 * elems}
    if op == "gate":
        return {"bytes": 4 * elems + out, "flops": 8 * elems}
    return {"bytes": (6 if case["residual"] else 2) * elems + 2 * case["cols"] + out, "flops": 8 * elems}


# ------------------------------------------------------------------ 64 bits, by the definitions
def _power(e):
    """2^e for whole e: by the bits, as a power function may be an ulp off and turn ties."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exponent(a):
    """floor(log2 a) for normal a > 0, from the bits."""
    return (a.view(torch.int64) >> 52) - 1023


def _exact_e4m3(v):
    a = v.abs()
    q = _power(_exponent(a.clamp_min(2.0 ** -12)).clamp_min(-6) - 3)
    return torch.sign(v) * (torch.round(a / q) * q).clamp_max(448.0)


def _exact_e2m1(v):
    a = v.abs()
    up = 0.5 * ((a > 0.25).double() + (a >= 0.75) + (a > 1.25) + (a >= 1.75)) + (a > 2.5) + (a >= 3.5) + 2.0 * (a > 5)
    return torch.sign(v) * up


def _exact_place(rows, n):
    """Where the scale of (row, block) lies, and the size of all tiles."""
    r = torch.arange(rows, device=DEVICE).unsqueeze(1)
    c = torch.arange(n, device=DEVICE).unsqueeze(0)
    wide = (n + 3) // 4
    return ((r // 128) * wide + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4, (rows + 127) // 128 * wide * 512


def _exact_quantize(x, fmt):
    rows, cols = x.shape
    n = cols // BLOCK[fmt]
    top = x.abs().view(rows, n, -1).max(-1).values
    place, size = _exact_place(rows, n)
    if fmt == "nvfp4":
        row = torch.clamp(top.max(1).values, min=2688 * 2.0 ** -100)
        rs = torch.where(top.max(1).values > 0, row / 2688, torch.ones_like(row))
        sf = _exact_e4m3(top * 448 / row.unsqueeze(1))
        out = torch.zeros(size, dtype=torch.float64, device=DEVICE)
        by = sf * row.unsqueeze(1)
        x = 2688 * x
    else:
        rs = None
        sf = _power((_exponent(top.clamp_min(2.0 ** -140)) - 2).clamp_min(-127))  # 2^-127 for an empty block
        out = torch.full((size,), 2.0 ** -127, dtype=torch.float64, device=DEVICE)
        by = sf
    out[place.reshape(-1)] = sf.reshape(-1)
    many = by.repeat_interleave(BLOCK[fmt], 1)
    codes = _exact_e2m1(torch.where(many > 0, x / many.clamp_min(1e-300), torch.zeros_like(x)))
    return codes, out, rs


def _exact_output(y, fmt):
    if fmt != "e4m3":
        return _exact_quantize(y, fmt)
    top = y.abs().max(1).values
    s = torch.where(top > 0, torch.clamp(top / 448, min=2.0 ** -126), torch.ones_like(top))
    return _exact_e4m3(y / s.unsqueeze(1)), s


def _exact_values(q, blocks, fmt):
    rows, cols = q.shape[0], 2 * q.shape[1]
    at = torch.arange(cols, device=DEVICE)
    code = (q[:, at // 2].int() >> (4 * (at % 2))) & 15
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=DEVICE)
    place, _ = _exact_place(rows, cols // BLOCK[fmt])
    b = blocks[place.reshape(-1)].double().view(rows, -1)
    if fmt == "nvfp4":
        e, m = torch.floor(b / 8), b % 8
        sf = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * _power(e - 10))
    else:
        sf = _power(b - 127)
    return grid[code.long()] * sf.repeat_interleave(BLOCK[fmt], 1)


def exact(case, seed):
    s = prepare(case, seed)
    op, fmt = s["op"], s["format"]
    if op == "quantize":
        return _exact_quantize(s["x"].double(), fmt)
    if op == "product":
        y = torch.matmul(_exact_values(s["x"], s["x_blocks"], fmt), _exact_values(s["w"], s["w_blocks"], fmt).t())
        return y if fmt == "mxfp4" else y * s["x_scales"].double().unsqueeze(1) * s["w_scales"].double().unsqueeze(0)
    if op == "norm":
        h = s["x"].double()
        if s["residual"] is not None:
            # the norm is of the stored sum, which has 16 bits
            h = (h + s["residual"].double()).to(torch.bfloat16).double()
        y = h / torch.sqrt((h * h).mean(1, keepdim=True) + s["eps"]) * s["weight"].double()
        return (_exact_output(y, fmt), h) if s["residual"] is not None else (_exact_output(y, fmt),)
    cols = s["x"].shape[1] // 2
    gate = s["x"][:, :cols].double()
    return _exact_output(gate * torch.sigmoid(gate) * s["x"][:, cols:].double(), fmt)
