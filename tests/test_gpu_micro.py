"""Block-scaled FP4 (quantiser, unpacking, product), the quantising norm and
gated activation, against the float64 oracle.

The quantiser of bf16 values is bit-exact.  Behind the norm and the activation
the values that are quantised carry fp32 rounding errors of a known relative
size d, so a code must lie between the codes of the reference value times
(1 - d) and (1 + d) under the kernel's own scales, and the scales likewise.
The product is held to half a bf16 step plus the fp32 accumulation's error.
"""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

from oracle import micro_oracle as MO
from oracle import sp24_oracle as O
from structured_sparse_fp8_b200 import workloads as WL

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
U = 2.0 ** -24   # half an fp32 step


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()
    torch.cuda.set_device(DEV)


def sp():
    import structured_sparse_fp8_b200 as m
    return m


def dev_bf16(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(torch.bfloat16).to(DEV)


def bits_of(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def unpack(b):
    b = b.cpu().numpy()
    out = np.empty((b.shape[0], 2 * b.shape[1]), dtype=np.uint8)
    out[:, 0::2], out[:, 1::2] = b & 0xF, b >> 4
    return out


def pack(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def rows_of(blocks, rows, cols, fmt):
    """Scale bytes [rows, n]; everything else in the tiles must be zero."""
    n = cols // MO.BLOCK[fmt]
    t = blocks.cpu().numpy()
    assert t.size == MO.tile_bytes(rows, n)
    byts = MO.from_tiles(t, rows, n)
    assert np.array_equal(MO.to_tiles(byts), t), "a scale outside the matrix is not zero"
    return byts


def same_codes(got, want):
    """Equal as values: a zero may carry either sign."""
    return np.array_equal(O.e2m1_decode(got), O.e2m1_decode(want))


# ------------------------------------------------------------------ quantiser
QSHAPES = [(1, 32), (1, 4096), (3, 64), (7, 96), (127, 160), (128, 256), (129, 1056), (300, 4096), (5, 16416),
           (2, 40000), (3000, 64), (2, 131072), (700, 1056), (333, 8224), (1500, 2048), (297, 33024)]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("shape", QSHAPES)
def test_quantize_bit_exact(fmt, shape):
    for i, (dist, scale) in enumerate((("normal", 1.0), ("student_t3", 0.02), ("ties", 1.0))):
        x = WL.random_bits(shape, 4000 + 10 * shape[1] + i, scale=scale, dist=dist)
        if shape[0] > 2:
            x[1] = 0                                        # an all-zero row
            x[2, :16] = 0                                   # and an empty block
        st = status()
        q, blocks, rs = sp().fp4_quantize_microscaled(dev_bf16(x), fmt, status=st)
        torch.cuda.synchronize()
        codes, byts, ref_rs = MO.quantize(O.bf16_to_f32(x).astype(np.float64), fmt)
        assert int(st.item()) == 0
        assert np.array_equal(rows_of(blocks, *shape, fmt), byts)
        assert same_codes(unpack(q), codes)
        if fmt == "nvfp4":
            assert np.array_equal(rs.cpu().numpy(), ref_rs)
        else:
            assert rs is None


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_quantize_every_finite_bf16_value(fmt):
    """Rows that hold every finite bf16 value in some block, beneath row
    maxima from a subnormal to the largest finite value."""
    bits = np.arange(65536, dtype=np.uint16)
    v = O.bf16_to_f32(bits)
    for top in (0x0001, 0x0100, 0x1400, 0x3F80, 0x4195, 0x7F7F):
        limit = O.bf16_to_f32(np.array([top], dtype=np.uint16))[0]
        keep = bits[np.isfinite(v) & (np.abs(v) <= limit)]
        flat = np.random.default_rng(top).permutation(keep)
        cols = 1024
        rows = -(-flat.size // (cols - 1))
        x = np.full((rows, cols), top, dtype=np.uint16)
        body = np.zeros(rows * (cols - 1), dtype=np.uint16)
        body[:flat.size] = flat
        x[:, 1:] = body.reshape(rows, cols - 1)
        st = status()
        q, blocks, rs = sp().fp4_quantize_microscaled(dev_bf16(x), fmt, status=st)
        codes, byts, ref_rs = MO.quantize(O.bf16_to_f32(x).astype(np.float64), fmt)
        assert int(st.item()) == 0
        assert np.array_equal(rows_of(blocks, rows, cols, fmt), byts), hex(top)
        assert same_codes(unpack(q), codes), hex(top)
        if fmt == "nvfp4":
            assert np.array_equal(rs.cpu().numpy(), ref_rs), hex(top)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("bad", [0x7F80, 0xFF80, 0x7FC0])
def test_quantize_flags_nonfinite_rows_and_keeps_the_others(fmt, bad):
    for shape in ((4, 64), (4, 20000), (600, 2048)):
        x = WL.random_bits(shape, 77)
        codes, byts, _ = MO.quantize(O.bf16_to_f32(x).astype(np.float64), fmt)
        y = x.copy()
        y[2, shape[1] - 3] = bad
        st = status()
        q, blocks, _ = sp().fp4_quantize_microscaled(dev_bf16(y), fmt, status=st)
        assert int(st.item()) == sp()._lib.SP24_STATUS_NONFINITE
        keep = [0, 1] + list(range(3, shape[0]))
        assert same_codes(unpack(q)[keep], codes[keep])
        assert np.array_equal(rows_of(blocks, *shape, fmt)[keep], byts[keep])


@pytest.mark.parametrize("shape", [(1, 32), (3, 96), (17, 4096), (1000, 1056)])
def test_unpack_is_exact(shape):
    codes = np.random.default_rng(shape[1]).integers(0, 16, shape).astype(np.uint8)
    out = sp().fp4_unpack_e4m3(torch.from_numpy(pack(codes)).to(DEV))
    assert out.shape == shape
    want = O.e4m3_encode(O.e2m1_decode(codes).astype(np.float32))
    assert np.array_equal(out.cpu().numpy(), want)


# ------------------------------------------------------------------ norm, gate
def between(got, lo, hi, what):
    ok = (got >= lo) & (got <= hi)
    assert ok.all(), f"{what}: {int((~ok).sum())} of {ok.size} outside; first at {np.argwhere(~ok)[:3].tolist()}"


def check_e4m3(q, s, y, d):
    """E4M3 codes and row scales of values y (float64) known to relative d."""
    q, s = q.cpu().numpy(), s.cpu().numpy().astype(np.float64)
    d = np.broadcast_to(d, y.shape)
    top = np.abs(y).max(axis=1)
    dr = d.max(axis=1) + 2 * U
    between(s, MO.e4m3_row_scale(top * (1 - dr)), MO.e4m3_row_scale(top * (1 + dr)), "row scale")
    t = np.abs(y) / s[:, None]
    got = np.abs(O.e4m3_decode(q))
    between(got, O.e4m3_decode(O.e4m3_encode((t * (1 - d - 4 * U)).astype(np.float32))),
            O.e4m3_decode(O.e4m3_encode((t * (1 + d + 4 * U)).astype(np.float32))), "code")
    nz = got > 0
    assert np.array_equal(np.signbit(O.e4m3_decode(q))[nz], np.signbit(y)[nz])


def check_fp4(q, blocks, rs, y, d, fmt):
    rows, cols = y.shape
    codes, byts = unpack(q), rows_of(blocks, rows, cols, fmt)
    d = np.broadcast_to(d, y.shape)
    n = cols // MO.BLOCK[fmt]
    top = np.abs(y).reshape(rows, n, -1).max(axis=2)
    db = d.reshape(rows, n, -1).max(axis=2) + 2 * U
    sv = MO.scale_values(byts, fmt)
    if fmt == "nvfp4":
        amax, dr = top.max(axis=1), d.max(axis=1) + 2 * U
        between(rs.cpu().numpy().astype(np.float64), MO.nvfp4_row_scale(amax * (1 - dr)) * (1 - U),
                MO.nvfp4_row_scale(amax * (1 + dr)) * (1 + U), "row scale")
        R = np.where(amax == 0, MO.ROW_FLOOR, rs.cpu().numpy().astype(np.float64) * 2688.0)
        t = 448.0 * top / R[:, None]
        lo, hi = ((t * (1 + sg * (db + 6 * U))).astype(np.float32) for sg in (-1, 1))
        between(sv, O.e4m3_decode(O.e4m3_encode(lo)), O.e4m3_decode(O.e4m3_encode(hi)), "block scale")
        many = np.repeat(sv, 16, axis=1) * R[:, None] / 2688.0
    else:
        assert rs is None
        between(byts.astype(int), MO.mxfp4_block_bytes(top * (1 - db)).astype(int),
                MO.mxfp4_block_bytes(top * (1 + db)).astype(int), "block scale")
        many = np.repeat(sv, 32, axis=1)
    t = np.where(many > 0, np.abs(y) / np.where(many > 0, many, 1.0), 0.0)
    got = np.abs(O.e2m1_decode(codes))
    lo, hi = (O.e2m1_decode(MO.e2m1_codes(t * (1 + sg * (d + 8 * U)))) for sg in (-1, 1))
    between(got, lo, hi, "code")
    nz = got > 0
    assert np.array_equal((codes & 8 != 0)[nz], np.signbit(y)[nz])


def norm_error(cols):
    """Relative error of y: the fp32 sum of squares (in any order over 32
    threads or more: cols / 32 + 16 additions deep, halved by the root), the
    mean, eps, the root and the two products."""
    return (cols / 64 + 16) * U


NSHAPES = [(1, 32), (1, 4096), (5, 64), (130, 96), (64, 4096), (3, 8192), (4, 11008), (2, 16416), (2, 70016), (333, 1056), (700, 4096), (1300, 2080), (300, 11008)]


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("shape", NSHAPES)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(fmt, shape, residual):
    rows, cols = shape
    x = WL.random_bits(shape, 5000 + cols, scale=2.0)
    r = WL.random_bits(shape, 5001 + cols, scale=3.0) if residual else None
    w = WL.random_bits((1, cols), 5002 + cols)[0]
    if rows > 3:
        x[3] = 0
        if residual:
            r[3] = 0
    eps = 1e-5
    y, h = MO.rmsnorm(x, r, w, eps)
    st = status()
    X, W, R = dev_bf16(x), dev_bf16(w), (dev_bf16(r) if residual else None)
    if fmt == "e4m3":
        q, s, hk = sp().fp8_rmsnorm_quantize_pertoken(X, W, eps, residual=R, status=st)
        check_e4m3(q, s, y, norm_error(cols))
    else:
        q, b, s, hk = sp().fp4_rmsnorm_quantize_microscaled(X, W, eps, fmt, residual=R, status=st)
        check_fp4(q, b, s, y, norm_error(cols), fmt)
    assert int(st.item()) == 0
    assert np.array_equal(bits_of(hk), h)
    assert np.array_equal(bits_of(X), x)
    if residual:
        assert np.array_equal(bits_of(R), r)
    else:
        assert hk is X


@pytest.mark.parametrize("where", ["x", "residual"])
@pytest.mark.parametrize("rows,cols", [(9, 64), (9, 4096), (9, 30000 // 32 * 32), (2000, 1056), (700, 4096)])
def test_norm_in_place(where, rows, cols):
    x, r = WL.random_bits((rows, cols), 61), WL.random_bits((rows, cols), 62)
    w = dev_bf16(WL.random_bits((1, cols), 63)[0])
    q0, s0, h0 = sp().fp8_rmsnorm_quantize_pertoken(dev_bf16(x), w, 1e-6, residual=dev_bf16(r))
    X, R = dev_bf16(x), dev_bf16(r)
    target = X if where == "x" else R
    q, s, h = sp().fp8_rmsnorm_quantize_pertoken(X, w, 1e-6, residual=R, residual_out=target)
    assert h is target
    assert torch.equal(h, h0) and torch.equal(q, q0) and torch.equal(s, s0)


def test_norm_of_a_zero_row_without_eps_and_with_a_zero_weight():
    x = WL.random_bits((2, 96), 5)
    x[1] = 0
    w = WL.random_bits((1, 96), 6)[0]
    w[:64] = 0
    st = status()
    y, _ = MO.rmsnorm(x, None, w, 0.0)
    q, s, _ = sp().fp8_rmsnorm_quantize_pertoken(dev_bf16(x), dev_bf16(w), 0.0, status=st)
    check_e4m3(q, s, y, norm_error(96))
    # zeros of the sign of 0 * weight
    assert s[1].item() == 1.0 and not (q[1] & 0x7F).any()
    for fmt in ("nvfp4", "mxfp4"):
        q, b, s, _ = sp().fp4_rmsnorm_quantize_microscaled(dev_bf16(x), dev_bf16(w), 0.0, fmt, status=st)
        check_fp4(q, b, s, y, norm_error(96), fmt)
    assert int(st.item()) == 0


@pytest.mark.parametrize("bad", [0x7F80, 0x7FC0, 0x7F00])  # Inf, NaN, and a square beyond fp32
def test_norm_flags_nonfinite_rows_and_keeps_the_others(bad):
    for rows, cols in ((5, 96), (5, 20000), (900, 2048)):
        x = WL.random_bits((rows, cols), 8)
        w = WL.random_bits((1, cols), 9)[0]
        good_q, good_s, _ = sp().fp8_rmsnorm_quantize_pertoken(dev_bf16(x), dev_bf16(w), 1e-5)
        x[1, 17] = bad
        st = status()
        q, s, _ = sp().fp8_rmsnorm_quantize_pertoken(dev_bf16(x), dev_bf16(w), 1e-5, status=st)
        assert int(st.item()) == sp()._lib.SP24_STATUS_NONFINITE
        keep = [0] + list(range(2, rows))
        assert torch.equal(q[keep], good_q[keep]) and torch.equal(s[keep], good_s[keep])


GSHAPES = [(1, 32), (1, 11008), (5, 64), (130, 96), (64, 1056), (7, 14336), (3, 33024), (333, 1056), (650, 4096), (300, 16416)]


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("shape", GSHAPES)
def test_gate(fmt, shape):
    rows, cols = shape
    gu = WL.random_bits((rows, 2 * cols), 6000 + cols, scale=2.0)
    gu[:, 5] = 0xC2C8                                       # a gate of -100: 0
    gu[:, 6] = 0x42C8                                       # and of 100
    gu[:, 7] = 0                                            # and of 0
    if rows > 3:
        gu[3] = 0
    y = MO.silu_mul(gu)
    # the exponential is off by 2 + 1.173 |g| steps at most, the quotient by 2;
    # the sum and the products round once each
    g = np.abs(O.bf16_to_f32(gu)[:, :cols].astype(np.float64))
    d = (1.173 * g + 8) * 2 * U
    st = status()
    if fmt == "e4m3":
        q, s = sp().fp8_silu_mul_quantize_pertoken(dev_bf16(gu), status=st)
        check_e4m3(q, s, y, d)
    else:
        q, b, s = sp().fp4_silu_mul_quantize_microscaled(dev_bf16(gu), fmt, status=st)
        check_fp4(q, b, s, y, d, fmt)
    assert int(st.item()) == 0


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("cols", [64, 4096, 40032])
def test_gate_of_far_negative_gates_and_large_up(fmt, cols):
    """Gates whose factor 1 / (1 + exp(-g)) is below 2^-126, and up values that
    bring the product back to ordinary size."""
    x = np.tile(np.float64([-86.0, -87.0, -88.0, -89.0]), cols // 4)
    up = np.tile(np.float64([3e38, 1e38, -2e38, 3e38]), cols // 4)
    gu = WL.to_bf16_bits(np.concatenate([x, up])[None])
    y = MO.silu_mul(gu)
    assert np.abs(y).min() > 1
    # as in test_gate, and the factor (at least 2^-129) is rounded to a multiple of 2^-149
    d = (1.173 * np.abs(x)[None] + 8) * 2 * U + 2.0 ** -21
    st = status()
    if fmt == "e4m3":
        q, s = sp().fp8_silu_mul_quantize_pertoken(dev_bf16(gu), status=st)
        check_e4m3(q, s, y, d)
    else:
        q, b, s = sp().fp4_silu_mul_quantize_microscaled(dev_bf16(gu), fmt, status=st)
        check_fp4(q, b, s, y, d, fmt)
    assert int(st.item()) == 0


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("power", [-118, -100, -70, 60, 100, 118])
@pytest.mark.parametrize("rows,cols", [(3, 96), (3, 4096), (1300, 8192), (2, 40032)])
def test_rows_of_any_size(fmt, power, rows, cols):
    """Values scaled by a power of two, through the norm's weight and the
    gate's up projection: quotients of a row's values stay in range."""
    few = slice(0, 3)                                       # rows that are checked
    x = np.tile(WL.random_bits((3, cols), 71), (rows // 3 + 1, 1))[:rows]
    up = WL.to_bf16_bits(O.bf16_to_f32(WL.random_bits((1, cols), 72)).astype(np.float64) * 2.0 ** power)
    st = status()
    y, _ = MO.rmsnorm(x[few], None, up[0], 1e-5)
    gu = np.concatenate([x, np.tile(up, (rows, 1))], axis=1)
    gy = MO.silu_mul(gu[few])
    d = (1.173 * np.abs(O.bf16_to_f32(x[few]).astype(np.float64)) + 8) * 2 * U
    X, W, GU = dev_bf16(x), dev_bf16(up[0]), dev_bf16(gu)
    if fmt == "e4m3":
        q, s, _ = sp().fp8_rmsnorm_quantize_pertoken(X, W, 1e-5, status=st)
        check_e4m3(q[few], s[few], y, norm_error(cols))
        q, s = sp().fp8_silu_mul_quantize_pertoken(GU, status=st)
        check_e4m3(q[few], s[few], gy, d)
    else:
        n = min(rows, 3)

        def first(b):                                       # the first rows' scales, as a matrix of their own
            byts = rows_of(b, rows, cols, fmt)[:n]
            return torch.from_numpy(MO.to_tiles(byts)).to(DEV)

        q, b, s, _ = sp().fp4_rmsnorm_quantize_microscaled(X, W, 1e-5, fmt, status=st)
        check_fp4(q[few], first(b), None if s is None else s[few], y, norm_error(cols), fmt)
        q, b, s = sp().fp4_silu_mul_quantize_microscaled(GU, fmt, status=st)
        check_fp4(q[few], first(b), None if s is None else s[few], gy, d, fmt)
    assert int(st.item()) == 0


@pytest.mark.parametrize("rows,cols", [(3, 96), (5, 4096), (1300, 8192), (2, 40032)])
def test_inputs_aligned_to_16_bytes_only(rows, cols):
    """Tensors that start 16 bytes into a 32-byte line give what others give."""
    def shifted(t):
        buf = torch.empty(t.numel() + 8, dtype=t.dtype, device=DEV)
        v = buf[8:].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 32 == 16
        return v

    x, r = dev_bf16(WL.random_bits((rows, cols), 91)), dev_bf16(WL.random_bits((rows, cols), 92))
    gu, w = dev_bf16(WL.random_bits((rows, 2 * cols), 93)), dev_bf16(WL.random_bits((1, cols), 94)[0])
    m = sp()
    for fmt in ("nvfp4", "mxfp4"):
        for a, b in zip(m.fp4_quantize_microscaled(x, fmt), m.fp4_quantize_microscaled(shifted(x), fmt)):
            assert a is None or torch.equal(a, b)
        for a, b in zip(m.fp4_silu_mul_quantize_microscaled(gu, fmt), m.fp4_silu_mul_quantize_microscaled(shifted(gu), fmt)):
            assert a is None or torch.equal(a, b)
        for a, b in zip(m.fp4_rmsnorm_quantize_microscaled(x, w, 1e-5, fmt, residual=r),
                        m.fp4_rmsnorm_quantize_microscaled(x, shifted(w), 1e-5, fmt, residual=shifted(r))):
            assert a is None or torch.equal(a, b)
    for a, b in zip(m.fp8_rmsnorm_quantize_pertoken(x, w, 1e-5, residual=r),
                    m.fp8_rmsnorm_quantize_pertoken(x, w, 1e-5, residual=r, residual_out=shifted(x))):
        assert torch.equal(a, b)
    for a, b in zip(m.fp8_silu_mul_quantize_pertoken(gu), m.fp8_silu_mul_quantize_pertoken(shifted(gu))):
        assert torch.equal(a, b)


def test_gate_flags_a_nonfinite_row():
    gu = WL.random_bits((4, 128), 12)
    good_q, good_s = sp().fp8_silu_mul_quantize_pertoken(dev_bf16(gu))
    gu[2, 3], gu[2, 64 + 3] = 0x7F00, 0x7F00                # a product beyond fp32
    st = status()
    q, s = sp().fp8_silu_mul_quantize_pertoken(dev_bf16(gu), status=st)
    assert int(st.item()) == sp()._lib.SP24_STATUS_NONFINITE
    keep = [0, 1, 3]
    assert torch.equal(q[keep], good_q[keep]) and torch.equal(s[keep], good_s[keep])


# ------------------------------------------------------------------ product
def operand(rows, k, fmt, seed):
    """Random codes and block-scale bytes (zeros among them): numpy codes and
    bytes, and the same on the device as the product takes them."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (rows, k)).astype(np.uint8)
    n = k // MO.BLOCK[fmt]
    byts = (rng.integers(0x20, 0x58, (rows, n)) if fmt == "nvfp4" else rng.integers(118, 132, (rows, n))).astype(np.uint8)
    byts[rng.random((rows, n)) < 0.05] = 0
    return codes, byts, torch.from_numpy(pack(codes)).to(DEV), torch.from_numpy(MO.to_tiles(byts)).to(DEV)


def dev_values(codes, byts, fmt):
    """code * block scale as float64 on the device."""
    grid = torch.from_numpy(O.e2m1_decode(np.arange(16, dtype=np.uint8))).to(DEV)
    v = grid[torch.from_numpy(codes.astype(np.int32)).to(DEV).long()]
    s = torch.from_numpy(MO.scale_values(byts, fmt)).to(DEV)
    return v * s.repeat_interleave(MO.BLOCK[fmt], 1)


def check_product(y, xv, wv, xs, ws):
    """|y - ref| <= half a bf16 step of ref + what fp32 sums may lose: every
    product is exact (12 significant bits); the sum of K of them in groups of
    64 is K / 64 + 64 roundings deep, a rounding taken as a whole fp32 step.
    fp32's normal numbers end at 2^-126 and bf16's steps at 2^-133: K products
    below the former (scale bytes of 0 stand for 2^-127) add up to K * 2^-126 at
    most and may be dropped, and a result is off by half the latter."""
    k = xv.shape[1]
    scale = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    if xs is not None:
        scale = scale * xs.double().reshape(-1, 1)
    if ws is not None:
        scale = scale * ws.double().reshape(1, -1)
    ref = xv @ wv.t() * scale
    mag = xv.abs() @ wv.abs().t() * scale.abs()
    lost = (k / 64 + 64) * 2 * U * mag + 2 * U * ref.abs() + k * 2.0 ** -126 * scale.abs()
    tol = 2.0 ** -8 * (ref.abs() + lost) + lost + 2.0 ** -134
    off = (y.double() - ref).abs()
    ok = off <= tol
    assert bool(ok.all()), f"{int((~ok).sum())} of {ok.numel()} outside; first {torch.argwhere(~ok)[:4].tolist()}"


PSHAPES = [(1, 8, 64), (1, 128, 256), (2, 136, 192), (3, 4104, 320), (8, 256, 4096), (16, 1000, 1024), (17, 512, 2112),
           (33, 384, 1024), (64, 2048, 512), (100, 264, 4160), (128, 4096, 448), (129, 520, 832), (256, 1024, 1088),
           (300, 2304, 2048), (515, 1160, 576), (1000, 520, 4160), (2050, 1032, 704), (1, 11008, 4096), (1, 96, 28672),
           (70, 9000, 576), (200, 4360, 5120), (250, 6152, 5184), (600, 4104, 4160), (2000, 4096, 1024), (3000, 6152, 320), (17000, 8, 128), (9000, 40, 64)]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("m,n,k", PSHAPES)
def test_product(fmt, m, n, k):
    xc, xb, xq, xt = operand(m, k, fmt, 7000 + m)
    wc, wb, wq, wt = operand(n, k, fmt, 8000 + n)
    g = torch.Generator(device=DEV).manual_seed(m * 7 + n)
    xs = torch.rand(m, device=DEV, generator=g) + 0.5
    ws = (torch.rand(n, device=DEV, generator=g) + 0.5) * 0.01
    st = status()
    # the result lies inside a larger buffer whose other values must stay
    buf = torch.full((m * n + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
    out = buf[32:32 + m * n].view(m, n)
    y = sp().fp4_gemm_microscaled(xq, xt, xs, wq, wt, ws, fmt, out=out, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert bool((buf[:32] == 7).all()) and bool((buf[32 + m * n:] == 7).all())
    check_product(y, dev_values(xc, xb, fmt), dev_values(wc, wb, fmt), xs, ws)
    again = sp().fp4_gemm_microscaled(xq, xt, xs, wq, wt, ws, fmt)
    assert torch.equal(again, y), "the same inputs gave other bits"


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_product_scale_forms(fmt):
    for m, n, k in ((5, 264, 512), (200, 512, 512)):
        xc, xb, xq, xt = operand(m, k, fmt, 1)
        wc, wb, wq, wt = operand(n, k, fmt, 2)
        xv, wv = dev_values(xc, xb, fmt), dev_values(wc, wb, fmt)
        vec_m, vec_n = torch.rand(m, device=DEV) + 0.1, torch.rand(n, device=DEV) + 0.1
        one = torch.tensor([0.37], device=DEV)
        for xs in (None, one, vec_m):
            for ws in (None, one, vec_n):
                check_product(sp().fp4_gemm_microscaled(xq, xt, xs, wq, wt, ws, fmt), xv, wv, xs, ws)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("m,n,k", [(4, 256, 512), (300, 512, 512)])
def test_product_keeps_a_bad_row_to_itself(fmt, m, n, k):
    """A NaN scale in one row of either operand reaches that row's (column's) results only."""
    nan = 0x7F if fmt == "nvfp4" else 0xFF
    xc, xb, xq, xt = operand(m, k, fmt, 3)
    wc, wb, wq, wt = operand(n, k, fmt, 4)
    good = sp().fp4_gemm_microscaled(xq, xt, None, wq, wt, None, fmt)
    xb2, wb2 = xb.copy(), wb.copy()
    xb2[2, 1], wb2[100, 0] = nan, nan
    y = sp().fp4_gemm_microscaled(xq, torch.from_numpy(MO.to_tiles(xb2)).to(DEV), None, wq,
                                  torch.from_numpy(MO.to_tiles(wb2)).to(DEV), None, fmt)
    assert bool(y[2].isnan().all()) and bool(y[:, 100].isnan().all())
    rows = [i for i in range(m) if i != 2]
    cols = [i for i in range(n) if i != 100]
    assert torch.equal(y[rows][:, cols], good[rows][:, cols])


@pytest.mark.parametrize("m,n,k", [(3, 520, 1024), (300, 520, 1024)])
def test_product_ignores_scales_outside_the_matrix(m, n, k):
    """The tiles' unused places may hold anything: only the matrix's rows and
    blocks are used."""
    for fmt in ("nvfp4", "mxfp4"):
        k2 = k + (64 if fmt == "mxfp4" else 0)              # a last tile half used
        xc, xb, xq, xt = operand(m, k2, fmt, 5)
        wc, wb, wq, wt = operand(n, k2, fmt, 6)
        y = sp().fp4_gemm_microscaled(xq, xt, None, wq, wt, None, fmt)
        for t, rows in ((xt, m), (wt, n)):
            mask = torch.ones_like(t, dtype=torch.bool)
            mask[torch.from_numpy(MO.tile_offsets(rows, k2 // MO.BLOCK[fmt])).to(DEV).reshape(-1)] = False
            t[mask] = 0xFF
        assert torch.equal(sp().fp4_gemm_microscaled(xq, xt, None, wq, wt, None, fmt), y)


def test_long_rows_pass_32_bit_offsets():
    """A matrix of more than 2^31 elements: its last rows are as when alone."""
    rows, cols = 66000, 32768
    x = torch.randn(128, cols, device=DEV).to(torch.bfloat16).repeat(-(-rows // 128), 1)[:rows].contiguous()
    q, b, s = sp().fp4_quantize_microscaled(x, "nvfp4")
    lo = (rows // 128) * 128
    q0, b0, s0 = sp().fp4_quantize_microscaled(x[lo:].contiguous(), "nvfp4")
    assert torch.equal(q[lo:], q0) and torch.equal(s[lo:], s0)
    assert torch.equal(b[lo // 128 * (cols // 64) * 512:], b0)
    del x
    # and as an operand of a product
    w = torch.randn(64, cols, device=DEV).to(torch.bfloat16)
    wq, wb, ws = sp().fp4_quantize_microscaled(w, "nvfp4")
    y = sp().fp4_gemm_microscaled(q, b, s, wq, wb, ws)
    y0 = sp().fp4_gemm_microscaled(q0, b0, s0, wq, wb, ws)
    torch.testing.assert_close(y[lo:].float(), y0.float(), rtol=2.0 ** -7, atol=1e-3)


def test_result_past_32_bit_offsets():
    """A result of more than 2^31 elements: its last rows as from a call of their own."""
    m, n, k = 70016, 32768, 64
    x = torch.randn(m, k, device=DEV).to(torch.bfloat16)
    w = torch.randn(n, k, device=DEV).to(torch.bfloat16)
    wq = sp().fp4_quantize_microscaled(w, "mxfp4")
    y = sp().fp4_gemm_microscaled(*sp().fp4_quantize_microscaled(x, "mxfp4"), *wq, "mxfp4")
    tail = sp().fp4_gemm_microscaled(*sp().fp4_quantize_microscaled(x[-64:].contiguous(), "mxfp4"), *wq, "mxfp4")
    assert torch.equal(y[-64:], tail)        # one MMA step deep: no order of sums


def test_unpacked_codes_feed_the_dense_fp8_product():
    """FP4 weights widened to E4M3, in front of the dense FP8 GEMM right away."""
    x, w = dev_bf16(WL.random_bits((64, 512), 81)), dev_bf16(WL.random_bits((256, 512), 82, scale=0.02))
    xq, sx = sp().fp8_quantize_pertensor(x)
    wq, sw = sp().fp4_quantize_pertensor(w)
    wide = sp().fp4_unpack_e4m3(wq)
    want = sp().fp8_gemm_dense(xq, sx, wide, sw)
    torch.cuda.synchronize()
    ref, bound = O.gemm_ref(O.e4m3_decode(xq.cpu().numpy()), O.e2m1_decode(unpack(wq)), sx.item(), sw.item())
    assert O.within_tolerance(O.bf16_to_f32(bits_of(want)).astype(np.float64), ref, bound).all()
    for _ in range(20):
        buf = torch.zeros_like(wide)
        y = sp().fp8_gemm_dense(xq, sx, sp().fp4_unpack_e4m3(wq, out=buf), sw)
        assert torch.equal(y, want)


# ------------------------------------------------------------------ use together
def _ffn_fp4(x, r, w, wgu, wd, fmt, st=None):
    m = sp()
    q, b, s, h = m.fp4_rmsnorm_quantize_microscaled(x, w, 1e-5, fmt, residual=r, status=st)
    gu = m.fp4_gemm_microscaled(q, b, s, *wgu, fmt, status=st)
    q, b, s = m.fp4_silu_mul_quantize_microscaled(gu, fmt, status=st)
    return m.fp4_gemm_microscaled(q, b, s, *wd, fmt, status=st), gu, h


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("m", [1, 37, 300])
def test_feed_forward_block_fp4(fmt, m):
    """norm -> gate/up product -> gated activation -> down product, each stage
    held to the oracle on what the stage before it gave."""
    d, f = 512, 1088
    x, r = WL.random_bits((m, d), 1), WL.random_bits((m, d), 2)
    w = WL.random_bits((1, d), 3)[0]
    gu_w, d_w = WL.random_bits((2 * f, d), 4, scale=0.05), WL.random_bits((d, f), 5, scale=0.05)
    wgu = sp().fp4_quantize_microscaled(dev_bf16(gu_w), fmt)
    wd = sp().fp4_quantize_microscaled(dev_bf16(d_w), fmt)
    st = status()
    y, gu, h = _ffn_fp4(dev_bf16(x), dev_bf16(r), dev_bf16(w), wgu, wd, fmt, st)
    assert int(st.item()) == 0
    yn, hn = MO.rmsnorm(x, r, w, 1e-5)
    assert np.array_equal(bits_of(h), hn)

    def decoded(q, b, s):
        rows, cols = q.shape[0], 2 * q.shape[1]
        v = MO.values(unpack(q), rows_of(b, rows, cols, fmt), fmt)
        return torch.from_numpy(v).to(DEV), s

    q, b, s, _ = sp().fp4_rmsnorm_quantize_microscaled(dev_bf16(x), dev_bf16(w), 1e-5, fmt, residual=dev_bf16(r))
    check_fp4(q, b, s, yn, norm_error(d), fmt)
    (xv, xs), (wv, ws) = decoded(q, b, s), decoded(*wgu)
    check_product(gu, xv, wv, xs, ws)
    q, b, s = sp().fp4_silu_mul_quantize_microscaled(gu, fmt)
    (xv, xs), (wv, ws) = decoded(q, b, s), decoded(*wd)
    check_product(y, xv, wv, xs, ws)


@pytest.mark.parametrize("m", [1, 40, 200])
def test_feed_forward_block_fp8_sparse(m):
    """The same run through the 2:4 FP8 product with per-token scales."""
    d, f = 512, 640
    x, r = dev_bf16(WL.random_bits((m, d), 1)), dev_bf16(WL.random_bits((m, d), 2))
    w = dev_bf16(WL.random_bits((1, d), 3)[0])
    st = status()
    packed = []
    for shape, seed in (((2 * f, d), 4), ((d, f), 5)):
        c = sp().sp24_prune_compress_perchannel(dev_bf16(WL.random_bits(shape, seed, scale=0.05)), status=st)
        packed.append((sp().sp24_pack_weights(c["values"], c["meta"]), c["scales"], c))
    q, s, h = sp().fp8_rmsnorm_quantize_pertoken(x, w, 1e-5, residual=r, status=st)
    gu = sp().sp24_gemm_packed_scaled(q, s, packed[0][0], packed[0][1], 2 * f, status=st)
    q2, s2 = sp().fp8_silu_mul_quantize_pertoken(gu, status=st)
    y = sp().sp24_gemm_packed_scaled(q2, s2, packed[1][0], packed[1][1], d, status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for out, (qq, ss), (_, wsc, c) in ((gu, (q, s), packed[0]), (y, (q2, s2), packed[1])):
        dense = O.decompress24(c["values"].cpu().numpy(), c["meta"].cpu().numpy(), qq.shape[1])
        ref, bound = O.gemm_ref_scaled(O.e4m3_decode(qq.cpu().numpy()), O.e4m3_decode(dense), ss.cpu().numpy(),
                                       wsc.cpu().numpy())
        got = O.bf16_to_f32(bits_of(out)).astype(np.float64)
        assert O.within_tolerance(got, ref, bound).all()


@pytest.mark.parametrize("m", [1, 200])
def test_capture_replay_and_two_graphs_at_once(m):
    """The block captured twice, replayed on new inputs on two streams at once:
    the results of eager calls."""
    fmt, d, f = "nvfp4", 512, 1024
    w = dev_bf16(WL.random_bits((1, d), 3)[0])
    wgu = sp().fp4_quantize_microscaled(dev_bf16(WL.random_bits((2 * f, d), 4, scale=0.05)), fmt)
    wd = sp().fp4_quantize_microscaled(dev_bf16(WL.random_bits((d, f), 5, scale=0.05)), fmt)
    ins = [dev_bf16(WL.random_bits((m, d), 10 + i)) for i in range(8)]
    want = [_ffn_fp4(ins[2 * i], ins[2 * i + 1], w, wgu, wd, fmt)[0].clone() for i in range(4)]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        x, r = torch.empty_like(ins[0]), torch.empty_like(ins[0])
        x.copy_(ins[0])
        r.copy_(ins[1])
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = _ffn_fp4(x, r, w, wgu, wd, fmt)[0]
        graphs.append((g, x, r, y))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for pair in ((0, 1), (2, 3)):
        for i, (g, x, r, y), s in zip(pair, graphs, streams):
            with torch.cuda.stream(s):
                x.copy_(ins[2 * i])
                r.copy_(ins[2 * i + 1])
                for _ in range(3):
                    g.replay()
        torch.cuda.synchronize()
        for i, (g, x, r, y) in zip(pair, graphs):
            assert torch.equal(y, want[i])


FIRST_CALLS_IN_A_CAPTURE = """
import torch
import structured_sparse_fp8_b200 as sp
torch.manual_seed(1)
w = torch.ones(1024, device="cuda", dtype=torch.bfloat16)
x = {m: torch.randn(m, 1024, device="cuda").to(torch.bfloat16) for m in (1, 300, 1500)}
big = torch.randn(2048, 1024, device="cuda").to(torch.bfloat16)

def block(m):
    wq = sp.fp4_quantize_microscaled(big)
    y = sp.fp4_gemm_microscaled(*sp.fp4_rmsnorm_quantize_microscaled(x[m], w, 1e-5)[:3], *wq)
    return sp.fp8_silu_mul_quantize_pertoken(y)[0]

for m in x:
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = block(m)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, block(m)) and bool(got.any()), m
print("same")
"""


def test_first_calls_of_a_process_may_be_captured():
    """No call prepares anything that a capture does not allow."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS_IN_A_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


def test_calls_from_two_threads():
    """Two threads on streams of their own, from a process's point of view at once."""
    torch.manual_seed(3)
    w = sp().fp4_quantize_microscaled(torch.randn(768, 1024, device=DEV).to(torch.bfloat16))
    xs = [torch.randn(m, 1024, device=DEV).to(torch.bfloat16) for m in (1, 300)]

    def run(x):
        return sp().fp4_gemm_microscaled(*sp().fp4_quantize_microscaled(x), *w)

    want = [run(x) for x in xs]
    torch.cuda.synchronize()
    same = [False, False]

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            got = [run(xs[i]) for _ in range(50)]
            torch.cuda.current_stream().synchronize()
            same[i] = all(torch.equal(g, want[i]) for g in got)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert same == [True, True]


def test_calls_on_two_streams_at_once_and_after_foreign_work():
    """Calls on side streams, each behind the kernel that makes its input."""
    fmt = "mxfp4"
    w = torch.randn(1024, 512, device=DEV).to(torch.bfloat16)
    wq = sp().fp4_quantize_microscaled(w, fmt)
    xs = [torch.randn(m, 512, device=DEV).to(torch.bfloat16) for m in (1, 70, 260, 1)]
    want = [sp().fp4_gemm_microscaled(*sp().fp4_quantize_microscaled(2 * x, fmt), *wq, fmt) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(5):
        got = []
        for x, s in zip(xs, streams):
            with torch.cuda.stream(s):
                got.append(sp().fp4_gemm_microscaled(*sp().fp4_quantize_microscaled(2 * x, fmt), *wq, fmt))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_python_refusals():
    m = sp()
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    q, b, s = m.fp4_quantize_microscaled(x)
    E = m.Sp24Error
    for bad in (x.float(), x[0], x.t(), x[:, :48].contiguous(), x[:0]):
        with pytest.raises(E):
            m.fp4_quantize_microscaled(bad)
        with pytest.raises(E):
            m.fp4_rmsnorm_quantize_microscaled(bad, w, 1e-5)
    with pytest.raises(E):
        m.fp4_quantize_microscaled(x, "fp4")
    for bad in (dict(q=q[:2]), dict(block_scales=b[:256]), dict(row_scales=s.double()), dict(q=q.cpu())):
        with pytest.raises(E):
            m.fp4_quantize_microscaled(x, out=bad)
    with pytest.raises(E):
        m.fp4_quantize_microscaled(x, status=torch.zeros(1, device=DEV))
    for kw in (dict(weight=w[:32]), dict(weight=w.float()), dict(residual=x[:2]), dict(residual=x.float()),
               dict(residual_out=x), dict(residual=x, residual_out=x.cpu()), dict(eps=-1.0), dict(eps=float("nan"))):
        with pytest.raises(E):
            m.fp8_rmsnorm_quantize_pertoken(x, **{"weight": w, "eps": 1e-5, **kw})
    with pytest.raises(E):
        m.fp8_silu_mul_quantize_pertoken(x[:, :33].contiguous())
    with pytest.raises(E):
        m.fp4_unpack_e4m3(q.view(torch.int8))
    for args in ((q, b, s[:2], q, b, s), (q, b[:256], s, q, b, s), (q, b, s, q[:, :16].contiguous(), b, s),
                 (q, b, s, q, b, s.cpu()), (q, b, s, q[:3], b, s), (q.view(torch.int8), b, s, q, b, s)):
        with pytest.raises(E):
            m.fp4_gemm_microscaled(*args)
    y = torch.zeros(4, 4, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(E):      # N = 4
        m.fp4_gemm_microscaled(q, b, s, q, b, s, out=y)
    with pytest.raises(E):      # out is of another type
        m.fp4_gemm_microscaled(q, b, s, torch.cat([q, q]), b, None, out=torch.zeros(4, 8, device=DEV))


def test_matrices_of_the_right_size_and_the_wrong_shape_are_refused():
    m = sp()
    x = torch.ones(4, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    q, b, s = m.fp4_quantize_microscaled(x)
    wq, wb, ws = m.fp4_quantize_microscaled(torch.ones(8, 64, dtype=torch.bfloat16, device=DEV))
    for call in (lambda: m.fp8_rmsnorm_quantize_pertoken(x, w, 1e-5, residual=x.view(64, 4)),
                 lambda: m.fp4_rmsnorm_quantize_microscaled(x, w, 1e-5, residual=x.view(8, 32)),
                 lambda: m.fp4_rmsnorm_quantize_microscaled(x, w, 1e-5, residual=x, residual_out=torch.empty_like(x).view(-1)),
                 lambda: m.fp4_quantize_microscaled(x, out=dict(q=q.view(8, 16))),
                 lambda: m.fp8_silu_mul_quantize_pertoken(x, out=dict(q=torch.empty(8, 16, dtype=torch.uint8, device=DEV))),
                 lambda: m.fp4_unpack_e4m3(q, out=torch.empty(8, 32, dtype=torch.uint8, device=DEV)),
                 lambda: m.fp4_gemm_microscaled(q, b, s, wq, wb, ws, out=torch.empty(8, 4, dtype=torch.bfloat16, device=DEV)),
                 lambda: m.fp4_gemm_microscaled(q, b, s, wq.view(16, 16), wb, ws)):
        with pytest.raises(m.Sp24Error):
            call()


def same_as_float64(y, xv, wv, xs, ws, band=2048):
    """check_product of every value, in bands of rows."""
    for i in range(0, y.shape[0], band):
        check_product(y[i:i + band], xv[i:i + band], wv, xs[i:i + band], ws)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("m,n,k", [(8192, 16384, 64), (8192, 16384, 256), (5000, 24600, 128), (16384, 4104, 320)])
def test_product_of_many_tiles_and_short_sums(fmt, m, n, k):
    """Tens of tiles for each pair of SMs whose epilogues take longer than
    their products: a tile's products must wait until both SMs have read the
    accumulator columns that they reuse.  Every value, several times."""
    xc, xb, xq, xt = operand(m, k, fmt, 9000 + k)
    wc, wb, wq, wt = operand(n, k, fmt, 9100 + n)
    g = torch.Generator(device=DEV).manual_seed(k)
    xs, ws = torch.rand(m, device=DEV, generator=g) + 0.5, torch.rand(n, device=DEV, generator=g) + 0.5
    st = status()
    y = sp().fp4_gemm_microscaled(xq, xt, xs, wq, wt, ws, fmt, status=st)
    same_as_float64(y, dev_values(xc, xb, fmt), dev_values(wc, wb, fmt), xs, ws)
    out = torch.empty_like(y)
    for _ in range(8):
        out.fill_(7.0)
        assert torch.equal(sp().fp4_gemm_microscaled(xq, xt, xs, wq, wt, ws, fmt, out=out, status=st), y)
    assert int(st.item()) == 0


LONG = (1 << 28) + 65536 + 32     # columns past which scale offsets pass 2^31, and segments the grid's second axis


def ends_of(blocks, q, lo, size, per_tile):
    """Codes and scale tiles of the first and the last columns of a row of one band."""
    return (q[:, :size // 2], blocks[:size // per_tile * 512]), (q[:, lo // 2:], blocks[lo // per_tile * 512:])


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("stage", ["plain", "gate"])
def test_rows_of_2_to_28_columns(fmt, stage):
    """The first and last columns of a very long row are quantised as in rows
    of their own with the same largest value."""
    per_tile, size = 4 * MO.BLOCK[fmt], 65536
    lo = LONG // per_tile * per_tile - size
    g = torch.Generator(device=DEV).manual_seed(5)

    def made():
        t = torch.randn(1, LONG, device=DEV, generator=g, dtype=torch.bfloat16)
        t[0, 3] = t[0, lo + 7] = 20.0
        return t

    parts = [made() for _ in range(1 if stage == "plain" else 2)]
    call = sp().fp4_quantize_microscaled if stage == "plain" else sp().fp4_silu_mul_quantize_microscaled
    st = status()
    q, b, s = call(torch.cat(parts, 1), fmt, status=st)
    assert int(st.item()) == 0
    for (gq, gb), cols in zip(ends_of(b, q, lo, size, per_tile), (slice(0, size), slice(lo, None))):
        q1, b1, s1 = call(torch.cat([t[:, cols] for t in parts], 1), fmt)
        assert torch.equal(gq, q1) and torch.equal(gb, b1) and (s is None or torch.equal(s, s1))


@pytest.mark.parametrize("fmt,cols", [("nvfp4", LONG), ("mxfp4", 2 * LONG)])
def test_norm_of_rows_of_2_to_28_columns(fmt, cols):
    """A row and weights that repeat: so do the codes and the block scales."""
    per_tile, period = 4 * MO.BLOCK[fmt], 65536
    x = dev_bf16(WL.random_bits((1, period), 51)).repeat(1, cols // period + 1)[:, :cols].contiguous()
    w = dev_bf16(WL.random_bits((1, period), 52)[0]).repeat(cols // period + 1)[:cols].contiguous()
    st = status()
    q, b, s, h = sp().fp4_rmsnorm_quantize_microscaled(x, w, 1e-5, fmt, status=st)
    assert int(st.item()) == 0 and h is x
    lo = cols // period * period
    tail = cols - lo
    assert torch.equal(q[:, lo // 2:], q[:, :tail // 2])
    scales = b.view(-1, 512)[:, :4].reshape(-1)      # row 0 of each tile, blocks in order
    n, first = tail // MO.BLOCK[fmt], lo // MO.BLOCK[fmt]
    assert torch.equal(scales[first:first + n], scales[:n]) and bool(scales[:n].any())
    whole = q[:, :lo // 2].view(-1, period // 2)
    assert bool((whole == whole[:1]).all())
    ws = scales[:first].view(-1, period // MO.BLOCK[fmt])
    assert bool((ws == ws[:1]).all())
    q1, b1, s1, _ = sp().fp4_rmsnorm_quantize_microscaled(x[:, :period].contiguous(), w[:period].contiguous(), 1e-5, fmt)
    if fmt == "nvfp4":                               # without the root, which enters the row's scale only
        assert torch.equal(q1, q[:, :period // 2]) and torch.equal(b1, b[:period // per_tile * 512])
        # squares are added over 1024 threads of two lanes, cols / 2048 additions deep (the short row: 32), and the
        # root halves their error; joining the threads, mean, root and scale are 20 roundings on either side; the
        # last 32 columns weigh 32 * max(x)^2 / cols, which is below 2^-20 for |x| < 8
        assert abs(s.item() / s1.item() - 1) < (cols / 4096 + 16 + 40) * U + 2.0 ** -20


@pytest.mark.parametrize("stage", ["norm", "gate"])
def test_codes_are_weights_behind_a_quantiser(stage):
    """E4M3 codes of a row stage as the dense FP8 GEMM's weights, with the short
    quantisation of X in between: the GEMM's early loads of weights must not
    start while the stage still writes them."""
    n, k = 4096, 2048
    m = sp()
    x8 = dev_bf16(WL.random_bits((8, k), 23))
    xq, sx = m.fp8_quantize_pertensor(x8)
    one = torch.ones(1, device=DEV)
    w = dev_bf16(WL.random_bits((1, k), 24)[0])
    ins = [torch.randn(n, k if stage == "norm" else 2 * k, device=DEV).to(torch.bfloat16) for _ in range(2)]
    out = dict(q=torch.empty(n, k, dtype=torch.uint8, device=DEV), scales=torch.empty(n, device=DEV))

    def codes(x):
        if stage == "norm":
            m.fp8_rmsnorm_quantize_pertoken(x, w, 1e-5, out=out)
        else:
            m.fp8_silu_mul_quantize_pertoken(x, out=out)

    want = []
    for x in ins:
        codes(x)
        torch.cuda.synchronize()
        want.append(m.fp8_gemm_dense(xq, sx, out["q"], one))
        torch.cuda.synchronize()
    assert not torch.equal(*want)
    y = torch.empty_like(want[0])
    ws = m.Workspace(DEV)
    same = torch.ones((), dtype=torch.bool, device=DEV)

    def run(i):
        codes(ins[i])
        a, sa = m.fp8_quantize_pertensor(x8, workspace=ws)
        m.fp8_gemm_dense(a, sa, out["q"], one, out=y, workspace=ws)
        same.logical_and_((y == want[i]).all())

    graphs = []
    for i in range(2):
        run(i)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            run(i)
    for i in range(100):
        graphs[i % 2].replay()
        run(i % 2)
    assert bool(same)


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("cols", [64, 4096, 40032])
@pytest.mark.parametrize("size", [1e-4, 1e-10, 1e-12, 1e-19, 1e-20, 1e-25, 1e-38])
def test_norm_of_small_rows_whose_products_are_zero(fmt, cols, size):
    """Without eps, rows that are small but not zero under weights that are zero
    wherever the row is not: zero codes, the scale 1, no status."""
    x, w = np.zeros((2, cols)), np.ones(cols)
    x[0, ::2], x[1, 5] = -size, size
    w[::2], w[5] = 0.0, 0.0
    X, W, st = dev_bf16(WL.to_bf16_bits(x)), dev_bf16(WL.to_bf16_bits(w)), status()
    if fmt == "e4m3":
        q, s, _ = sp().fp8_rmsnorm_quantize_pertoken(X, W, 0.0, status=st)
    else:
        q, b, s, _ = sp().fp4_rmsnorm_quantize_microscaled(X, W, 0.0, fmt, status=st)
        assert not b.any()
        q = torch.from_numpy(unpack(q) & 7)
    assert not (q & 0x7F).any() and (s is None or s.tolist() == [1.0, 1.0]) and int(st.item()) == 0


@pytest.mark.parametrize("fmt", ["e4m3", "nvfp4", "mxfp4"])
@pytest.mark.parametrize("cols", [96, 4096, 40032])
def test_norm_of_rows_whose_squares_vanish(fmt, cols):
    """Without eps, a row whose mean square is 0 in fp32 is a row of zeros,
    under weights of any size."""
    x, w = np.full((2, cols), 2.0 ** -80), np.full(cols, 2.0 ** 120)
    x[1] = 1.0
    st = status()
    X, W = dev_bf16(WL.to_bf16_bits(x)), dev_bf16(WL.to_bf16_bits(w))
    if fmt == "e4m3":
        q, s, _ = sp().fp8_rmsnorm_quantize_pertoken(X, W, 0.0, status=st)
    else:
        q, _, s, _ = sp().fp4_rmsnorm_quantize_microscaled(X, W, 0.0, fmt, status=st)
    assert not q[0].any() and bool(q[1].all()) and (s is None or s[0].item() == 1.0) and int(st.item()) == 0


@pytest.mark.parametrize("fmt,size,weight", [("e4m3", 2.0 ** -12, 2.0 ** -121), ("e4m3", 2.0 ** 40, 2.0 ** -122),
                                             ("nvfp4", 2.0 ** -30, 2.0 ** -93), ("nvfp4", 2.0 ** 50, 2.0 ** -95)])
@pytest.mark.parametrize("cols", [96, 4096, 40032])
def test_norm_of_rows_below_the_least_scale(fmt, size, weight, cols):
    """Rows whose largest value is below what the least row scale stands for."""
    x, w = WL.random_bits((3, cols), 31, scale=size), WL.random_bits((1, cols), 32, scale=weight)[0]
    y, _ = MO.rmsnorm(x, None, w, 0.0)
    # h * w is rounded to a multiple of 2^-149
    z = np.abs(O.bf16_to_f32(x).astype(np.float64) * O.bf16_to_f32(w).astype(np.float64))
    d = norm_error(cols) + np.where(z > 0, 2.0 ** -150 / np.where(z > 0, z, 1.0), 0.0)
    assert np.abs(y).max() < (448.0 * 2.0 ** -126 if fmt == "e4m3" else MO.ROW_FLOOR)
    X, W, st = dev_bf16(x), dev_bf16(w), status()
    if fmt == "e4m3":
        q, s, _ = sp().fp8_rmsnorm_quantize_pertoken(X, W, 0.0, status=st)
        assert s.tolist() == [2.0 ** -126] * 3
        check_e4m3(q, s, y, d)
    else:
        q, b, s, _ = sp().fp4_rmsnorm_quantize_microscaled(X, W, 0.0, fmt, status=st)
        assert s.tolist() == [2.0 ** -100] * 3
        check_fp4(q, b, s, y, d, fmt)
    assert int(st.item()) == 0


def test_product_of_the_longest_sum():
    """K at its limit: what lies at either end of the row arrives, alone."""
    m, n, k, end = 1, 8, (1 << 31) - 256, 512
    n_end, tile = end // 32, 512
    xc, xb, xq, xt = operand(m, 2 * end, "mxfp4", 41)
    wc, wb, wq, wt = operand(n, 2 * end, "mxfp4", 42)

    def long(q, t, rows):
        lq = torch.zeros(rows, k // 2, dtype=torch.uint8, device=DEV)
        lt = torch.zeros(k // 128 * tile, dtype=torch.uint8, device=DEV)
        for got, src, cut in ((lq, q, end // 2), (lt.view(1, -1), t.view(1, -1), n_end // 4 * tile)):
            got[:, :cut], got[:, -cut:] = src[:, :cut], src[:, -cut:]
        return lq, lt

    (lxq, lxt), (lwq, lwt), st = long(xq, xt, m), long(wq, wt, n), status()
    y = sp().fp4_gemm_microscaled(lxq, lxt, None, lwq, lwt, None, "mxfp4", status=st)
    check_product(y, dev_values(xc, xb, "mxfp4"), dev_values(wc, wb, "mxfp4"), None, None)
    assert int(st.item()) == 0 and bool(y.any())


@pytest.mark.parametrize("stage", ["nvfp4", "mxfp4", "norm e4m3", "norm nvfp4", "gate e4m3", "gate mxfp4", "unpack"])
def test_last_rows_of_matrices_past_32_bit_offsets(stage):
    """More than 2^31 elements (and 2^32 bytes in each input), whose last rows
    are like no others: they come out as from a call of their own, and not as
    rows that lie 2^31 elements or 2^32 bytes before them."""
    rows, cols = 131200, 32768
    lo = rows - 128
    op, _, fmt = stage.partition(" ")
    m, g = sp(), torch.Generator(device=DEV).manual_seed(7)

    def made(width):
        t = torch.randn(512, width, device=DEV, generator=g).to(torch.bfloat16).repeat(-(-rows // 512), 1)[:rows]
        t[lo:] = torch.randn(rows - lo, width, device=DEV, generator=g).to(torch.bfloat16)
        return t

    if op == "norm":
        ins = [made(cols)]
        w = dev_bf16(WL.random_bits((1, cols), 8)[0])
        if fmt == "e4m3":
            ins.append(made(cols))
            call = lambda x, r: m.fp8_rmsnorm_quantize_pertoken(x, w, 1e-5, residual=r)
        else:
            call = lambda x: m.fp4_rmsnorm_quantize_microscaled(x, w, 1e-5, fmt)[:3]
    elif op == "gate":
        ins = [made(2 * cols)]
        call = m.fp8_silu_mul_quantize_pertoken if fmt == "e4m3" else lambda x: m.fp4_silu_mul_quantize_microscaled(x, fmt)
    elif op == "unpack":
        ins = [torch.randint(0, 256, (512, cols), device=DEV, generator=g, dtype=torch.uint8).repeat(-(-rows // 512), 1)[:rows]]
        ins[0][lo:] = torch.randint(0, 256, (rows - lo, cols), device=DEV, generator=g, dtype=torch.uint8)
        call = lambda x: (m.fp4_unpack_e4m3(x),)
    else:
        ins = [made(cols)]
        call = lambda x: m.fp4_quantize_microscaled(x, op)
    got = call(*ins)
    want = call(*(t[lo:].contiguous() for t in ins))
    other = call(*(t[lo - 65536:lo - 65536 + 128].contiguous() for t in ins))
    assert not torch.equal(other[0], want[0])
    for a, b in zip(got, want):
        if a is not None:
            # blocks' scales: the last band of 128 rows
            assert torch.equal(a[-b.numel():] if a.dim() == 1 else a[lo:], b)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("n", [8, 256])
def test_product_of_rows_past_32_bit_offsets(fmt, n):
    """Codes of more than 2^31 bytes whose last rows are like no others."""
    rows, cols = 131200, 32768 + 128
    x = torch.randn(512, cols, device=DEV).to(torch.bfloat16)
    x = x.repeat(-(-rows // 512), 1)[:rows]
    x[-128:] = torch.randn(128, cols, device=DEV).to(torch.bfloat16)
    q, b, s = sp().fp4_quantize_microscaled(x, fmt)
    del x
    assert q.numel() > 1 << 31
    w = sp().fp4_quantize_microscaled(torch.randn(n, cols, device=DEV).to(torch.bfloat16), fmt)
    size = b.numel() // (rows // 128)
    wv = dev_values(unpack(w[0]), rows_of(w[1], n, cols, fmt), fmt)

    def check(y, lo):
        bt = b[lo // 128 * size:(lo // 128 + 1) * size]
        xv = dev_values(unpack(q[lo:lo + 128]), rows_of(bt, 128, cols, fmt), fmt)
        check_product(y, xv, wv, None if s is None else s[lo:lo + 128], w[2])

    y = sp().fp4_gemm_microscaled(q, b, s, *w, fmt)
    for lo in (0, 65536, rows - 256, rows - 128):
        check(y[lo:lo + 128], lo)
    # and as the weights
    y = sp().fp4_gemm_microscaled(*w, q, b, s, fmt)
    for lo in (0, 65536, rows - 256, rows - 128):
        check(y[:, lo:lo + 128].t(), lo)


def masked(b, rows, cols, fmt, keep):
    return MO.from_tiles(b.cpu().numpy(), rows, cols // MO.BLOCK[fmt])[keep]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("stage", ["norm", "norm residual", "gate"])
@pytest.mark.parametrize("bad", ["inf", "nan", "overflow"])
@pytest.mark.parametrize("rows,cols", [(5, 96), (900, 2048), (5, 20000 // 32 * 32), (3, 40032)])
def test_fp4_row_stages_flag_nonfinite_rows_and_keep_the_others(fmt, stage, bad, rows, cols):
    """One value of a row that is not finite, or whose product (the norm's: its
    square, or the sum with the residual) leaves its type's range."""
    m, at = sp(), cols - 3
    x = WL.random_bits((rows, 2 * cols if stage == "gate" else cols), 8)
    r = WL.random_bits((rows, cols), 10)
    w = dev_bf16(WL.random_bits((1, cols), 9)[0])

    def call(x, r, st=None):
        if stage == "gate":
            return m.fp4_silu_mul_quantize_microscaled(dev_bf16(x), fmt, status=st)
        return m.fp4_rmsnorm_quantize_microscaled(dev_bf16(x), w, 1e-5, fmt, status=st,
                                                  residual=dev_bf16(r) if stage == "norm residual" else None)

    st = status()
    good = call(x, r, st)
    assert int(st.item()) == 0
    x[1, at] = dict(inf=0xFF80, nan=0x7FC0, overflow=0x7F7F)[bad]
    if bad == "overflow":
        r[1, at] = 0x7F7F
        if stage == "gate":
            x[1, cols + at] = 0x7F00
    got = call(x, r, st)
    assert int(st.item()) == m._lib.SP24_STATUS_NONFINITE
    keep = [0] + list(range(2, rows))
    assert torch.equal(got[0][keep], good[0][keep])
    assert np.array_equal(masked(got[1], rows, cols, fmt, keep), masked(good[1], rows, cols, fmt, keep))
    assert got[2] is None or torch.equal(got[2][keep], good[2][keep])
    if stage != "gate":
        assert torch.equal(got[3][keep], good[3][keep])


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("where", ["x", "residual"])
@pytest.mark.parametrize("rows,cols", [(9, 64), (9, 4096), (700, 4096), (300, 11008), (5, 40032)])
def test_fp4_norm_in_place(fmt, where, rows, cols):
    x, r = WL.random_bits((rows, cols), 61), WL.random_bits((rows, cols), 62)
    w = dev_bf16(WL.random_bits((1, cols), 63)[0])
    want = sp().fp4_rmsnorm_quantize_microscaled(dev_bf16(x), w, 1e-6, fmt, residual=dev_bf16(r))
    X, R = dev_bf16(x), dev_bf16(r)
    target = X if where == "x" else R
    got = sp().fp4_rmsnorm_quantize_microscaled(X, w, 1e-6, fmt, residual=R, residual_out=target)
    assert got[3] is target
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, want))
