"""Plain float64 reference of block-scaled FP4 and of the row stages that
quantise their output (root-mean-square norm, gated activation).

Test infrastructure; shares no code with the CUDA kernels.  Quotients of bf16
values are formed in float64 from exact products, so every tie is met exactly
(numerator and denominator have at most 13 and 12 significant bits: a quotient
that is not on a rounding boundary is at least 2^-14 away from it).
"""
from __future__ import annotations

import numpy as np

from . import sp24_oracle as O

BLOCK = {"nvfp4": 16, "mxfp4": 32}
ROW_FLOOR = 2688.0 * 2.0 ** -100


def tile_offsets(rows: int, n: int) -> np.ndarray:
    """Byte offset of block scale (row, block) in the tiles of 128 rows x 4 scales."""
    r = np.arange(rows)[:, None]
    b = np.arange(n)[None, :]
    wide = (n + 3) // 4
    return ((r // 128) * wide + b // 4) * 512 + (r % 32) * 16 + (r // 32 % 4) * 4 + b % 4


def tile_bytes(rows: int, n: int) -> int:
    return (rows + 127) // 128 * ((n + 3) // 4) * 512


def to_tiles(scales: np.ndarray) -> np.ndarray:
    """[rows, n] scale bytes in tile order; zero outside the matrix."""
    rows, n = scales.shape
    out = np.zeros(tile_bytes(rows, n), dtype=np.uint8)
    out[tile_offsets(rows, n)] = scales
    return out


def from_tiles(tiles: np.ndarray, rows: int, n: int) -> np.ndarray:
    return np.asarray(tiles)[tile_offsets(rows, n)]


def e2m1_codes(v: np.ndarray) -> np.ndarray:
    """E2M1 code of float64 values: nearest, ties to the even code, saturating,
    the sign kept on a value that rounds to zero."""
    a = np.abs(np.asarray(v, dtype=np.float64))
    code = ((a > 0.25).astype(np.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return (code + np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def row_top(amax: np.ndarray) -> np.ndarray:
    """R of each row: the row's amax, at least 2688 * 2^-100."""
    return np.maximum(amax, ROW_FLOOR)


def nvfp4_row_scale(amax: np.ndarray) -> np.ndarray:
    s = (row_top(amax).astype(np.float32) / np.float32(2688.0)).astype(np.float32)
    return np.where(amax == 0, np.float32(1.0), s).astype(np.float32)


def nvfp4_block_bytes(block_amax: np.ndarray, amax: np.ndarray) -> np.ndarray:
    """E4M3 codes of 448 amax_b / R, the quotient rounded once to fp32."""
    return O.e4m3_encode((448.0 * block_amax / row_top(amax)[:, None]).astype(np.float32))


def mxfp4_block_bytes(block_amax: np.ndarray) -> np.ndarray:
    _, e = np.frexp(block_amax)          # amax = m 2^e, m in [0.5, 1)
    return np.where(block_amax == 0, 0, np.maximum(e - 1 - 2 + 127, 0)).astype(np.uint8)


def scale_values(byts: np.ndarray, fmt: str) -> np.ndarray:
    return O.e4m3_decode(byts) if fmt == "nvfp4" else np.ldexp(1.0, byts.astype(np.int32) - 127)


def codes_for(x: np.ndarray, byts: np.ndarray, amax: np.ndarray, fmt: str) -> np.ndarray:
    """Codes of float64 x [rows, cols] under given block-scale bytes."""
    rows, cols = x.shape
    sf = np.repeat(scale_values(byts, fmt), BLOCK[fmt], axis=1)
    if fmt == "mxfp4":
        return e2m1_codes(x / sf)
    d = sf * row_top(amax)[:, None]
    # a zero scale gives a zero of the element's sign
    return e2m1_codes(np.where(d > 0, 2688.0 * x / np.where(d > 0, d, 1.0), 0.0 * x))


def quantize(x: np.ndarray, fmt: str):
    """x float64 [rows, cols] -> (codes u8 one per element, block bytes [rows, n],
    row scales f32 [rows] or None)."""
    rows, cols = x.shape
    top = np.abs(x).reshape(rows, cols // BLOCK[fmt], BLOCK[fmt]).max(axis=2)
    amax = top.max(axis=1)
    byts = nvfp4_block_bytes(top, amax) if fmt == "nvfp4" else mxfp4_block_bytes(top)
    return codes_for(x, byts, amax, fmt), byts, (nvfp4_row_scale(amax) if fmt == "nvfp4" else None)


def values(codes: np.ndarray, byts: np.ndarray, fmt: str) -> np.ndarray:
    """code * block scale, float64 (without the row scales)."""
    return O.e2m1_decode(codes) * np.repeat(scale_values(byts, fmt), BLOCK[fmt], axis=1)


def rmsnorm(x_bits: np.ndarray, residual_bits, weight_bits: np.ndarray, eps: float):
    """(y float64, h bf16 bits): h = bf16(x + residual), y = h / sqrt(mean h^2 + eps) * w."""
    h = x_bits
    if residual_bits is not None:
        h = O.f32_to_bf16_rne(O.bf16_to_f32(x_bits) + O.bf16_to_f32(residual_bits))
    hv = O.bf16_to_f32(h).astype(np.float64)
    ms = (hv * hv).mean(axis=1, keepdims=True) + np.float64(np.float32(eps))
    rstd = np.where(ms > 0, 1.0 / np.sqrt(np.where(ms > 0, ms, 1.0)), 0.0)
    return hv * rstd * O.bf16_to_f32(weight_bits).astype(np.float64), h


def silu_mul(gu_bits: np.ndarray) -> np.ndarray:
    cols = gu_bits.shape[1] // 2
    v = O.bf16_to_f32(gu_bits).astype(np.float64)
    g, u = v[:, :cols], v[:, cols:]
    return g / (1.0 + np.exp(-np.clip(g, -700.0, None))) * u


def e4m3_row_scale(amax: np.ndarray) -> np.ndarray:
    """max(amax / 448, 2^-126), 1 for a zero row (float64)."""
    return np.where(amax == 0, 1.0, np.maximum(amax / 448.0, 2.0 ** -126))
