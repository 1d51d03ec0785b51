"""Reference of the MXFP4 operators and of the RMS norm with a quantised output, in float64 (numpy).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  Written from the definitions in ``include/dg.h``; pinned in
``tests/test_oracle_mx.py``.
"""

import numpy as np

from .formats import (
    E2M1_TABLE,
    E4M3_TABLE,
    bf16_bits_to_f64,
    pow2_scale_exponent,
    round_to_bf16,
    unpack_e2m1,
    unpack_ue8m0_int32,
)

E2M1_GRID = E2M1_TABLE[:8]                # 0 .. 6, increasing
E4M3_GRID = E4M3_TABLE[:0x7F]             # 0 .. 448, increasing


def nearest_code(x, grid) -> np.ndarray:
    """|x| (float64, on or below grid's end) -> the index of the nearest grid value, ties to the even index."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    hi = np.minimum(np.searchsorted(grid, a, side="left"), len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    over, under = grid[hi] - a, a - grid[lo]
    return np.where((over < under) | ((over == under) & (hi % 2 == 0)), hi, lo)


def mx_blocks(x):
    """float64 [R, C], C a multiple of 32 -> (codes uint8 [R, C], exponent bytes [R, C/32]): per 32 values the
    smallest e >= -127 with 6 * 2^e >= max|x|; a block with a NaN or an infinity: byte 255, codes 0."""
    x = np.asarray(x, dtype=np.float64)
    R, C = x.shape
    b = x.reshape(R, C // 32, 32)
    finite = np.isfinite(b).all(axis=2)
    safe = np.where(finite[..., None], b, 0.0)
    e = np.maximum(pow2_scale_exponent(np.abs(safe).max(axis=2), 6.0), -127)
    scaled = np.ldexp(safe, -e[..., None])
    code = nearest_code(scaled, E2M1_GRID) + 8 * np.signbit(scaled)
    byte = np.where(finite, e + 127, 255)
    return np.where(finite[..., None], code, 0).reshape(R, C).astype(np.uint8), byte.astype(np.uint8)


def pack_pairs(codes) -> np.ndarray:
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def pack_words(byte) -> np.ndarray:
    """Exponent bytes [R, S], S a multiple of 4 -> int32 [R, S/4], byte i of a word from the least significant end."""
    b = byte.reshape(byte.shape[0], -1, 4).astype(np.uint32)
    return (b[..., 0] | b[..., 1] << 8 | b[..., 2] << 16 | b[..., 3] << 24).view(np.int32)


def quantize_mxfp4(x):
    """float64 [m, k] -> (q [m, k/2] uint8, sf [k/128, m] int32, values [m, k] float64)."""
    codes, byte = mx_blocks(x)
    with np.errstate(invalid="ignore"):
        scale = np.where(byte == 255, np.nan, np.ldexp(1.0, byte.astype(np.int64) - 127))
        values = E2M1_TABLE[codes] * np.repeat(scale, 32, axis=1)
    return pack_pairs(codes), np.ascontiguousarray(pack_words(byte).T), values


def quantize_mxfp4_transposed(x):
    """float64 [m, k] -> (qt [k, mp/2], sft [mp/128, k]): the transpose, rows m .. mp-1 zero, quantised along m."""
    x = np.asarray(x, dtype=np.float64)
    m, k = x.shape
    full = np.zeros((k, (m + 127) // 128 * 128))
    full[:, :m] = x.T
    q, sf, _ = quantize_mxfp4(full)
    return q, sf


def dequant_mxfp4(q, sf) -> np.ndarray:
    """q [r, k/2], sf [k/128, r] -> float64 [r, k]."""
    scale = unpack_ue8m0_int32(np.ascontiguousarray(np.asarray(sf).T))            # [r, k/32]
    with np.errstate(invalid="ignore"):
        return unpack_e2m1(q) * np.repeat(scale, 32, axis=1)


def mxfp4_gemm_nt(a, a_sf, b, b_sf, c=None) -> np.ndarray:
    """D = C + A . B^T, unrounded float64 [m, n]."""
    ref = dequant_mxfp4(a, a_sf) @ dequant_mxfp4(b, b_sf).T
    return ref if c is None else ref + bf16_bits_to_f64(c)


def add_rms_norm(x, residual, weight, eps):
    """bf16 bits -> (h float64 on the bf16 grid, r [m], y [m, k] unrounded)."""
    h = bf16_bits_to_f64(x)
    if residual is not None:
        h = round_to_bf16(h + bf16_bits_to_f64(residual))
    r = 1.0 / np.sqrt(np.mean(h * h, axis=1) + eps)
    return h, r, h * r[:, None] * bf16_bits_to_f64(weight)


def add_rms_norm_backward(dy, dh, h, weight, r):
    """float64 arrays (dh may be None) -> (dx [m, k], dweight [k])."""
    n = h * r[:, None]
    g = dy * weight
    dx = r[:, None] * (g - n * np.mean(g * n, axis=1, keepdims=True))
    return dx if dh is None else dx + dh, np.sum(dy * n, axis=0)
