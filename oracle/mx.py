"""Reference of the MXFP4 operators and of the RMS norm with a quantised output, in float64 (numpy).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).  Written from the definitions in ``include/dg.h``; pinned in
``tests/test_oracle_mx.py``.
"""

import numpy as np
from scipy.special import ndtr

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


def sandwich_norm(x, residual, post_weight, gate, scale, eps):
    """float64 arrays, gate [m, k] by row (post_weight and gate may be None) -> (h unrounded [m, k], rx [m])."""
    rx = 1.0 / np.sqrt(np.mean(x * x, axis=1) + eps) if post_weight is not None else np.ones(len(x))
    n = x * rx[:, None] * (1.0 if post_weight is None else post_weight)
    return residual + scale * (1.0 if gate is None else gate) * n, rx


def sandwich_norm_backward(dy, dh, x, h, post_weight, gate, weight, rx, r, scale):
    """float64 arrays, gate [m, k] by row (dh, post_weight and gate may be None; rx is 1 without post_weight) ->
    (D = dresidual, dx, dy * n, v * nx, scale * post_weight * D * nx); the last three [m, k], to be summed over rows."""
    n, nx = h * r[:, None], x * rx[:, None]
    a = dy * weight
    d = r[:, None] * (a - n * np.mean(a * n, axis=1, keepdims=True))
    if dh is not None:
        d = d + dh
    v = scale * (1.0 if gate is None else gate) * d
    u = v if post_weight is None else v * post_weight
    dx = u if post_weight is None else rx[:, None] * (u - nx * np.mean(u * nx, axis=1, keepdims=True))
    return d, dx, dy * n, v * nx, scale * (1.0 if post_weight is None else post_weight) * d * nx


def activation(u, name):
    """float64 -> (act(u), act'(u)); ReLU's derivative at 0 is 0."""
    if name == "none":
        return u, np.ones_like(u)
    if name == "relu":
        return np.maximum(u, 0), (u > 0).astype(np.float64)
    with np.errstate(over="ignore"):
        if name == "gelu":
            phi = ndtr(u)
            return u * phi, phi + u * np.exp(-u * u / 2) / np.sqrt(2 * np.pi)
        c = np.sqrt(2 / np.pi)
        w, dw = (u, 1.0) if name == "silu" else (2 * c * (u + 0.044715 * u ** 3), 2 * c * (1 + 3 * 0.044715 * u ** 2))
        s, not_s = 1 / (1 + np.exp(-w)), 1 / (1 + np.exp(w))
        return u * s, s + u * s * not_s * dw


def linear_epilogue(u, name, gated, residual=None):
    """u [m, n] float64 -> d unrounded."""
    half = u.shape[1] // 2
    y = activation(u[:, :half], name)[0] * u[:, half:] if gated else activation(u, name)[0]
    return y if residual is None else y + residual


def linear_epilogue_backward(dy, z, name, gated):
    """dz [m, n], unrounded."""
    if not gated:
        return dy * activation(z, name)[1]
    half = z.shape[1] // 2
    a, d = activation(z[:, :half], name)
    return np.hstack([dy * z[:, half:] * d, dy * a])


def group_rows(ms, m):
    """Row counts -> [(first row, end)] of each group: negative counts are 0, rows are cut at m."""
    ends = np.minimum(np.cumsum(np.maximum(np.asarray(ms, dtype=np.int64), 0)), m)
    return list(zip(np.concatenate([[0], ends[:-1]]).astype(int), ends.astype(int)))


def quantize_mxfp4_ragged(x, ms, blocks):
    """float64 [m, k] -> (qt [k, 64 blocks], sft [blocks, k], 128-row blocks used): each group's rows quantised along the
    rows, padded to 128, one group behind another."""
    m, k = x.shape
    qt, sft, at = np.zeros((k, blocks * 64), np.uint8), np.zeros((blocks, k), np.int32), 0
    for s, e in group_rows(ms, m):
        if e > s:
            q, sf = quantize_mxfp4_transposed(x[s:e])
            nb = sf.shape[0]
            qt[:, at * 64:(at + nb) * 64], sft[at:at + nb], at = q, sf, at + nb
    return qt, sft, at


def m_grouped_mxfp4_gemm_nt_ragged(a, a_sf, b, b_sf, ms):
    """[(rows of a group, its D unrounded float64, sum |a b|)]."""
    av = dequant_mxfp4(a, a_sf)
    out = []
    for g, (s, e) in enumerate(group_rows(ms, len(av))):
        bv = dequant_mxfp4(b[g], b_sf[g]) if e > s else np.zeros((b.shape[1], av.shape[1]))
        out.append((slice(s, e), av[s:e] @ bv.T, np.abs(av[s:e]) @ np.abs(bv).T))
    return out


def k_grouped_mxfp4_gemm_nt_ragged(a, a_sf, b, b_sf, ms):
    """(D [G, m, n] unrounded float64, sum |a b|)."""
    av, bv = dequant_mxfp4(a, a_sf), dequant_mxfp4(b, b_sf)
    kb, at, d, s = a_sf.shape[0], 0, [], []
    for rows in ms:
        end = min(kb, at + (max(int(rows), 0) + 127) // 128)
        k = slice(at * 128, end * 128)
        d.append(av[:, k] @ bv[:, k].T)
        s.append(np.abs(av[:, k]) @ np.abs(bv[:, k]).T)
        at = end
    return np.stack(d), np.stack(s)
