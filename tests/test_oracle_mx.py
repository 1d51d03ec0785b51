"""Pins of ``oracle/mx.py``: each function against an exact rational evaluation, a closed form, another library's
encoder or differences, and mistakes planted in the oracle that the pins have to catch."""

from fractions import Fraction

import numpy as np
import pytest
import torch

import synth
from oracle import formats as F
from oracle import mx as X

RNG = np.random.default_rng(11)


def exact_block(vals):
    """One block by rationals: the least e >= -127 with 6 * 2^e >= amax, nearest codes, ties to the even code."""
    fr = [Fraction(float(v)) for v in vals]
    amax = max(abs(f) for f in fr)
    e = 0
    if amax:
        e = -127
        while 6 * Fraction(2) ** e < amax:
            e += 1
    grid = [Fraction(float(g)) for g in X.E2M1_GRID]
    codes = []
    for f, v in zip(fr, vals):
        d = [abs(abs(f) / Fraction(2) ** e - g) for g in grid]
        best = [i for i in range(8) if d[i] == min(d)]
        codes.append((best[0] if len(best) == 1 else [i for i in best if i % 2 == 0][0]) + (8 if np.signbit(v) else 0))
    return codes, e + 127


def edge_blocks():
    """Blocks whose values sit on codes, on the midpoints between them and just beside, at several scales."""
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    base = [0.0, -0.0, 6.0, -6.0, 1.0, -0.5] + mids + [-m for m in mids]
    base += [np.nextafter(m, 0) for m in mids[:5]]
    base += [np.nextafter(m, 9) for m in mids[:7]]
    blocks = [np.float64(base)]
    blocks += [np.ldexp(blocks[0], s) for s in (-130, -126, -60, 1, 100)]
    blocks += [RNG.standard_normal(32), np.zeros(32), np.full(32, 6.0), np.full(32, np.nextafter(6.0, 9)),
               np.r_[2.0 ** -149, np.zeros(31)], np.r_[-3e38, RNG.standard_normal(31) * 1e38]]
    return np.stack(blocks)


def check_mx_blocks(fn):
    x = edge_blocks()
    codes, byte = fn(x)
    for i, row in enumerate(x):
        want, wb = exact_block(row)
        assert list(codes[i]) == want and byte[i, 0] == wb, i


def test_mx_blocks_against_rationals():
    check_mx_blocks(X.mx_blocks)


def test_mx_blocks_nonfinite():
    x = RNG.standard_normal((3, 64))
    x[0, 3], x[1, 40], x[2, 63] = np.nan, np.inf, -np.inf
    codes, byte = X.mx_blocks(x)
    assert [list(b) for b in (byte == 255)] == [[True, False], [False, True], [False, True]]
    assert not codes[0, :32].any() and not codes[1, 32:].any() and codes[0, 32:].any()
    assert np.isnan(X.quantize_mxfp4(np.tile(x, 2))[2][0, :32]).all()


def test_quantize_matches_the_generator_and_round_trips():
    x = torch.from_numpy(RNG.standard_normal((7, 384)).astype(np.float32))
    q, sf, values = X.quantize_mxfp4(x.double().numpy())
    gq, gsf = synth.quant_fp4_1x32(x)                          # torch-based encoder, scale words [R, C/128]
    assert np.array_equal(q, gq.numpy()) and np.array_equal(sf, gsf.numpy().T)
    assert np.array_equal(X.dequant_mxfp4(q, sf), values)
    again = X.quantize_mxfp4(values)
    assert np.array_equal(again[2], values)                    # codes are a fixed point of the rounding
    # each value is within half a step of its source: half the widest gap (4 .. 6) of the block's scale
    e = np.frexp(np.abs(x.numpy()).reshape(7, 12, 32).max(axis=2))[1]
    assert (np.abs(values - x.double().numpy()).reshape(7, 12, 32) <= np.ldexp(1.0, e - 2)[..., None]).all()


def test_transposed_pads_with_zeros():
    x = RNG.standard_normal((150, 128))
    q, sf = X.quantize_mxfp4_transposed(x)
    assert q.shape == (128, 128) and sf.shape == (2, 128)
    v = X.dequant_mxfp4(q, sf)
    assert not v[:, 150:].any() and np.array_equal(v[:, :128], X.quantize_mxfp4(x[:128].T.copy())[2])


def check_gemm(fn):
    # distinct powers of two per 32-block and small integers: every product is told apart, the sum is exact
    codes = RNG.integers(0, 16, (5, 256)).astype(np.uint8), RNG.integers(0, 16, (3, 256)).astype(np.uint8)
    byte = [(127 + RNG.integers(-4, 5, (c.shape[0], 8))).astype(np.uint8) for c in codes]
    a, b = (X.pack_pairs(c) for c in codes)
    sa, sb = (np.ascontiguousarray(X.pack_words(v).T) for v in byte)
    c = F.f64_to_bf16_bits(RNG.integers(-8, 9, (5, 3)).astype(np.float64))
    got = fn(a, sa, b, sb, c)
    for i in range(5):
        for j in range(3):
            s = Fraction(float(F.bf16_bits_to_f64(c)[i, j]))
            for k in range(256):
                s += (Fraction(float(F.E2M1_TABLE[codes[0][i, k]])) * Fraction(float(F.E2M1_TABLE[codes[1][j, k]]))
                      * Fraction(2) ** (int(byte[0][i, k // 32]) - 127 + int(byte[1][j, k // 32]) - 127))
            assert Fraction(float(got[i, j])) == s, (i, j)


def test_gemm_against_rationals():
    check_gemm(X.mxfp4_gemm_nt)


def test_norm_against_torch():
    x, res, w = (F.f64_to_bf16_bits(RNG.standard_normal(s)) for s in ((6, 256), (6, 256), (256,)))
    h, r, y = X.add_rms_norm(x, res, w, 1e-5)
    t = [torch.from_numpy(v.view(np.int16)).view(torch.bfloat16) for v in (x, res, w)]
    ht = (t[0].float() + t[1].float()).to(torch.bfloat16)
    assert np.array_equal(h, ht.double().numpy())
    want = torch.nn.functional.rms_norm(ht.double(), (256,), t[2].double(), 1e-5)
    np.testing.assert_allclose(y, want.numpy(), rtol=1e-13)


def check_backward(fn):
    rng = np.random.default_rng(5)
    h, dy, dh, w = rng.standard_normal((3, 128)), rng.standard_normal((3, 128)), rng.standard_normal((3, 128)), \
        rng.standard_normal(128)
    eps = 1e-3

    def loss(hh, ww):
        return float(np.sum(dy * hh / np.sqrt(np.mean(hh * hh, axis=1, keepdims=True) + eps) * ww) + np.sum(dh * hh))

    r = 1 / np.sqrt(np.mean(h * h, axis=1) + eps)
    dx, dw = fn(dy, dh, h, w, r)
    step = 1e-5                               # central differences: error ~ step^2 * third derivative, ~1e-8 here
    for i, j in ((0, 0), (1, 77), (2, 127)):
        hp, hm = h.copy(), h.copy()
        hp[i, j] += step
        hm[i, j] -= step
        assert abs((loss(hp, w) - loss(hm, w)) / (2 * step) - dx[i, j]) < 1e-7
        wp, wm = w.copy(), w.copy()
        wp[j] += step
        wm[j] -= step
        assert abs((loss(h, wp) - loss(h, wm)) / (2 * step) - dw[j]) < 1e-7


def test_backward_against_differences():
    check_backward(X.add_rms_norm_backward)


def test_planted_mistakes_are_caught():
    def floor_rule(x):                         # the exponent floor(log2 amax) - 2, which lets values saturate
        codes, byte = X.mx_blocks(x)
        return codes, np.where(byte > 0, byte - 1, byte)

    def half_up(x):                            # ties away from zero
        codes, byte = X.mx_blocks(x)
        v = np.abs(np.ldexp(x, -(byte.astype(np.int64) - 127)))
        mids = np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0])
        return (np.searchsorted(mids, v, side="right") + 8 * np.signbit(x)).astype(np.uint8), byte

    for bad in (floor_rule, half_up):
        with pytest.raises(AssertionError):
            check_mx_blocks(bad)
    for bad in (lambda a, sa, b, sb, c: X.mxfp4_gemm_nt(a, sa, b, sb),
                lambda a, sa, b, sb, c: X.mxfp4_gemm_nt(a, sa[::-1].copy(), b, sb, c)):
        with pytest.raises(AssertionError):
            check_gemm(bad)
    for bad in (lambda dy, dh, h, w, r: X.add_rms_norm_backward(dy, None, h, w, r),
                lambda dy, dh, h, w, r: (r[:, None] * dy * w + dh, X.add_rms_norm_backward(dy, dh, h, w, r)[1])):
        with pytest.raises(AssertionError):
            check_backward(bad)
