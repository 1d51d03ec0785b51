"""The MXFP4 linear layer's plans on the GPU: the epilogue's hand-over from unit to unit on every tile that has one (the
wait that counts the stores of d and z, the bias of the units in flight, the residual's reads between stores), whole tiles
beside slices in one workgroup, and the tiles with K groups.

Exact integers (sums and products of the epilogue below 2^24), so that d and z are the oracle's bf16 roundings bit for bit
and a unit that finished on another's bias, or on stages that had not landed, shows in some place."""

import functools

import numpy as np
import pytest
import torch

from oracle import mx as X
from oracle.formats import bf16_bits_to_f64, f64_to_bf16_bits
from tests.helpers import check_bit_exact
from tests.test_gpu_linear import run
from tests.test_gpu_mxfp4_plans import LINE, TILES

pytestmark = pytest.mark.gpu

# (bias, residual, z): the first wait has another count with z, and reads of the residual and copies of the bias come and go
SETS = [(True, True, True), (True, False, False), (False, True, False), (False, False, True)]


@functools.lru_cache(maxsize=4)
def integers(m, n, k):
    """Operands of 0, 1, 2, -1, -2 with scales of 1 and 2, and their product: some 5 sqrt(k) large at random, so that the
    product of two of its numbers is below 2^24 for k = 8192 as well."""
    rng = np.random.default_rng(m + n + k)
    ints = np.array([0, 2, 4, 10, 12], dtype=np.uint8)
    a, b = (X.pack_pairs(ints[rng.integers(0, 5, (r, k))]) for r in (m, n))
    sa, sb = (np.ascontiguousarray(X.pack_words((127 + rng.integers(0, 2, (r, k // 32))).astype(np.uint8)).T) for r in (m, n))
    return a, sa, b, sb, X.mxfp4_gemm_nt(a, sa, b, sb)


@pytest.fixture
def linear(dg, monkeypatch, capfd):
    """linear(kernel, cap, m, n, k, gated, set) -> (tiles, whole, slices, workgroups) of the plan, after the comparison."""
    monkeypatch.setenv("DG_LOG", "1")

    def go(kernel, cap, m, n, k, gated, bias, res, z):
        monkeypatch.setenv("DG_FORCE_MXFP4", str(kernel))
        dg.dg_set_num_cus(cap)
        try:
            # (the bias repeats after 257 columns: two tiles differ in most of theirs)
            a, sa, b, sb, u = integers(m, n, k)
            vb = f64_to_bf16_bits((np.arange(n) * 37 % 257 - 128).astype(np.float64)) if bias else None
            rr = np.random.default_rng(m).integers(-100, 101, (m, n // 2 if gated else n))
            vr = f64_to_bf16_bits(rr.astype(np.float64)) if res else None
            if bias:
                u = u + bf16_bits_to_f64(vb)
            capfd.readouterr()
            act = ("none", "relu")[(m + n // 16 + k // 128) % 2]
            got_d, got_z = run(dg, a, sa, b, sb, vb, act, gated, vr, z)
            line = LINE.search(capfd.readouterr().err)
            assert line, "no plan logged"
            bm, bn, kg, tiles, whole, slices, wgs, _ = map(int, line.groups())
            assert (bm, bn, kg) == TILES[kernel], "another kernel ran"
            what = f"{kernel} {cap} {m} {n} {k} {act}"
            if z:
                check_bit_exact(got_z, u, f"z {what}")
            # (no residual is a residual of 0 in include/dg.h: -0 + 0 is 0)
            want = X.linear_epilogue(u, act, gated, bf16_bits_to_f64(vr) if res else 0.0)
            assert np.abs(want).max() < 2 ** 24
            check_bit_exact(got_d, want, f"d {what}")
            return tiles, whole, slices, wgs
        finally:
            dg.dg_set_num_cus(0)
    return go


@pytest.mark.parametrize("k", [128, 256, 640, 2176])
@pytest.mark.parametrize("kernel", [0, 1, 2, 3])
def test_several_units_per_workgroup(linear, kernel, k):
    """Units of one stage (K blocks one and two: the copies' cursor runs ahead by as many units as the ring has slots), of
    a few and of more than the ring holds; partial last tiles in both directions."""
    bm, bn, _ = TILES[kernel]
    for cap, m, n in ((1, 2 * bm + 5, bn + 32), (2, 3 * bm - 7, 2 * bn - 64), (3, bm + 1, 4 * bn), (1, 3 * bm, 3 * bn + 32)):
        for gated in (False, True):
            for given in SETS:
                tiles, whole, _, wgs = linear(kernel, cap, m, n, k, gated, *given)
                assert whole == tiles > wgs == cap


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("kernel", [0, 1, 2, 3])
def test_whole_tiles_beside_split_ones(linear, kernel, which):
    """A workgroup's whole units and then slices, whose stores and bias are others; slices of even length and a shorter
    last one."""
    bm, bn, _ = TILES[kernel]
    k, m, n, want = ((8192, 2 * bm + 31, 2 * bn + 96, 1), (6272, 2 * bm + 1, 3 * bn + 32, 4), (7552, 3 * bm - 9, 3 * bn, 1))[which]
    for gated in (False, True):
        for given in SETS:
            tiles, whole, slices, wgs = linear(kernel, 8, m, n, k, gated, *given)
            assert 0 < whole == tiles - want and slices > 1 and wgs == 8


@pytest.mark.parametrize("kernel", [4, 5, 6, 7])
def test_tiles_with_k_groups(linear, kernel):
    bm, bn, _ = TILES[kernel]
    for i, (m, n) in enumerate(((1, 32), (bm + 3, bn + 32), (3 * bm, 2 * bn), (4 * bm - 1, 5 * bn - 32))):
        for gated in (False, True):
            for given in SETS:
                tiles, whole, _, wgs = linear(kernel, 0, m, n, (128, 384, 1152, 2176)[i], gated, *given)
                assert whole == tiles == wgs


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kernel", [0, 1])
def test_many_units_repeat_bit_for_bit(dg, kernel, gated, monkeypatch):
    """Some thirty units a workgroup on the whole chip, with a nonlinear activation, residual and z: every run the same."""
    monkeypatch.setenv("DG_FORCE_MXFP4", str(kernel))
    m, n, k = 4096, 16384, 256
    g = torch.Generator(device="cuda").manual_seed(kernel)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")                 # noqa: E731
    ops = dg.quantize_mxfp4(randn(m, k))[:2] + dg.quantize_mxfp4(randn(n, k) * k ** -0.5)[:2]
    bias, res = randn(n).bfloat16(), randn(m, n // 2 if gated else n).bfloat16()
    act = dg.ACT_SILU | (dg.ACT_GATED if gated else 0)
    dg.dg_set_num_cus(32)
    try:
        want = dg.mxfp4_linear(*ops, bias, act, res, pre_activation=True)
        for _ in range(5):
            for w, t in zip(want, dg.mxfp4_linear(*ops, bias, act, res, pre_activation=True)):
                assert torch.equal(w.view(torch.int16), t.view(torch.int16))
    finally:
        dg.dg_set_num_cus(0)
