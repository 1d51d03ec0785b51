"""The MXFP4 GEMM's plans on the GPU: several units per workgroup, whole tiles beside split ones, split calls in flight
together, and that a pinned kernel is the one that runs (read from the DG_LOG line).  Exact integers: D has to equal the
oracle's bf16 rounding bit for bit (every sum is a multiple of 1 below 2^24, whatever the order)."""

import re

import numpy as np
import pytest
import torch

from oracle import mx as X
from oracle.formats import f64_to_bf16_bits
from tests.helpers import check_bit_exact
from tests.test_gpu_mxfp4 import rand_mx, run_gemm

pytestmark = pytest.mark.gpu

# id -> rows, columns, K groups
TILES = {0: (256, 256, 1), 1: (128, 256, 1), 2: (128, 128, 1), 3: (64, 128, 1), 4: (64, 128, 2), 5: (96, 128, 2),
         6: (64, 64, 2), 7: (128, 128, 2)}
LINE = re.compile(r"tile (\d+)x(\d+), (\d+) K groups?, (\d+) tiles \((\d+) whole, the rest x (\d+) K slices\), (\d+) workgroups, "
                  r"workspace (\d+)")


def integers(seed, m, n, k, with_c):
    """Integer codes, scales of 1 and 2, C an integer."""
    rng = np.random.default_rng(seed)
    ints = np.array([0, 2, 4, 6, 10, 12], dtype=np.uint8)                # 0, 1, 2, 4, -1, -2
    a, b = (X.pack_pairs(ints[rng.integers(0, 6, (r, k))]) for r in (m, n))
    sa, sb = (np.ascontiguousarray(X.pack_words((127 + rng.integers(0, 2, (r, k // 32))).astype(np.uint8)).T) for r in (m, n))
    return a, sa, b, sb, f64_to_bf16_bits(rng.integers(-100, 101, (m, n)).astype(np.float64)) if with_c else None


@pytest.fixture
def run(dg, monkeypatch, capfd):
    """run(kernel, cap, m, n, k, with_c) -> (tiles, whole, slices, workgroups) of the plan, after the comparison."""
    monkeypatch.setenv("DG_LOG", "1")

    def go(kernel, cap, m, n, k, with_c):
        monkeypatch.setenv("DG_FORCE_MXFP4", str(kernel))
        dg.dg_set_num_cus(cap)
        try:
            args = integers(m + n + k, m, n, k, with_c)
            capfd.readouterr()
            got = run_gemm(dg, *args)
            line = LINE.search(capfd.readouterr().err)
            assert line, "no plan logged"
            bm, bn, kg, tiles, whole, slices, wgs, _ = map(int, line.groups())
            assert (bm, bn, kg) == TILES[kernel], "another kernel ran"
            check_bit_exact(got, X.mxfp4_gemm_nt(*args), f"{kernel} {cap} {m} {n} {k}")
            return tiles, whole, slices, wgs
        finally:
            dg.dg_set_num_cus(0)
    return go


@pytest.mark.parametrize("with_c", [False, True])
@pytest.mark.parametrize("k", [128, 640, 1024, 2176])
@pytest.mark.parametrize("kernel", [0, 1, 2, 3])
def test_several_units_per_workgroup(run, kernel, k, with_c):
    """The hand-over from unit to unit: the copies that run on into the next tile, the last stage's late ones, the wait
    that passes over the stores; K blocks even, odd and one."""
    bm, bn, _ = TILES[kernel]
    for cap, m, n in ((1, 2 * bm + 5, bn + 16), (2, 3 * bm - 7, 2 * bn - 48), (3, bm + 1, 4 * bn), (3, 3 * bm, 3 * bn + 16)):
        tiles, whole, _, wgs = run(kernel, cap, m, n, k, with_c)
        assert whole == tiles > wgs == cap


@pytest.mark.parametrize("with_c", [False, True])
@pytest.mark.parametrize("kernel", [0, 1, 2, 3])
def test_whole_tiles_beside_split_ones(run, kernel, with_c):
    """Plans with 0 < whole tiles < tiles, slices of even length and a shorter last one."""
    bm, bn, _ = TILES[kernel]
    for k, m, n, want in ((8192, 2 * bm + 31, 2 * bn + 80, 1), (6272, 2 * bm + 1, 3 * bn + 16, 4), (7552, 3 * bm - 9, 3 * bn, 1)):
        tiles, whole, slices, wgs = run(kernel, 8, m, n, k, with_c)
        assert 0 < whole == tiles - want and slices > 1 and wgs == 8


@pytest.mark.parametrize("kernel", [4, 5, 6, 7])
@pytest.mark.parametrize("k", [128, 256, 384, 1152, 2176])
def test_tiles_with_k_groups(run, kernel, k):
    bm, bn, _ = TILES[kernel]
    for i, (m, n) in enumerate(((1, 16), (bm + 3, bn + 48), (3 * bm, 2 * bn), (4 * bm - 1, 5 * bn - 16))):
        tiles, whole, _, wgs = run(kernel, 0, m, n, k, bool(i & 1))
        assert whole == tiles == wgs


def test_split_calls_on_two_streams(dg, monkeypatch):
    """Split plans in flight together, each with a workspace of its own, given and not."""
    monkeypatch.setenv("DG_FORCE_MXFP4", "2")
    rng = np.random.default_rng(12)
    shapes = [(256, 1040, 4096), (500, 528, 6144)]
    ts = [[torch.from_numpy(v).cuda() for v in rand_mx(rng, m, k) + rand_mx(rng, n, k)] for m, n, k in shapes]
    need = [dg.dg_mxfp4_gemm_workspace_bytes(*s) for s in shapes]
    assert min(need) > 0
    want = [dg.mxfp4_gemm_nt(*t) for t in ts]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    ws = [torch.empty(b, dtype=torch.uint8, device="cuda") for b in need]
    torch.cuda.synchronize()
    for turn in range(6):
        for i, (t, s) in enumerate(zip(ts, streams)):
            with torch.cuda.stream(s):
                if turn % 2:
                    got.append((i, dg.mxfp4_gemm_nt(*t)))
                else:
                    got.append((i, dg.dg_mxfp4_gemm_nt(*t, None, torch.empty_like(want[i]), ws[i])))
    torch.cuda.synchronize()
    for i, g in got:
        assert torch.equal(g, want[i])


@pytest.mark.parametrize("kernel,m,n,k", [(100, 9, 48, 640), (101, 30, 48, 640), (0, 300, 272, 384), (1, 140, 272, 640), (2, 512, 528, 8192),
                                          (3, 70, 144, 384), (4, 70, 144, 640), (5, 100, 144, 640), (6, 70, 144, 384), (7, 130, 144, 640)])
@pytest.mark.parametrize("e", [-138, -143, -148])
def test_subnormal_sums_are_kept(dg, monkeypatch, kernel, m, n, k, e):
    """Integers times 2^e: products, sums and C below 2^-126 are exact down to fp32's last bit, 2^-149, and D is their
    rounding to bf16, whose own last bit is 2^-133 (also through split K's partial sums: kernel 2)."""
    monkeypatch.setenv("DG_FORCE_MXFP4", str(kernel))
    assert kernel != 2 or dg.dg_mxfp4_gemm_workspace_bytes(m, n, k) > 0
    a, sa, b, sb, _ = integers(k + m, m, n, k, False)
    one = lambda t, by: (t.view(np.uint8) + np.uint8(by % 256)).view(np.int32)     # noqa: E731  (both bytes stay in range)
    sa, sb = one(sa, -60), one(sb, e + 60)
    rng = np.random.default_rng(m)
    c = rng.integers(0, 256, (m, n)).astype(np.uint16) | (rng.integers(0, 2, (m, n)).astype(np.uint16) << 15)
    want = X.mxfp4_gemm_nt(a, sa, b, sb, c)
    small = (np.abs(want) < 2.0 ** -126) & (want != 0)
    assert small.mean() > 0.2
    check_bit_exact(run_gemm(dg, a, sa, b, sb, c), want, f"{kernel} {e}")
