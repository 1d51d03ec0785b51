"""The plans of the products by expert, read from the DG_LOG line: the pinned kernel is the one that runs, with several of its
tiles per workgroup.  Exact integers, as in tests/test_gpu_ragged.py."""

import re

import numpy as np
import pytest

from tests.test_gpu_mxfp4_plans import TILES
from tests.test_gpu_ragged import check_k, check_m, integers

pytestmark = pytest.mark.gpu

ALL = {**TILES, 8: (192, 256, 1)}   # id -> rows, columns, K groups
LINE = re.compile(r"\[dg\] (\w+) m=(\d+) n=(\d+) k=(\d+) groups=(\d+) -> tile (\d+)x(\d+), (\d+) K groups?, at most (\d+) tiles, "
                  r"(\d+) workgroups\n")
SIZES = [5, 300, 0, 129, 1]


@pytest.fixture
def plan(dg, monkeypatch, capfd):
    """plan(kernel, cap, call) -> (entry, m, n, k, groups, tiles at most, workgroups), logged by the one call."""
    monkeypatch.setenv("DG_LOG", "1")

    def go(kernel, cap, call):
        monkeypatch.setenv("DG_FORCE_MXFP4", str(kernel))
        dg.dg_set_num_cus(cap)
        try:
            capfd.readouterr()
            call()
            (line,) = LINE.findall(capfd.readouterr().err)
            assert tuple(map(int, line[5:8])) == ALL[kernel], "another kernel ran"
            return line[0], *map(int, line[1:5] + line[8:])
        finally:
            dg.dg_set_num_cus(0)
    return go


@pytest.mark.parametrize("kernel", list(ALL))
def test_m_grouped_plan(dg, plan, kernel):
    bm, bn, kg = ALL[kernel]
    rng = np.random.default_rng(kernel)
    m, n, k, cap = sum(SIZES) + 7, 2 * bn + 16, 640, 0 if kg > 1 else 3
    a, sa = integers(rng, m, k)
    b, sb = (np.stack(t) for t in zip(*(integers(rng, n, k) for _ in SIZES)))
    got = plan(kernel, cap, lambda: check_m(dg, a, sa, b, sb, SIZES, exact=True))
    tiles = sum(-(-r // bm) for r in SIZES) * 3
    assert got[:5] == ("m_grouped_mxfp4_gemm_nt_ragged", m, n, k, len(SIZES))
    assert got[5] >= tiles and (got[6] == got[5] if kg > 1 else tiles > got[6] == cap)


@pytest.mark.parametrize("kernel", list(ALL))
def test_k_grouped_plan(dg, plan, kernel):
    bm, bn, kg = ALL[kernel]
    rng = np.random.default_rng(kernel)
    m, n, cap = bm + 8, 2 * bn + 16, 0 if kg > 1 else 3
    k = 128 * dg.dg_mxfp4_ragged_blocks(sum(SIZES), len(SIZES))
    got = plan(kernel, cap, lambda: check_k(dg, *integers(rng, m, k), *integers(rng, n, k), SIZES, exact=True))
    assert got[:6] == ("k_grouped_mxfp4_gemm_nt_ragged", m, n, k, len(SIZES), 6 * len(SIZES))
    assert got[6] == (got[5] if kg > 1 else cap)
