"""The norms' codes around a block with fp32 scales, by exact arithmetic: the code of a value is the e4m3 nearest to
448 |h w| / max |h w| of its block (1 / rms cancels), ties to the even one.  h w has 16 bits, a point midway between two
codes five: 448 |h w| and midpoint * max |h w| are exact in float64, so a tie shows as equality.  (Some values in 2600 are
ties; a quotient in fp32 or fp64 decides those by its roundings.)"""

import numpy as np
import pytest

from oracle import mx as X
from oracle.formats import bf16_bits_to_f64
from tests.test_gpu_norm import F32
from tests.test_gpu_sandwich import inputs, run

pytestmark = pytest.mark.gpu


def exact_codes(h, w):
    """e4m3 magnitudes' places in the grid [m, k], and how many are ties."""
    m, k = h.shape
    a = np.abs(h * w).reshape(m, k // 128, 128)
    top = a.max(axis=2, keepdims=True)
    a = 448 * a
    code, ties = np.zeros(a.shape, dtype=int), 0
    for i, mid in enumerate((X.E4M3_GRID[:-1] + X.E4M3_GRID[1:]) / 2):
        tie = (a == mid * top) & (top > 0)
        code += (a > mid * top) | (tie & (i % 2 == 1))      # (up to place i + 1, which is even)
        ties += int(tie.sum())
    return code.reshape(m, k), ties


@pytest.mark.parametrize("m,k,gate_rows", [(3, 7168, 3), (300, 1280, 70), (2048, 4224, 500), (90, 12288, 1), (7, 32768, 7)])
def test_codes_are_the_nearest_and_ties_even(dg, m, k, gate_rows):
    a = inputs(m + k, m, k, gate_rows)
    (q, _, h, _), _ = run(dg, *a, F32, gate_rows, 0.7)
    hw = bf16_bits_to_f64(h), bf16_bits_to_f64(a[4])
    want, ties = exact_codes(*hw)
    assert ties > 0
    bad = (q & 0x7f) != want
    assert not bad.any(), f"{bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}"
    assert np.array_equal(q >> 7, np.signbit(hw[0] * hw[1]))
