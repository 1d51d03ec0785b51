"""The sums over rows of the operators around a block (weight, gate and bias gradients) on integers, whose every partial sum
is exact in fp32: the results are equal to the last bit, so that a partial row or tile left out, added twice or taken from
a neighbour shows at any size."""

import pytest
import torch

pytestmark = pytest.mark.gpu

LARGE = 264 * 1024   # rows: 2.2 * 10^9 elements of 8192 columns


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def ints(seed, lo, hi, *shape):
    """bf16 integers lo .. hi, made by blocks of rows."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
    for part in out.split(8192) if out.dim() > 1 else (out,):
        part.copy_(torch.randint(lo, hi + 1, part.shape, generator=g, device="cuda"))
    return out


def check(got, want, what):
    bad = got.double() != want
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} wrong, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("m,k,gate_rows", [
    (1, 128, 1), (255, 128, 7), (1025, 384, 256), (1500, 512, 1), (4100, 256, 1000), (5000, 128, 77), (3001, 2176, 3000),
    (2049, 7168, 100), (600, 9216, 33), (515, 16384, 600), (LARGE, 8192, 256)])
def test_sandwich_sums(dg, m, k, gate_rows):
    """rstd and rstd_x of 1, and pairs of columns with the same h and opposite dy * weight, so that a row's mean(a n) is 0 and
    D = dh + dy * weight: dweight = sum dy h, dpost_weight = sum scale gate D x, dgate = sum scale post_weight D x."""
    x, h, dy, dh = (ints(s, -1, 1, m, k) for s in range(1, 5))
    h[:, 1::2] = h[:, ::2]
    dy[:, 1::2] = -dy[:, ::2]
    pw, w, gate = ints(5, 1, 2, k), ints(6, 1, 2, k), ints(7, -1, 2, -(-m // gate_rows), k)
    w[1::2] = w[::2]
    one, scale = torch.ones(m, device="cuda"), 0.5
    dx, dres, dweight, dpost, dgate = dg.sandwich_norm_backward(dy, dh, x, h, pw, gate, w, one, one, scale, gate_rows)
    want_w, want_p = (torch.zeros(k, dtype=torch.float64, device="cuda") for _ in range(2))
    want_g = torch.zeros(len(gate), k, dtype=torch.float64, device="cuda")
    for r in range(0, m, 4096):
        rows = slice(r, min(m, r + 4096))
        d = dh[rows].double() + dy[rows].double() * w.double()
        check(dres[rows], d, f"dresidual from row {r}")
        g = torch.arange(rows.start, rows.stop, device="cuda") // gate_rows
        want_w += (dy[rows].double() * h[rows].double()).sum(dim=0)
        d *= x[rows].double() * scale
        want_p += (d * gate[g].double()).sum(dim=0)
        want_g.index_add_(0, g, d * pw.double())
    for got, want, what in ((dweight, want_w, "dweight"), (dpost, want_p, "dpost_weight"), (dgate, want_g, "dgate")):
        check(got, want, what)


@pytest.mark.parametrize("act", ["none", "relu", "none gated", "relu gated"])
@pytest.mark.parametrize("m,n", [(1, 256), (33, 512), (129, 1024), (500, 2048), (2049, 4096), (4224, 4096), (4097, 33024), (70000, 256),
                                 (LARGE, 8192)])
def test_bias_gradients(dg, m, n, act):
    gated = act.endswith("gated")
    code = {"none": dg.ACT_NONE, "relu": dg.ACT_RELU}[act.split()[0]] | (dg.ACT_GATED if gated else 0)
    dy, z = ints(1, -1, 1, m, n // 2 if gated else n), ints(2, -2, 2, m, n)
    dbias = dg.activation_backward(dy, z, code)[4]
    want = torch.zeros(n, dtype=torch.float64, device="cuda")
    for r in range(0, m, 4096):
        y, v = dy[r:r + 4096].double(), z[r:r + 4096].double()
        g = v[:, :n // 2] if gated else v
        on = (g > 0).double() if act.startswith("relu") else torch.ones_like(g)
        dz = torch.hstack([y * v[:, n // 2:] * on, y * g * on]) if gated else y * on
        want += dz.sum(dim=0)
    check(dbias, want, "dbias")
