"""Tensors of more than 2^31 elements (2^32 bytes) through the operators around a block's products: the same PERIOD rows
again and again, so that every repetition has the first one's results bit for bit, and those are the ones of a small call."""

import pytest
import torch

from tests.test_gpu_norm import F32, MX, UE8M0

pytestmark = pytest.mark.gpu

PERIOD, TIMES, K = 1024, 264, 8192   # 2.2 * 10^9 elements
M = PERIOD * TIMES


def randn(*shape, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def again(t):
    return t.repeat(TIMES, *[1] * (t.dim() - 1))


def same(big, small, dim, what):
    """big is small TIMES over along dim."""
    n = small.shape[dim]
    assert big.shape[dim] == n * TIMES
    for i in (*range(0, TIMES, 50), TIMES - 1):
        assert torch.equal(big.narrow(dim, i * n, n), small), f"{what}: repetition {i}"


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("fmt", [F32, UE8M0, MX])
def test_sandwich_norm(dg, fmt):
    x, res = randn(PERIOD, K, seed=1), randn(PERIOD, K, seed=2)
    pw, w, gate = randn(K, seed=3), randn(K, seed=4), randn(PERIOD // 256, K, seed=5)
    small = dg.sandwich_norm(x, res, pw, gate, w, 0.7, 256, quant_format=fmt)
    big = dg.sandwich_norm(again(x), again(res), pw, again(gate), w, 0.7, 256, quant_format=fmt)
    for i, what in enumerate(("q", "sf", "h", "rstd_x", "rstd")):
        same(big[i], small[i], 1 if what == "sf" and fmt != UE8M0 else 0, what)


def test_sandwich_norm_backward(dg):
    x, h, dy, dh = (randn(PERIOD, K, seed=s) for s in (1, 2, 3, 4))
    pw, w, gate = randn(K, seed=5), randn(K, seed=6), randn(PERIOD // 256, K, seed=7)
    rx, r = (1 / t.float().square().mean(1).sqrt() for t in (x, h))
    small = dg.sandwich_norm_backward(dy, dh, x, h, pw, gate, w, rx, r, 0.7, 256)
    big = dg.sandwich_norm_backward(again(dy), again(dh), again(x), again(h), pw, again(gate), w, again(rx), again(r), 0.7, 256)
    for i, what in ((0, "dx"), (1, "dresidual")):
        same(big[i], small[i], 0, what)
    # Sums of n terms in another order: n additions, each rounded by 2^-24 of a partial sum at most.  A workgroup's partial
    # sums are those of some 1000 terms of any sign and sizes around 3, and the last 300 additions are of such sums: on
    # average below 100 sqrt(n).
    u = 2.0 ** -24
    for i, what, times in ((2, "dweight", TIMES), (3, "dpost_weight", TIMES)):
        assert (big[i] - small[i] * times).abs().max().item() < 100 * M * M ** 0.5 * u, what
    for i in (0, TIMES // 2, TIMES - 1):
        off = (big[4][i * 4:i * 4 + 4] - small[4]).abs().max().item()
        assert off < 100 * 256 * 256 ** 0.5 * u, f"dgate: repetition {i}"


@pytest.mark.parametrize("act", [3, 18])
def test_activation_backward(dg, act):
    gated = act & 16
    dy, z = randn(PERIOD, K // 2 if gated else K, seed=1), randn(PERIOD, K, seed=2)
    small = dg.activation_backward(dy, z, act, bias=False)
    big = dg.activation_backward(again(dy), again(z), act)
    for i, what, dim in ((0, "q", 0), (1, "sf", 1), (2, "qt", 1), (3, "sft", 0)):
        same(big[i], small[i], dim, what)
    want = dg.activation_backward(dy, z, act)[4] * TIMES
    # (as the norms' sums)
    assert (big[4] - want).abs().max().item() < 100 * M * M ** 0.5 * 2.0 ** -24


def test_quantize_ragged(dg):
    """The small call's groups TIMES over: 1000 rows, none, and the 24 that fill the last block of 128."""
    x = randn(PERIOD, K, seed=1)
    ms = torch.tensor([1000, 0, 24], dtype=torch.int32, device="cuda")
    small = dg.quantize_mxfp4_ragged(x, ms)
    q, sf, qt, sft = dg.quantize_mxfp4_ragged(again(x), again(ms))
    same(q, small[0], 0, "q")
    same(sf, small[1], 1, "sf")
    blocks = 9   # of 128 rows that a period's groups fill: 8 and 1
    for i in (0, 100, TIMES - 1):
        assert torch.equal(qt[:, i * blocks * 64:(i + 1) * blocks * 64], small[2][:, :blocks * 64]), i
        assert torch.equal(sft[i * blocks:(i + 1) * blocks], small[3][:blocks]), i


def test_m_grouped_ragged(dg):
    """Weights of 4.7 GB: 320 experts alike, 5 rows each (the same rows)."""
    G, n, k = 320, 4096, 7168
    aq, asf = dg.quantize_mxfp4(randn(5, k, seed=1))
    bq, bsf = dg.quantize_mxfp4(randn(n, k, seed=2))
    ms = torch.full((G,), 5, dtype=torch.int32, device="cuda")
    want = dg.m_grouped_mxfp4_gemm_nt_ragged(aq, asf, bq[None], bsf[None], ms[:1])
    d = dg.m_grouped_mxfp4_gemm_nt_ragged(aq.repeat(G, 1), asf.repeat(1, G), bq.repeat(G, 1, 1), bsf.repeat(G, 1, 1), ms)
    assert torch.equal(d.view(G, 5, n), want.expand(G, 5, n))


def test_k_grouped_ragged(dg):
    """Gradients of 5.2 GB: 320 experts, every third without rows, the others with the same 130."""
    G, m, n = 320, 4096, 2048
    dy, x = randn(130, m, seed=1), randn(130, n, seed=2)
    one = torch.full((1,), 130, dtype=torch.int32, device="cuda")
    ms = torch.full((G,), 130, dtype=torch.int32, device="cuda")
    ms[::3] = 0
    full = int((ms > 0).sum())

    def operands(t, ms, times):
        return dg.quantize_mxfp4_ragged(t.repeat(times, 1), ms)[2:]

    want = dg.k_grouped_mxfp4_gemm_nt_ragged(*operands(dy, one, 1), *operands(x, one, 1), one)[0]
    d = torch.full((G, m, n), float("nan"), dtype=torch.bfloat16, device="cuda")
    dg.k_grouped_mxfp4_gemm_nt_ragged(*operands(dy, ms, full), *operands(x, ms, full), ms, out=d)
    for g in range(G):
        assert torch.equal(d[g], want if g % 3 else torch.zeros_like(want)), g
