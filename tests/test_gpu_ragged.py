"""MXFP4 products grouped by expert with ragged sizes, and their quantiser, against the float64 oracle.

The quantiser's outputs equal the oracle's bit for bit.  The products' tolerance is that of tests/test_gpu_mxfp4.py:
|D - ref| <= 2^-8 |ref| + (K/8 + 1) 2^-23 (1 + 2^-8) S, K of the product (along K: a group's padded rows) and S the sum
of |a b|.  With integers whose sums are exact D is the oracle's bf16 rounding bit for bit.
"""

import numpy as np
import pytest
import torch

from oracle import mx as X
from oracle.formats import bf16_bits_to_f64, f64_to_bf16_bits
from tests.helpers import bits
from tests.test_gpu_mxfp4 import guarded, rand_mx, to_dev, values
from tests.test_gpu_norm import bf, dev

pytestmark = pytest.mark.gpu

# sizes of the groups: none, one row, whole tiles, a row past them, one large group among small ones
SIZES = [[1], [0, 1, 0], [5, 0, 3, 1], [128, 128], [129, 1, 127, 0, 255], [0, 0, 0], [300, 2, 70, 0, 0, 64, 31, 16],
         [1] * 70, [700, 0, 3], [3, 0, 0, 0, 600, 17]]
INTS = np.array([0, 2, 4, 6, 10, 12], dtype=np.uint8)                     # 0, 1, 2, 4, -1, -2


def device_ms(ms):
    return torch.tensor(ms, dtype=torch.int32, device="cuda")


def integers(rng, r, k):
    return X.pack_pairs(INTS[rng.integers(0, 6, (r, k))]), np.ascontiguousarray(
        X.pack_words((127 + rng.integers(0, 2, (r, k // 32))).astype(np.uint8)).T)


def run_m(dgm, a, sa, b, sb, ms, n):
    t = [torch.from_numpy(v).cuda() for v in (a, sa, b, sb)]
    d, check = guarded((a.shape[0], n), torch.bfloat16)
    d.view(torch.int16).fill_(-1)
    dgm.dg_m_grouped_mxfp4_gemm_nt_ragged(*t, device_ms(ms), d)
    torch.cuda.synchronize()
    check()
    return bits(d)


def check_m(dgm, a, sa, b, sb, ms, exact=False):
    got = run_m(dgm, a, sa, b, sb, ms, b.shape[1])
    end = 0
    for g, (rows, ref, s) in enumerate(X.m_grouped_mxfp4_gemm_nt_ragged(a, sa, b, sb, ms)):
        end = max(end, rows.stop)
        if exact:
            bad = got[rows] != f64_to_bf16_bits(ref)
        else:
            bad = ~(np.abs(bf16_bits_to_f64(got[rows]) - ref) <= 2.0 ** -8 * np.abs(ref)
                    + (a.shape[1] / 4 + 1) * 2.0 ** -23 * (1 + 2.0 ** -8) * s)
        assert not bad.any(), f"group {g}: {bad.sum()} of {bad.size} wrong, first at {np.argwhere(bad)[0]}"
    assert (got[end:] == 0xFFFF).all(), "rows behind the last group were written"


@pytest.mark.parametrize("tail", [0, 9])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_m_grouped_sizes(dg, sizes, tail):
    m, G = max(sum(sizes) + tail, 1), len(sizes)
    n, k = ((16, 384), (272, 640), (528, 256))[(G + tail) % 3]
    rng = np.random.default_rng(m)
    a, sa = rand_mx(rng, m, k)
    b, sb = (np.stack(t) for t in zip(*(rand_mx(rng, n, k) for _ in range(G))))
    check_m(dg, a, sa, b, sb, sizes)


@pytest.mark.parametrize("kernel", [0, 1, 2, 3, 4, 5, 6, 7, 8])
def test_m_grouped_every_kernel(dg, kernel, monkeypatch):
    """Each tile pinned, on all CUs and on eight (several tiles of several groups per workgroup, odd and even counts of K
    blocks, fewer than the ring's slots too); exact integers."""
    monkeypatch.setenv("DG_FORCE_MXFP4", str(kernel))
    for sizes in ([300, 0, 70, 1], [5, 129, 0, 0, 33, 256, 2, 64, 17]):
        for n, k, cap in ((272, 128, 0), (528, 1152, 8), (400, 2176, 8), (784, 256, 4)):
            dg.dg_set_num_cus(cap)
            try:
                rng = np.random.default_rng(n + k)
                a, sa = integers(rng, sum(sizes) + 3, k)
                b, sb = (np.stack(t) for t in zip(*(integers(rng, n, k) for _ in sizes)))
                check_m(dg, a, sa, b, sb, sizes, exact=True)
            finally:
                dg.dg_set_num_cus(0)


@pytest.mark.parametrize("ms", [[-5, 7, -1, 4], [10, 100], [2 ** 31 - 1, 2 ** 31 - 1, 3], [-2 ** 31, 20]], ids=str)
def test_malformed_sizes_are_cut(dg, ms):
    """Negative counts are 0 and rows are cut at m, in all three calls."""
    m, n, k, G = 20, 144, 256, len(ms)
    rng = np.random.default_rng(1)
    a, sa = integers(rng, m, k)
    b, sb = (np.stack(t) for t in zip(*(integers(rng, n, k) for _ in ms)))
    check_m(dg, a, sa, b, sb, ms, exact=True)
    x, x64 = to_dev(values(2, m, k), torch.bfloat16)
    check_quantize(dg, x, x64, ms)
    kb = dg.dg_mxfp4_ragged_blocks(m, G)
    check_k(dg, *integers(rng, 48, kb * 128), *integers(rng, 80, kb * 128), ms, exact=True)


def check_quantize(dgm, x, x64, ms, rows=True):
    m, k = x.shape
    blocks = dgm.dg_mxfp4_ragged_blocks(m, len(ms))
    outs = dict(qt=((k, blocks * 64), torch.uint8), sft=((blocks, k), torch.int32))
    if rows:
        outs |= dict(q=((m, k // 2), torch.uint8), sf=((k // 128, m), torch.int32))
    made = {n: guarded(*o) for n, o in outs.items()}
    for t, _ in made.values():
        t.view(torch.uint8).fill_(0x5A)
    dgm.dg_quantize_mxfp4_ragged(x, device_ms(ms), **{n: t for n, (t, _) in made.items()})
    torch.cuda.synchronize()
    got = {}
    for n, (t, check) in made.items():
        check()
        got[n] = t.cpu().numpy()
    qt, sft, used = X.quantize_mxfp4_ragged(x64, ms, blocks)
    q, sf, _ = X.quantize_mxfp4(x64)
    end = X.group_rows(ms, m)[-1][1]
    assert np.array_equal(got["qt"][:, :used * 64], qt[:, :used * 64]), "qt"
    assert np.array_equal(got["sft"][:used], sft[:used]), "sft"
    assert (got["qt"][:, used * 64:] == 0x5A).all() and (got["sft"][used:].view(np.uint8) == 0x5A).all(), "blocks behind the last"
    if rows:
        assert np.array_equal(got["q"][:end], q[:end]) and np.array_equal(got["sf"][:, :end], sf[:, :end])
        assert (got["q"][end:] == 0x5A).all() and (np.ascontiguousarray(got["sf"][:, end:]).view(np.uint8) == 0x5A).all(), "rows behind the last"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_quantize_ragged(dg, sizes, dtype):
    m = max(sum(sizes) + len(sizes) % 2 * 5, 1)
    x, x64 = to_dev(values(m, m, 128 + 256 * (m % 2)), dtype)
    check_quantize(dg, x, x64, sizes, rows=m % 3 != 0)


def test_quantize_ragged_of_one_group_is_the_plain_one(dg):
    x, _ = to_dev(values(1, 300, 640), torch.bfloat16)
    x[7, 3], x[200, 100] = float("nan"), float("inf")
    for a, b in zip(dg.quantize_mxfp4_ragged(x, device_ms([300])), dg.quantize_mxfp4(x, transposed=True)):
        assert torch.equal(a, b)


def check_k(dgm, a, sa, b, sb, ms, exact=False):
    m, n = a.shape[0], b.shape[0]
    t = [torch.from_numpy(v).cuda() for v in (a, sa, b, sb)]
    d, check = guarded((len(ms), m, n), torch.bfloat16)
    dgm.dg_k_grouped_mxfp4_gemm_nt_ragged(*t, device_ms(ms), d)
    torch.cuda.synchronize()
    check()
    got = bits(d)
    ref, s = X.k_grouped_mxfp4_gemm_nt_ragged(a, sa, b, sb, ms)
    if exact:
        bad = got != f64_to_bf16_bits(ref)
    else:
        rows = np.maximum(np.asarray(ms, dtype=np.float64), 0)[:, None, None] + 127
        bad = ~(np.abs(bf16_bits_to_f64(got) - ref) <= 2.0 ** -8 * np.abs(ref) + (rows / 8 + 1) * 2.0 ** -23 * (1 + 2.0 ** -8) * s)
    assert not bad.any(), f"{bad.sum()} of {bad.size} wrong, first at {np.argwhere(bad)[0]}"


@pytest.mark.parametrize("sizes", SIZES, ids=str)
def test_k_grouped_sizes(dg, sizes):
    kb = dg.dg_mxfp4_ragged_blocks(max(sum(sizes), 1), len(sizes))
    m, n = ((48, 272), (272, 128), (640, 528))[len(sizes) % 3]
    rng = np.random.default_rng(kb)
    check_k(dg, *rand_mx(rng, m, kb * 128), *rand_mx(rng, n, kb * 128), sizes)


@pytest.mark.parametrize("kernel", [0, 1, 2, 3, 4, 5, 6, 7, 8])
def test_k_grouped_every_kernel(dg, kernel, monkeypatch):
    monkeypatch.setenv("DG_FORCE_MXFP4", str(kernel))
    for sizes in ([300, 0, 70, 1], [5, 129, 0, 0, 1300, 256, 2]):
        for m, n, cap in ((272, 528, 0), (528, 400, 8), (70, 144, 4)):
            dg.dg_set_num_cus(cap)
            try:
                rng = np.random.default_rng(n + m)
                kb = dg.dg_mxfp4_ragged_blocks(sum(sizes), len(sizes))
                check_k(dg, *integers(rng, m, kb * 128), *integers(rng, n, kb * 128), sizes, exact=True)
            finally:
                dg.dg_set_num_cus(0)


def test_many_groups(dg):
    """The most groups that a call takes, most of them empty."""
    rng = np.random.default_rng(4)
    ms = np.where(rng.random(1024) < 0.2, rng.integers(0, 5, 1024), 0).tolist()
    m, n, k = sum(ms) + 4, 32, 128
    a, sa = integers(rng, m, k)
    b, sb = (np.stack(t) for t in zip(*(integers(rng, n, k) for _ in ms)))
    check_m(dg, a, sa, b, sb, ms, exact=True)
    kb = dg.dg_mxfp4_ragged_blocks(m, 1024)
    check_k(dg, *integers(rng, 16, kb * 128), *integers(rng, 32, kb * 128), ms, exact=True)
    for dtype in (torch.bfloat16, torch.float32):
        x, x64 = to_dev(values(2, m, 128), dtype)
        check_quantize(dg, x, x64, ms)


def test_nan_scales_stay_in_their_rows(dg):
    """A row with a NaN scale gives NaN in its row of D alone, beside rows of other groups in the same tile."""
    rng = np.random.default_rng(2)
    ms, n, k = [30, 40, 20], 96, 256
    a, sa = integers(rng, 90, k)
    b, sb = (np.stack(t) for t in zip(*(integers(rng, n, k) for _ in ms)))
    sa.view(np.uint8).reshape(2, 90, 4)[1, 30, 2] = 255
    a[30, 96:112] = 0
    got = bf16_bits_to_f64(run_m(dg, a, sa, b, sb, ms, n))
    nan = np.zeros((90, n), dtype=bool)
    nan[30] = True
    assert np.array_equal(np.isnan(got), nan)


def test_training_step_of_experts(dg):
    """Quantisers and products together, as an expert layer's step runs them: y, dx and dw against the oracle's products
    of the same operands, and near the unquantised gradients."""
    ms, n, k = [130, 0, 37, 200], 256, 384
    m, G = sum(ms), len(ms)
    x, w, dy = bf(1, m, k), bf(2, G, n, k, scale=k ** -0.5), bf(3, m, n, scale=1e-2)
    tx, tw, tdy, tms = dev(x), dev(w), dev(dy), device_ms(ms)
    wq, wsf, wqt, wsft = dg.quantize_mxfp4(tw, transposed=True)
    xq, xsf, xqt, xsft = dg.quantize_mxfp4_ragged(tx, tms)
    dyq, dysf, dyqt, dysft = dg.quantize_mxfp4_ragged(tdy, tms)
    y = dg.m_grouped_mxfp4_gemm_nt_ragged(xq, xsf, wq, wsf, tms)
    dx = dg.m_grouped_mxfp4_gemm_nt_ragged(dyq, dysf, wqt, wsft, tms)
    dw = dg.k_grouped_mxfp4_gemm_nt_ragged(dyqt, dysft, xqt, xsft, tms)
    torch.cuda.synchronize()
    xv, wv, dyv = (bf16_bits_to_f64(t) for t in (x, w, dy))
    yv, dxv, dwv = (bf16_bits_to_f64(bits(t)) for t in (y, dx, dw))
    c = lambda t: t.cpu().numpy()                                           # noqa: E731
    for got, args in ((yv, (xq, xsf, wq, wsf)), (dxv, (dyq, dysf, wqt, wsft))):
        for rows, ref, s in X.m_grouped_mxfp4_gemm_nt_ragged(*map(c, args), ms):
            assert (np.abs(got[rows] - ref) <= 2.0 ** -8 * np.abs(ref) + (k / 8 + 1) * 2.0 ** -23 * (1 + 2.0 ** -8) * s).all()
    ref, s = X.k_grouped_mxfp4_gemm_nt_ragged(*map(c, (dyqt, dysft, xqt, xsft)), ms)
    assert (np.abs(dwv - ref) <= 2.0 ** -8 * np.abs(ref) + (256 / 8 + 1) * 2.0 ** -23 * (1 + 2.0 ** -8) * s).all()
    # (E2M1 leaves an operand some 10 % off at random, a product's sum 15 % of its size)
    for g, (a, e) in enumerate(X.group_rows(ms, m)):
        for got, want in ((yv[a:e], xv[a:e] @ wv[g].T), (dxv[a:e], dyv[a:e] @ wv[g]), (dwv[g], dyv[a:e].T @ xv[a:e])):
            assert np.linalg.norm(got - want) <= 0.25 * np.linalg.norm(want)


@pytest.mark.parametrize("kernel", [0, 1, 4])
def test_graph_replays_follow_new_sizes(dg, kernel, monkeypatch):
    """The sizes are read on the device: a captured step replayed with other sizes in the same buffer computes those."""
    monkeypatch.setenv("DG_FORCE_MXFP4", str(kernel))
    n, k, G, m = 272, 384, 4, 300
    rng = np.random.default_rng(5)
    a, sa = integers(rng, m, k)
    b, sb = (np.stack(t) for t in zip(*(integers(rng, n, k) for _ in range(G))))
    t = [torch.from_numpy(v).cuda() for v in (a, sa, b, sb)]
    x, _ = to_dev(values(2, m, 256), torch.bfloat16)
    blocks = dg.dg_mxfp4_ragged_blocks(m, G)
    ms, d = device_ms([300, 0, 0, 0]), torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    qt, sft = torch.empty(256, blocks * 64, dtype=torch.uint8, device="cuda"), torch.empty(blocks, 256, dtype=torch.int32, device="cuda")
    dw = torch.empty(G, 256, 256, dtype=torch.bfloat16, device="cuda")

    def step():
        dg.dg_m_grouped_mxfp4_gemm_nt_ragged(*t, ms, d)
        dg.dg_quantize_mxfp4_ragged(x, ms, qt=qt, sft=sft)
        dg.dg_k_grouped_mxfp4_gemm_nt_ragged(qt, sft, qt, sft, ms, dw)

    step()
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for sizes in ([1, 2, 3, 4], [0, 299, 0, 1], [100, 0, 100, 100], [0, 0, 0, 0]):
        ms.copy_(torch.tensor(sizes, dtype=torch.int32))
        want = []
        for replay in (False, True):
            for o in (d, dw, qt, sft):
                o.view(torch.uint8).fill_(255 if o is d else 0)
            torch.cuda.synchronize()
            if replay:
                graph.replay()
            else:
                step()
            torch.cuda.synchronize()
            want.append([o.view(torch.uint8).cpu() for o in (d, dw, qt, sft)])
        assert all(torch.equal(p, q) for p, q in zip(*want)), sizes


def test_two_streams_at_once(dg):
    """Calls in flight together on two streams (they share nothing): each gives what it gives alone."""
    rng = np.random.default_rng(6)
    n, k = 528, 640
    sets = []
    for sizes in ([300, 0, 70, 1], [17, 200, 90]):
        a, sa = integers(rng, sum(sizes), k)
        b, sb = (np.stack(t) for t in zip(*(integers(rng, n, k) for _ in sizes)))
        t = [torch.from_numpy(v).cuda() for v in (a, sa, b, sb)] + [device_ms(sizes)]
        sets.append((t, dg.m_grouped_mxfp4_gemm_nt_ragged(*t)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = [[], []]
    for _ in range(10):
        for i, (t, _) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                outs[i].append(dg.m_grouped_mxfp4_gemm_nt_ragged(*t))
    torch.cuda.synchronize()
    for (_, want), got in zip(sets, outs):
        assert all(torch.equal(want, g) for g in got)
