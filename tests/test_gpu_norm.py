"""RMS norm with the residual's addition and a quantised output, and its backward pass, against the float64 oracle.

Tolerances.  The sum of k squares (positive terms) in fp32, added over at most k/64 values per thread and 16 steps
between threads, is off by (k/64 + 16) 2^-24 of itself; r = 1/sqrt by half of that and 4 roundings of 2^-24; y = h r w
and its scale by two more each.  D below is the sum, relative to y.  A code is one nearest to a value within D of the
exact y, so its value is no further from y than the nearest point of the grid is, by 2 D |y| (the move of y counts on
both sides), and a block's scale follows an amax within D of the exact one.
y is an fp32 value: below 2^-126 its two products are each off by half the subnormal step, 2^-150, besides, so a value
of at most 2^-150 may be 0 (and its block all zeros) and every bound on y has 2^-149 added.
"""

import numpy as np
import pytest
import torch

from oracle import mx as X
from oracle.formats import bf16_bits_to_f64, decode_e4m3, f64_to_bf16_bits, pow2_scale_exponent
from tests.helpers import bits
from tests.test_gpu_mxfp4 import guarded

pytestmark = pytest.mark.gpu

F32, UE8M0, MX = 0, 1, 2


def rel(k):
    return ((k / 64 + 16) / 2 + 8) * 2.0 ** -24


def bf(seed, *shape, scale=1.0):
    return f64_to_bf16_bits(np.random.default_rng(seed).standard_normal(shape) * scale)


def dev(b):
    return None if b is None else torch.from_numpy(b.view(np.int16).copy()).cuda().view(torch.bfloat16)


def run_norm(dgm, x, res, w, fmt, eps=1e-6, want_h=True, inplace=None):
    m, k = x.shape
    tx, tr, tw = dev(x), dev(res), dev(w)
    q, cq = guarded((m, k // 2 if fmt == MX else k), torch.uint8)
    sf, cs = guarded((m, (k + 511) // 512) if fmt == UE8M0 else (k // 128, m), torch.float32 if fmt == F32 else torch.int32)
    rstd, cr = guarded((m,), torch.float32)
    h, ch = guarded((m, k), torch.bfloat16) if want_h else (None, lambda: None)
    if inplace:
        h = {"x": tx, "residual": tr}[inplace]
    dgm.dg_add_rms_norm(tx, tr, tw, h, q, sf, eps, fmt, rstd)
    torch.cuda.synchronize()
    for c in (cq, cs, cr, ch):
        c()
    return q.cpu().numpy(), sf.cpu().numpy(), None if h is None else bits(h), rstd.cpu().numpy().astype(np.float64)


def block_scales(sf, fmt, m, k):
    """The scales per block [m, k/128] (or k/32) in float64."""
    if fmt == F32:
        return sf.T.astype(np.float64)
    if fmt == MX:
        return X.unpack_ue8m0_int32(np.ascontiguousarray(sf.T))
    s = X.unpack_ue8m0_int32(sf)
    assert (s[:, k // 128:] == 1).all(), "unused bytes of the last word"
    return s[:, :k // 128]


def check_norm(got, x, res, w, fmt, eps=1e-6):
    q, sf, hb, rstd = got
    m, k = x.shape
    h, r, y = X.add_rms_norm(x, res, w, eps)
    y = np.where(np.abs(y) <= 2.0 ** -150, 0.0, y)
    if hb is not None:
        assert np.array_equal(hb, f64_to_bf16_bits(h)), "h"
    d = rel(k)
    assert (np.abs(rstd - r) <= d * r).all(), "rstd"
    blk = 32 if fmt == MX else 128
    s = block_scales(sf, fmt, m, k)
    amax = np.abs(y).reshape(m, k // blk, blk).max(axis=2)
    if fmt == F32:
        want = np.where(amax > 0, np.maximum(amax / 448, 2.0 ** -126), 1.0)
        assert (np.abs(s - want) <= d * want).all(), "scales"
        unit = s
    else:
        qmax = 6.0 if fmt == MX else 448.0
        e = np.log2(s)
        assert (e == np.round(e)).all()
        zero = amax == 0
        assert (s[zero] == 1).all()
        assert (qmax * s >= amax * (1 - d))[~zero].all(), "a scale too small"
        assert ((qmax * s / 2 < amax * (1 + d)) | (e == -127))[~zero].all(), "a scale too large"
        unit = s
    unit = np.repeat(unit, blk, axis=1)
    grid = X.E2M1_GRID if fmt == MX else X.E4M3_GRID
    v = (X.unpack_e2m1(q) if fmt == MX else decode_e4m3(q)) * unit
    a = np.minimum(np.abs(y) / unit, grid[-1])
    best = np.abs(grid[X.nearest_code(a, grid)] * unit - np.abs(y))
    bad = ~(np.abs(v - y) <= best + 2 * (d * np.abs(y) + 2.0 ** -149))
    assert not bad.any(), f"{bad.sum()} codes, first at {np.argwhere(bad)[0]}: {v[bad][0]} for {y[bad][0]}"


@pytest.mark.parametrize("fmt", [F32, UE8M0, MX])
@pytest.mark.parametrize("m,k", [(1, 128), (3, 7168), (9, 640), (130, 2048), (33, 5120), (2, 16384), (5, 32768),
                                 (700, 1536), (2100, 384)])
def test_norm_shapes(dg, m, k, fmt):
    x, res, w = bf(m, m, k, scale=2.0), bf(k, m, k), f64_to_bf16_bits(1 + 0.3 * np.random.default_rng(1).standard_normal(k))
    r = res if (m + k // 128) % 3 else None
    check_norm(run_norm(dg, x, r, w, fmt), x, r, w, fmt)


@pytest.mark.parametrize("fmt", [F32, UE8M0, MX])
def test_norm_edges(dg, fmt):
    """Rows of zeros, of tiny values (eps decides), with one large value; weights that are 0 over a block, and that
    make amax subnormal; a row whose sum cancels."""
    m, k = 8, 768
    x, res, w = bf(3, m, k), bf(4, m, k), bf(5, k)
    x[0], res[0] = 0, 0
    x[1] = f64_to_bf16_bits(np.full(k, 2.0 ** -130))
    res[1] = 0
    x[2, 5] = f64_to_bf16_bits(np.float64(3e4))
    res[3] = x[3] ^ 0x8000                                  # h = 0
    w[128:256] = 0
    w[256:384] = f64_to_bf16_bits(np.full(128, 2.0 ** -128))
    check_norm(run_norm(dg, x, res, w, fmt), x, res, w, fmt)


@pytest.mark.parametrize("fmt", [F32, UE8M0, MX])
@pytest.mark.parametrize("value", [np.nan, np.inf, -np.inf])
def test_norm_nonfinite(dg, fmt, value):
    """A NaN makes its whole row NaN; an infinity its own block (r = 0 makes the others 0); other rows are unharmed."""
    m, k = 5, 512
    x, w = bf(6, m, k), f64_to_bf16_bits(np.ones(k))
    x[2, 200] = f64_to_bf16_bits(np.float64(value)) if not np.isnan(value) else 0x7fc0
    q, sf, _, rstd = run_norm(dg, x, None, w, fmt)
    blk = 32 if fmt == MX else 128
    s = block_scales(sf, fmt, m, k)
    nan_block = np.zeros((m, k // blk), dtype=bool)
    nan_block[2, :] = np.isnan(value)
    nan_block[2, 200 // blk] = True
    assert np.array_equal(np.isnan(s), nan_block)
    v = X.unpack_e2m1(q) if fmt == MX else decode_e4m3(q)
    if fmt != MX:
        assert np.isnan(v[2, 200])
    keep = [0, 1, 3, 4]
    sub = (q[keep], (sf[keep] if fmt == UE8M0 else np.ascontiguousarray(sf[:, keep])), None, rstd[keep])
    check_norm(sub, x[keep], None, w, fmt)


@pytest.mark.parametrize("inplace", ["x", "residual"])
def test_norm_in_place(dg, inplace):
    x, res, w = bf(7, 40, 1024), bf(8, 40, 1024), bf(9, 1024)
    check_norm(run_norm(dg, x, res, w, F32, inplace=inplace), x, res, w, F32)


def test_norm_without_h(dg):
    x, res, w = bf(7, 12, 1024), bf(8, 12, 1024), bf(9, 1024)
    check_norm(run_norm(dg, x, res, w, UE8M0, want_h=False), x, res, w, UE8M0)


def test_norm_large_batch_same_rows(dg):
    """A row's outputs do not depend on the batch it is in (the row counts cross the kernel's variants)."""
    k = 1536
    x, res, w = bf(10, 5000, k), bf(11, 5000, k), bf(12, k)
    big = run_norm(dg, x, res, w, MX)
    for m in (1, 40, 1300):
        part = run_norm(dg, x[:m], res[:m], w, MX)
        v = [X.dequant_mxfp4(part[0], part[1]), X.dequant_mxfp4(big[0][:m], np.ascontiguousarray(big[1][:, :m]))]
        assert np.array_equal(part[2], big[2][:m])
        # (the row sum's order may differ between the variants: only codes at a border may)
        assert (v[0] != v[1]).mean() <= 1e-3
    check_norm(big, x, res, w, MX)


def run_back(dgm, dy, dh, h, w, rstd, into=None):
    m, k = dy.shape
    t = dict(dy=dev(dy), dh=dev(dh), h=dev(h), w=dev(w), r=torch.from_numpy(rstd.astype(np.float32)).cuda())
    dx, cx = guarded((m, k), torch.bfloat16) if into is None else (t[into], lambda: None)
    dw, cw = guarded((k,), torch.float32)
    ws, cws = guarded((dgm.dg_add_rms_norm_backward_workspace_bytes(m, k),), torch.uint8)
    dgm.dg_add_rms_norm_backward(t["dy"], t["dh"], t["h"], t["w"], t["r"], dx, dw, ws)
    torch.cuda.synchronize()
    for c in (cx, cw, cws):
        c()
    return bits(dx), dw.cpu().numpy().astype(np.float64)


def back_inputs(m, k, with_dh, seed=0):
    h, w = bf(seed, m, k, scale=1.5), f64_to_bf16_bits(1 + 0.3 * np.random.default_rng(seed + 1).standard_normal(k))
    dy, dh = bf(seed + 2, m, k, scale=0.1), bf(seed + 3, m, k, scale=0.1) if with_dh else None
    r = 1 / np.sqrt(np.mean(bf16_bits_to_f64(h) ** 2, axis=1) + 1e-6)
    return dy, dh, h, w, r.astype(np.float32)


def check_back(got, dy, dh, h, w, rstd):
    """dx: the bf16 rounding, 2^-8 of it, and fp32: the mean of k products within (k/64 + 16) 2^-24 of the mean of
    their magnitudes, and 8 roundings of each term.  dweight: m products added in any order, (m + 4) 2^-24 of their
    magnitudes' sum."""
    m, k = dy.shape
    f = [bf16_bits_to_f64(v) for v in (dy, h, w)]
    d = None if dh is None else bf16_bits_to_f64(dh)
    r = rstd.astype(np.float64)
    dx, dw = X.add_rms_norm_backward(f[0], d, f[1], f[2], r)
    n, g = f[1] * r[:, None], f[0] * f[2]
    terms = r[:, None] * (np.abs(g) + np.abs(n) * np.mean(np.abs(g * n), axis=1, keepdims=True)) + (0 if d is None else np.abs(d))
    bound = 2.0 ** -8 * np.abs(dx) + (k / 64 + 24) * 2.0 ** -24 * (1 + 2.0 ** -8) * terms
    err = np.abs(bf16_bits_to_f64(got[0]) - dx)
    assert (err <= bound).all(), f"dx: {(err > bound).sum()}, worst {np.max(err / np.maximum(bound, 1e-300))} of the bound"
    bound = (m + 4) * 2.0 ** -24 * np.sum(np.abs(f[0] * n), axis=0)
    assert (np.abs(got[1] - dw) <= bound).all(), "dweight"


@pytest.mark.parametrize("with_dh", [False, True])
@pytest.mark.parametrize("m,k", [(1, 128), (2, 7168), (130, 2048), (37, 640), (600, 1536), (1500, 384), (3, 32768),
                                 (520, 5120), (9, 16384)])
def test_backward_shapes(dg, m, k, with_dh):
    a = back_inputs(m, k, with_dh, seed=m + k)
    check_back(run_back(dg, *a), *a)


@pytest.mark.parametrize("m,k", [(256, 4096), (257, 4096), (256, 4224), (256, 8192), (257, 8320), (200, 16512), (1024, 640),
                                 (1025, 128), (1025, 640), (1100, 7168), (1030, 16384), (1027, 32768)])
def test_backward_at_the_kernels_borders(dg, m, k):
    a = back_inputs(m, k, True, seed=m + k)
    check_back(run_back(dg, *a), *a)


@pytest.mark.parametrize("into", ["dy", "dh"])
def test_backward_of_many_rows_in_place(dg, into):
    a = back_inputs(1300, 1024, True)
    want = run_back(dg, *a)
    got = run_back(dg, *a, into=into)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


@pytest.mark.parametrize("into", ["dy", "dh"])
def test_backward_in_place(dg, into):
    a = back_inputs(70, 1024, True)
    want = run_back(dg, *a)
    got = run_back(dg, *a, into=into)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_backward_nonfinite_rows_stay_apart(dg):
    """A NaN gradient makes its row of dx and its column of dweight NaN, and no other row of dx."""
    dy, dh, h, w, r = back_inputs(300, 512, True)
    dy[17, 100] = 0x7fc0
    dx, dw = run_back(dg, dy, dh, h, w, r)
    nan = np.isnan(bf16_bits_to_f64(dx))
    assert nan[17].all() and not np.delete(nan, 17, axis=0).any()
    assert np.isnan(dw[100]) and np.isfinite(np.delete(dw, 100)).all()


def test_backward_against_differences_of_the_forward(dg):
    """dx along a direction against the difference of the norm's own forward: with r and the scales of the F32 format
    the unquantised y is not returned, so the forward is the oracle's, at the kernel's h and eps."""
    m, k, eps = 3, 256, 1e-6
    dy, _, h, w, r = back_inputs(m, k, False, seed=40)
    dx = bf16_bits_to_f64(run_back(dg, dy, None, h, w, r)[0])
    hv, wv, gv = (bf16_bits_to_f64(v) for v in (h, w, dy))
    u = np.random.default_rng(3).standard_normal((m, k))

    def loss(hh):
        return np.sum(gv * hh / np.sqrt(np.mean(hh * hh, axis=1, keepdims=True) + eps) * wv, axis=1)
    t = 1e-4                                               # central: error ~ t^2
    diff = (loss(hv + t * u) - loss(hv - t * u)) / (2 * t)
    got = np.sum(dx * u, axis=1)
    # dx is rounded to bf16 (2^-8 of each term); r is fp32; the third derivative's share is t^2 ~ 1e-8 of the terms
    assert (np.abs(got - diff) <= (2.0 ** -8 + 1e-6) * np.sum(np.abs(dx * u), axis=1)).all()


@pytest.mark.parametrize("m", [333, 1333])
def test_backward_repeats_and_graph_replays(dg, m):
    k = 7168
    a = back_inputs(m, k, True, seed=50)
    t = [dev(v) for v in a[:4]] + [torch.from_numpy(a[4]).cuda()]
    want = dg.add_rms_norm_backward(*t)
    dx, dw = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty(dg.dg_add_rms_norm_backward_workspace_bytes(m, k), dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dg.dg_add_rms_norm_backward(*t, dx, dw, ws)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dg.dg_add_rms_norm_backward(*t, dx, dw, ws)
    for i in range(4):
        for v in (dx, dw):
            v.fill_(float("nan"))
        ws.fill_(255 - i)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(dx, want[0]) and torch.equal(dw, want[1]), f"replay {i}"


def test_a_block_of_calls_and_its_graph(dg):
    """Norm -> MXFP4 GEMM -> norm -> FP8 GEMM with UE8M0 scales, as a layer runs them, eagerly against the oracle's
    products on the kernels' own operands, and captured in a graph whose replays follow changed inputs."""
    import synth
    from oracle import ref as R
    m, k, n = 70, 512, 768
    x, res, w1, w2 = bf(60, m, k), bf(61, m, k), bf(62, k), bf(63, n)
    tx, tr, tw1, tw2 = dev(x), dev(res), dev(w1), dev(w2)
    wq, wsf = dg.quantize_mxfp4(torch.randn(n, k, device="cuda"))
    b = synth.gen_dense_ue8m0(16, 256, n, seed=1, with_c=False)
    b2, sfb2 = b["b"].cuda(), b["sfb"].cuda()

    def block():
        q, sf, h, _ = dg.add_rms_norm(tx, tr, tw1, 1e-6, dg.QUANT_MXFP4)
        y = dg.mxfp4_gemm_nt(q, sf, wq, wsf)
        q2, sf2, _, _ = dg.add_rms_norm(y, None, tw2, 1e-6, dg.QUANT_E4M3_UE8M0)
        d = torch.empty(m, 256, dtype=torch.bfloat16, device="cuda")
        dg.dg_fp8_gemm_nt_ue8m0(q2, sf2, b2, sfb2, None, d)
        return q, sf, h, y, q2, sf2, d

    q, sf, h, y, q2, sf2, d = block()
    n_ = lambda t: t.cpu().numpy()                                                      # noqa: E731
    check_norm((n_(q), n_(sf), bits(h), 1 / np.sqrt(np.mean(bf16_bits_to_f64(bits(h)) ** 2, axis=1) + 1e-6)), x, res, w1, MX)
    ref = X.mxfp4_gemm_nt(n_(q), n_(sf), n_(wq), n_(wsf))
    a_, b_ = X.dequant_mxfp4(n_(q), n_(sf)), X.dequant_mxfp4(n_(wq), n_(wsf))
    assert (np.abs(bf16_bits_to_f64(bits(y)) - ref) <= 2.0 ** -8 * np.abs(ref) + (k / 8 + 1) * 2.0 ** -22 * (np.abs(a_) @ np.abs(b_).T)).all()
    yb = bits(y)
    check_norm((n_(q2), n_(sf2), None, 1 / np.sqrt(np.mean(bf16_bits_to_f64(yb) ** 2, axis=1) + 1e-6)), yb, None, w2, UE8M0)
    ref = R.fp8_gemm_nt_ue8m0(n_(q2), n_(sf2), n_(b2), n_(sfb2))
    from tests.helpers import check_parity
    check_parity(bits(d), ref, what="block")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = block()
    for i in range(3):
        tx.copy_(dev(bf(70 + i, m, k)))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, block()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), f"replay {i}"


def test_training_step_of_norm_and_layer(dg):
    """h = x + residual, y = q(norm(h)) . q(w)^T and back: the layer's input gradient dn = q(dy) . qt(w)^T feeds the
    norm's backward pass with the residual branch's gradient; each step against the oracle on the step's own inputs."""
    T, K, N = 90, 384, 256
    x, res, wn = bf(80, T, K), bf(81, T, K), f64_to_bf16_bits(1 + 0.3 * np.random.default_rng(82).standard_normal(K))
    w, dy, dh = bf(83, N, K), bf(84, T, N), bf(85, T, K)
    q, sf, h, rstd = dg.add_rms_norm(dev(x), dev(res), dev(wn), 1e-6, dg.QUANT_MXFP4)
    wq, wsf, wqt, wsft = dg.quantize_mxfp4(dev(w), transposed=True)
    y = dg.mxfp4_gemm_nt(q, sf, wq, wsf)
    dyq, dysf = dg.quantize_mxfp4(dev(dy))
    dn = dg.mxfp4_gemm_nt(dyq, dysf, wqt, wsft)
    dx, dw = dg.add_rms_norm_backward(dn, dev(dh), h, dev(wn), rstd)
    n_ = lambda t: t.cpu().numpy()                                                      # noqa: E731
    for got, a, asf, b, bsf, k in ((y, q, sf, wq, wsf, K), (dn, dyq, dysf, wqt, wsft, N)):
        a_, b_ = X.dequant_mxfp4(n_(a), n_(asf)), X.dequant_mxfp4(n_(b), n_(bsf))
        ref, s = a_ @ b_.T, np.abs(a_) @ np.abs(b_).T
        assert (np.abs(bf16_bits_to_f64(bits(got)) - ref) <= 2.0 ** -8 * np.abs(ref) + (k / 8 + 1) * 2.0 ** -22 * s).all()
    check_back((bits(dx), n_(dw).astype(np.float64)), bits(dn), dh, bits(h), wn, n_(rstd))


@pytest.mark.parametrize("m", [500, 1500])
def test_two_calls_at_once_on_two_streams(dg, m):
    """Backward passes in flight together, each with a workspace of its own, and forward passes between them."""
    a = [back_inputs(m, 1024, True, seed=s) for s in (1, 2)]
    t = [[dev(v) for v in i[:4]] + [torch.from_numpy(i[4]).cuda()] for i in a]
    want = [dg.add_rms_norm_backward(*i) for i in t]
    fwd = [dg.add_rms_norm(i[2], i[0], i[3]) for i in t]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, dg.add_rms_norm_backward(*t[i]), dg.add_rms_norm(t[i][2], t[i][0], t[i][3])))
    torch.cuda.synchronize()
    for i, b, f in got:
        assert torch.equal(b[0], want[i][0]) and torch.equal(b[1], want[i][1])
        assert all(torch.equal(u, v) for u, v in zip(f, fwd[i]))


@pytest.mark.parametrize("m,k", [(3, 7168), (200, 2048), (64, 16384), (70, 640)])
def test_fp32_scale_codes_and_ties(dg, m, k):
    """The codes of the fp32-scale format are those of 448 y / max|y| exactly, ties to the even code: the row's r
    cancels, and 448 (h w) / max|h w| is a ratio of integers of at most 25 bits, so that float64's quotient is a midpoint
    of two codes if and only if the exact one is.  The scale is max|y| / 448 in fp32 of the kernel's own r."""
    x, res, w = bf(90 + m, m, k, scale=2.0), bf(91, m, k), f64_to_bf16_bits(1 + 0.2 * np.random.default_rng(2).standard_normal(k))
    q, sf, hb, rstd = run_norm(dg, x, res, w, F32)
    p = bf16_bits_to_f64(hb) * bf16_bits_to_f64(w)                       # exact
    blocks = np.abs(p).reshape(m, k // 128, 128)
    amax = blocks.max(axis=2)
    v = (blocks * 448 / amax[..., None]).reshape(m, k)
    if m * k >= 200 * 2048:                                              # the inputs meet ties
        mids = (X.E4M3_GRID[1:] + X.E4M3_GRID[:-1]) / 2
        assert np.isin(v, mids).sum() >= 20
    want = X.nearest_code(v, X.E4M3_GRID).astype(np.uint8) | (np.signbit(p).astype(np.uint8) << 7)
    assert np.array_equal(q, want), f"{np.count_nonzero(q != want)} of {q.size} codes differ"
    top = amax.astype(np.float32) * rstd.astype(np.float32)[:, None]
    assert np.array_equal(sf.T, top / np.float32(448))


@pytest.mark.parametrize("fmt", [F32, UE8M0, MX])
@pytest.mark.parametrize("he,we,eps", [(55, 75, 1e-6), (-80, -60, 2.0 ** -120), (-100, -60, 2.0 ** -126), (-30, -40, 1e-6)])
def test_norm_products_outside_fp32(dg, fmt, he, we, eps):
    """h * weight leaves fp32's range (to infinity, to subnormals, to 0) where y = h * r * weight does not; in one row of
    blocks or in some of its blocks only.  One rounding to fp32 is within the bound on y."""
    m, k = 6, 1024
    x, w = bf(100, m, k, scale=2.0 ** he), bf(101, k, scale=2.0 ** we)
    x[1, :512] = bf(102, 512, scale=2.0 ** (he // 2))
    x[2, 7::64] = 0
    w[128:256] = bf(103, 128)
    check_norm(run_norm(dg, x, None, w, fmt, eps=eps), x, None, w, fmt, eps)


@pytest.mark.parametrize("m,k", [(1, 2048), (70, 2048), (1000, 1152), (1300, 2048), (1030, 20480)])
@pytest.mark.parametrize("with_dh", [False, True])
def test_backward_into_h(dg, m, k, with_dh):
    """dx written over h: the workgroups that sum dweight have read h before a row of it is overwritten."""
    a = back_inputs(m, k, with_dh, seed=7)
    want = run_back(dg, *a)
    for _ in range(4):
        got = run_back(dg, *a, into="h")
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


@pytest.mark.parametrize("fmt", [F32, UE8M0, MX])
@pytest.mark.parametrize("k", [384, 1536, 7168, 16384])
def test_norm_rows_do_not_depend_on_the_batch(dg, k, fmt):
    """The kernel is a function of k and the format: a row's outputs are bit for bit the same in any batch."""
    m = 1500
    x, res, w = bf(10, m, k), bf(11, m, k), bf(12, k)
    big = run_norm(dg, x, res, w, fmt)
    for rows in (slice(0, 1), slice(3, 43), slice(700, 1500)):
        q, sf, h, r = run_norm(dg, x[rows], res[rows], w, fmt)
        assert np.array_equal(q, big[0][rows]) and np.array_equal(h, big[2][rows]) and np.array_equal(r, big[3][rows])
        assert np.array_equal(sf, big[1][rows] if fmt == UE8M0 else big[1][:, rows])


@pytest.mark.parametrize("m,k", [(3, 128), (40, 2048), (9, 7168), (5, 32768)])
def test_norm_rstd(dg, m, k):
    """r is formed in 64 bits (squares of bf16 numbers are exact there) and rounded once: half a place, 2^-24 of it."""
    x, res, w = bf(110, m, k, scale=3.0), bf(111, m, k), bf(112, k)
    _, _, hb, rstd = run_norm(dg, x, res, w, UE8M0)
    r = 1 / np.sqrt(np.mean(bf16_bits_to_f64(hb) ** 2, axis=1) + float(np.float32(1e-6)))
    assert (np.abs(rstd - r) <= 2.0 ** -24 * (1 + 2.0 ** -20) * r).all()


def test_block_of_calls_keeps_rstd_and_feeds_the_fp32_scale_gemm(dg):
    """Norm -> MXFP4 GEMM -> norm with fp32 scales -> FP8 GEMM, each stage on the operands that the one before it made:
    both rstd are the kernel's own, and the products hold to (K/8 + 1) 2^-23 of their magnitudes."""
    import synth
    from oracle import ref as R
    from tests.helpers import check_parity
    m, k, n = 70, 512, 768
    x, res, w1, w2 = bf(60, m, k), bf(61, m, k), bf(62, k), bf(63, n)
    wq, wsf = dg.quantize_mxfp4(torch.randn(n, k, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)))
    g = synth.gen_dense(16, 256, n, seed=1, with_c=False)
    b2, sfb2 = g["b"].cuda(), g["sfb"].cuda()
    q, sf, h, rstd = dg.add_rms_norm(dev(x), dev(res), dev(w1), 1e-6, dg.QUANT_MXFP4)
    y = dg.mxfp4_gemm_nt(q, sf, wq, wsf)
    q2, sf2, h2, rstd2 = dg.add_rms_norm(y, None, dev(w2), 1e-6, dg.QUANT_E4M3_F32)
    d = torch.empty(m, 256, dtype=torch.bfloat16, device="cuda")
    dg.dg_fp8_gemm_nt(q2, sf2, b2, sfb2, None, d)
    n_ = lambda t: t.cpu().numpy()                                                      # noqa: E731
    check_norm((n_(q), n_(sf), bits(h), n_(rstd).astype(np.float64)), x, res, w1, MX)
    a_, b_ = X.dequant_mxfp4(n_(q), n_(sf)), X.dequant_mxfp4(n_(wq), n_(wsf))
    ref, s = a_ @ b_.T, np.abs(a_) @ np.abs(b_).T
    assert (np.abs(bf16_bits_to_f64(bits(y)) - ref) <= 2.0 ** -8 * np.abs(ref) + (k / 8 + 1) * 2.0 ** -23 * (1 + 2.0 ** -8) * s).all()
    check_norm((n_(q2), n_(sf2), bits(h2), n_(rstd2).astype(np.float64)), bits(y), None, w2, F32)
    check_parity(bits(d), R.fp8_gemm_nt(n_(q2), n_(sf2), n_(b2), n_(sfb2)), what="fp8 gemm on the norm's codes")


def test_training_step_with_the_weight_gradient(dg):
    """The layer's dw = qt(dy) . qt(y)^T behind a norm: y leaves the norm as codes with blocks along k only, so the
    caller forms it again in bf16 from h and rstd; all three products to (K/8 + 1) 2^-23 of their magnitudes."""
    T, K, N = 150, 384, 256
    x, res, wn = bf(80, T, K), bf(81, T, K), f64_to_bf16_bits(1 + 0.3 * np.random.default_rng(82).standard_normal(K))
    w, dy, dh = bf(83, N, K), bf(84, T, N), bf(85, T, K)
    q, sf, h, rstd = dg.add_rms_norm(dev(x), dev(res), dev(wn), 1e-6, dg.QUANT_MXFP4)
    y = (h.float() * rstd[:, None] * dev(wn).float()).to(torch.bfloat16)
    _, _, yt, yst = dg.quantize_mxfp4(y, transposed=True)
    wq, wsf, wqt, wsft = dg.quantize_mxfp4(dev(w), transposed=True)
    dyq, dysf, dyt, dyst = dg.quantize_mxfp4(dev(dy), transposed=True)
    out, dn, dw = dg.mxfp4_gemm_nt(q, sf, wq, wsf), dg.mxfp4_gemm_nt(dyq, dysf, wqt, wsft), dg.mxfp4_gemm_nt(dyt, dyst, yt, yst)
    dx, dweight = dg.add_rms_norm_backward(dn, dev(dh), h, dev(wn), rstd)
    n_ = lambda t: t.cpu().numpy()                                                      # noqa: E731
    for got, a, asf, b, bsf, k in ((out, q, sf, wq, wsf, K), (dn, dyq, dysf, wqt, wsft, N), (dw, dyt, dyst, yt, yst, 256)):
        a_, b_ = X.dequant_mxfp4(n_(a), n_(asf)), X.dequant_mxfp4(n_(b), n_(bsf))
        ref, s = a_ @ b_.T, np.abs(a_) @ np.abs(b_).T
        assert (np.abs(bf16_bits_to_f64(bits(got)) - ref) <= 2.0 ** -8 * np.abs(ref) + (k / 8 + 1) * 2.0 ** -23 * (1 + 2.0 ** -8) * s).all()
    ty, tsy = X.quantize_mxfp4_transposed(bf16_bits_to_f64(bits(y)))
    assert np.array_equal(n_(yt), ty) and np.array_equal(n_(yst), tsy)
    check_back((bits(dx), n_(dweight).astype(np.float64)), bits(dn), dh, bits(h), wn, n_(rstd))


@pytest.mark.parametrize("fmt", [UE8M0, MX])
@pytest.mark.parametrize("m,k", [(3, 7168), (300, 7168), (1000, 2048), (40, 32768)])
def test_power_of_two_scales_and_codes_are_the_nearest(dg, m, k, fmt):
    """Codes and scales are bit for bit those of y in float64: an r of 48 bits moves y by 2^-48 of itself, float64 by 2^-51,
    and of these few million values none lies as near as 2^-40 to a midpoint of two codes (asserted).  The roundings of
    r and y to fp32 would decide one code in some two million."""
    x, res, w = bf(120 + m, m, k, scale=2.0), bf(121, m, k), f64_to_bf16_bits(1 + 0.2 * np.random.default_rng(3).standard_normal(k))
    q, sf, hb, _ = run_norm(dg, x, res, w, fmt)
    h = bf16_bits_to_f64(hb)
    y = h * (1 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + float(np.float32(1e-6)))) * bf16_bits_to_f64(w)
    blk, grid = (32, X.E2M1_GRID) if fmt == MX else (128, X.E4M3_GRID)
    b = np.abs(y).reshape(m, k // blk, blk)
    e = pow2_scale_exponent(b.max(axis=2), grid[-1])
    assert np.array_equal(block_scales(sf, fmt, m, k), np.exp2(e))
    v = np.ldexp(b, -e[..., None]).reshape(m, k)
    mids = (grid[1:] + grid[:-1]) / 2
    near = np.abs(v - mids[np.minimum(np.searchsorted(mids, v), len(mids) - 1)])
    assert (np.minimum(near, np.abs(v - mids[np.maximum(np.searchsorted(mids, v) - 1, 0)])) > 2.0 ** -40 * v).all()
    want = X.nearest_code(v, grid).astype(np.uint8)
    got = np.stack([q & 15, q >> 4], axis=-1).reshape(m, k) if fmt == MX else q
    assert np.array_equal(got & (7 if fmt == MX else 127), want), f"{np.count_nonzero((got & (7 if fmt == MX else 127)) != want)} codes"


@pytest.mark.parametrize("fmt", [F32, UE8M0, MX])
def test_norm_squares_outside_fp32(dg, fmt):
    """Rows whose squares pass fp32's range, at either end."""
    m, k = 4, 1024
    x, w = bf(130, m, k), f64_to_bf16_bits(1 + 0.2 * np.random.default_rng(3).standard_normal(k))
    x[1], x[2], x[3] = bf(131, k, scale=2.0 ** 100), bf(132, k, scale=2.0 ** 122), bf(133, k, scale=2.0 ** -90)
    check_norm(run_norm(dg, x, None, w, fmt, eps=2.0 ** -126), x, None, w, fmt, 2.0 ** -126)


@pytest.mark.parametrize("fmt", [F32, UE8M0, MX])
def test_norm_values_past_fp32(dg, fmt):
    """A y past fp32's range makes its block's scale NaN; the largest y that is inside it does not."""
    m, k = 3, 512
    x = bf(140, m, k, scale=2.0 ** -10)                                 # (h * weight stays inside)
    w = f64_to_bf16_bits(np.ones(k))
    w[200], w[300] = 0x7f7f, 0x7f7f                                     # 3.39e38
    x[:, 200], x[:, 300] = f64_to_bf16_bits(np.float64(3 / 1024)), f64_to_bf16_bits(np.float64(0.5 / 1024))
    q, sf, _, _ = run_norm(dg, x, None, w, fmt)
    y = X.add_rms_norm(x, None, w, 1e-6)[2]
    assert (np.abs(y[:, 200]) > 3.5e38).all() and (np.abs(y[:, 300]) < 3e38).all()
    blk = 32 if fmt == MX else 128
    nan = np.zeros((m, k // blk), dtype=bool)
    nan[:, 200 // blk] = True
    assert np.array_equal(np.isnan(block_scales(sf, fmt, m, k)), nan)
    v = X.unpack_e2m1(q) if fmt == MX else decode_e4m3(q)
    bad = np.repeat(nan, blk, axis=1)
    assert (v[bad] == 0).all() if fmt == MX else np.isnan(v[bad]).all()
    assert (np.abs(v[:, 300]) > (2 if fmt == MX else 200)).all()
