"""The norms around a block (gate, residual scale, quantised output) and their backward pass, against the float64 oracle.

Tolerances.  h is one fp64 expression of bf16 numbers, rounded to fp32 and to bf16: the oracle's, rounded the same way,
bit for bit (the two fp64 values differ by some 2^-51 of themselves, so they lie on two sides of an fp32 midpoint once
in 2^27 values; no input here has such a value).  q, sf and rstd are those of the norm of the stored h and are held to
what tests/test_gpu_norm.py derives.

Backward, u = 2^-24: a sum over a row takes at most 32 additions a thread, 6 between lanes and 16 between waves, and its
terms carry at most 4 roundings: off by 64 u of the sum of magnitudes.  What follows it has at most 8 roundings of each
term.  A sum over m rows makes m additions at most, of terms with up to 8 roundings.  bf16 outputs add 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

from oracle import mx as X
from oracle.formats import bf16_bits_to_f64, f64_to_bf16_bits
from tests.helpers import bits
from tests.test_gpu_mxfp4 import guarded
from tests.test_gpu_norm import F32, MX, UE8M0, bf, check_norm, dev

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def bf16_of_fp32(v):
    """float64 -> bf16 bits through fp32, both to nearest even."""
    with np.errstate(over="ignore"):
        return f64_to_bf16_bits(np.asarray(v).astype(np.float32).astype(np.float64))


def by_row(gate, gate_rows, m):
    return None if gate is None else np.repeat(bf16_bits_to_f64(gate), gate_rows, axis=0)[:m]


def inputs(seed, m, k, gate_rows, post=True):
    x, res = bf(seed, m, k, scale=2.0), bf(seed + 1, m, k)
    w, pw = (f64_to_bf16_bits(1 + 0.3 * np.random.default_rng(seed + s).standard_normal(k)) for s in (2, 3))
    gate = bf(seed + 4, -(-m // gate_rows), k) if gate_rows else None
    return x, res, pw if post else None, gate, w


def run(dgm, x, res, pw, gate, w, fmt, gate_rows, scale, eps=1e-6, inplace=None):
    m, k = x.shape
    t = [dev(v) for v in (x, res, pw, gate, w)]
    q, cq = guarded((m, k // 2 if fmt == MX else k), torch.uint8)
    sf, cs = guarded((m, (k + 511) // 512) if fmt == UE8M0 else (k // 128, m), torch.float32 if fmt == F32 else torch.int32)
    rstd, cr = guarded((m,), torch.float32)
    rstd_x, cx = guarded((m,), torch.float32)
    h, ch = guarded((m, k), torch.bfloat16)
    if inplace is not None:
        h = t[inplace]
    dgm.dg_sandwich_norm(*t, h, q, sf, fmt, rstd_x, rstd, gate_rows or 1, scale, eps)
    torch.cuda.synchronize()
    for c in (cq, cs, cr, cx, ch):
        c()
    return (q.cpu().numpy(), sf.cpu().numpy(), bits(h), rstd.cpu().numpy().astype(np.float64)), rstd_x.cpu().numpy().astype(np.float64)


def check(got, rstd_x, x, res, pw, gate, w, fmt, gate_rows, scale, eps=1e-6, fp64=False):
    """fp64: h is anything between the roundings of values 2^-48 of the magnitudes in it below and above the oracle's."""
    m, k = x.shape
    f = [None if v is None else bf16_bits_to_f64(v) for v in (x, res, pw)]
    h, rx = X.sandwich_norm(*f, by_row(gate, gate_rows, m), scale, eps)
    want = bf16_of_fp32(h)
    bad = got[2] != want
    if fp64:
        # Where the residual cancels the branch but for the roundings on the way (scale 0.7: 0.7 * 0.2734375 - 0.19140625 is
        # some 10^-17), h is what they leave.  The oracle rounds three products, 1/rms (a sum of k squares in pairs, a
        # root and a division: 2^-49 at most here) and the sum; the kernel c = scale * rx (rx within 2^-49) and one fma:
        # together below 2^-48 of |residual| + |branch|, and both roundings behind it keep the order.
        off = 2.0 ** -48 * (np.abs(f[1]) + np.abs(h - f[1]))
        lo, hi, is_ = (bf16_bits_to_f64(v) for v in (bf16_of_fp32(h - off), bf16_of_fp32(h + off), got[2]))
        bad &= ~((lo <= is_) & (is_ <= hi))
    assert not bad.any(), f"h: {bad.sum()} differ, first at {np.argwhere(bad)[0]}"
    if pw is not None:
        assert (np.abs(rstd_x - rx) <= 2 * U * rx).all(), "rstd_x"
    check_norm(got, got[2], None, w, fmt, eps)


@pytest.mark.parametrize("fmt", [F32, UE8M0, MX])
@pytest.mark.parametrize("m,k,gate_rows", [(1, 128, 1), (3, 7168, 3), (9, 640, 0), (130, 2048, 50), (33, 5120, 1), (2, 16384, 7),
                                           (5, 32768, 2), (300, 1536, 128), (1100, 384, 256)])
def test_sandwich_shapes(dg, m, k, gate_rows, fmt):
    a = inputs(m + k, m, k, gate_rows, post=(m + k // 128) % 4 != 0)
    scale = (1.0, 0.7, -2.5)[m % 3]
    check(*run(dg, *a, fmt, gate_rows, scale), *a, fmt, gate_rows, scale)


@pytest.mark.parametrize("fmt", [F32, UE8M0, MX])
def test_sandwich_edges(dg, fmt):
    """Rows of zeros, of tiny and of huge values (products that leave fp32's range on the way), gates of zero, a residual
    that cancels, a scale of 0."""
    m, k = 9, 768
    x, res, pw, gate, w = inputs(3, m, k, 2)
    x[0], res[0] = 0, 0
    x[1] = f64_to_bf16_bits(np.full(k, 2.0 ** -120))
    pw[:40] = f64_to_bf16_bits(np.full(40, 2.0 ** -30))          # 2^-150 with row 1: by fp64
    x[2] = f64_to_bf16_bits(bf16_bits_to_f64(x[2]) * 2.0 ** 120)
    pw[300:340] = f64_to_bf16_bits(np.full(40, 2.0 ** 20))       # 2^140 with row 2
    x[3] = 0
    gate[2] = 0
    res[6] = f64_to_bf16_bits(np.full(k, 2.0 ** -133))
    for scale in (0.7, 0.0):
        check(*run(dg, x, res, pw, gate, w, fmt, 2, scale), x, res, pw, gate, w, fmt, 2, scale)


@pytest.mark.parametrize("value", [np.nan, np.inf])
def test_sandwich_nonfinite(dg, value):
    """A NaN in x makes its row NaN, an infinity itself alone (rx is 0: the others are the residual); other rows are unharmed."""
    m, k = 5, 512
    x, res, pw, gate, w = inputs(6, m, k, 1)
    clean, _ = run(dg, x, res, pw, gate, w, F32, 1, 1.0)
    x[2, 200] = 0x7fc0 if np.isnan(value) else f64_to_bf16_bits(np.float64(value))
    (q, sf, h, rstd), rstd_x = run(dg, x, res, pw, gate, w, F32, 1, 1.0)
    hv = bf16_bits_to_f64(h)
    assert np.isnan(hv[2, 200]) and np.isnan(rstd[2])
    if np.isnan(value):
        assert np.isnan(hv[2]).all() and np.isnan(rstd_x[2])
    else:
        assert rstd_x[2] == 0 and np.array_equal(np.delete(h[2], 200), np.delete(res[2], 200))
    keep = [0, 1, 3, 4]
    assert np.array_equal(h[keep], clean[2][keep]) and np.array_equal(q[keep], clean[0][keep])
    assert np.array_equal(sf[:, keep], clean[1][:, keep])


@pytest.mark.parametrize("which", [0, 1])
def test_sandwich_in_place(dg, which):
    a = inputs(11, 7, 1280, 3)
    got, rx = run(dg, *a, MX, 3, 0.5, inplace=which)
    check(got, rx, *a, MX, 3, 0.5)


@pytest.mark.parametrize("fmt", [F32, UE8M0, MX])
@pytest.mark.parametrize("m,k,gate_rows,post", [(2048, 4224, 700, True), (2065, 7168, 1, True), (2100, 8192, 2100, False),
                                                (100, 8320, 7, True), (64, 12288, 64, True), (90, 11008, 1, False)])
def test_sandwich_long_rows_many(dg, m, k, gate_rows, post, fmt):
    """Long rows, and many of them, run on other kernels: the rows of two halves, bit for bit, and the oracle's on some."""
    a = inputs(m, m, k, gate_rows, post)
    a[0][7], a[1][7] = 0, 0                       # eps alone decides
    a[0][40], a[1][40] = a[0][40] & 0x87ff, 0     # far below 1: products of fp64
    a[0][m - 1, 5] = 0x7fc0
    got, rx = run(dg, *a, fmt, gate_rows, 0.7)
    half = -(-m // 2 // gate_rows) * gate_rows if gate_rows <= m // 2 else m // 2 + 1
    for lo, hi in ((0, half), (half, m)):
        gate = a[3] if gate_rows >= m else a[3][lo // gate_rows:]
        part, prx = run(dg, a[0][lo:hi], a[1][lo:hi], a[2], gate[:-(-(hi - lo) // gate_rows)], a[4], fmt, gate_rows, 0.7)
        assert np.array_equal(prx.view(np.int64), rx[lo:hi].view(np.int64)) or not post
        for i, (g, w) in enumerate(zip(got, part)):
            g = g[:, lo:hi] if i == 1 and fmt != UE8M0 else g[lo:hi]
            assert np.array_equal(np.ascontiguousarray(g).view(np.uint8), np.ascontiguousarray(w).view(np.uint8)), i
    few = [v[:48] for v in a[:2]] + [a[2], a[3][:-(-48 // gate_rows)], a[4]]
    sf = got[1][:, :48] if fmt != UE8M0 else got[1][:48]
    check((got[0][:48], sf, got[2][:48], got[3][:48]), rx[:48], *few, fmt, gate_rows, 0.7, fp64=True)


def test_sandwich_wrapper_matches_the_plain_norm(dg):
    """Without a post-norm and gate and with scale 1 it is add_rms_norm, bit for bit."""
    x, res, _, _, w = inputs(12, 40, 2048, 0)
    t = [dev(v) for v in (x, res, w)]
    q, sf, h, rx, r = dg.sandwich_norm(t[0], t[1], None, None, t[2], quant_format=dg.QUANT_MXFP4)
    want = dg.add_rms_norm(t[0], t[1], t[2], quant_format=dg.QUANT_MXFP4)
    assert rx is None
    for a, b in zip((q, sf, h, r), want):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------- backward

def back_inputs(seed, m, k, gate_rows, post=True, with_dh=True):
    x, res, pw, gate, w = inputs(seed, m, k, gate_rows, post)
    f = [None if v is None else bf16_bits_to_f64(v) for v in (x, res, pw)]
    h, rx = X.sandwich_norm(*f, by_row(gate, gate_rows, m), 0.7, 1e-6)
    h = bf16_of_fp32(h)
    hv = bf16_bits_to_f64(h)
    r = (1.0 / np.sqrt(np.mean(hv * hv, axis=1) + 1e-6)).astype(np.float32)
    return bf(seed + 8, m, k, scale=1e-3), bf(seed + 9, m, k, scale=1e-3) if with_dh else None, x, h, pw, gate, w, rx.astype(np.float32), r


def run_back(dgm, a, gate_rows, scale, over=None):
    dy, dh, x, h, pw, gate, w, rx, r = a
    m, k = dy.shape
    t = [dev(v) for v in (dy, dh, x, h, pw, gate, w)]
    trx, tr = (torch.from_numpy(v.copy()).cuda() for v in (rx, r))
    (dx, c0), (dres, c1) = (guarded((m, k), torch.bfloat16) for _ in range(2))
    if over is not None:
        dx, dres = t[over[0]], t[over[1]]
    dw, c2 = guarded((k,), torch.float32)
    dpw, c3 = guarded((k,), torch.float32) if pw is not None else (None, lambda: None)
    dg, c4 = guarded((len(gate), k), torch.float32) if gate is not None else (None, lambda: None)
    ws, c5 = guarded((dgm.dg_sandwich_norm_backward_workspace_bytes(m, k, pw is not None, gate is not None),), torch.uint8)
    ws.fill_(255)
    dgm.dg_sandwich_norm_backward(t[0], t[1], t[2], t[3], t[4], t[5], t[6], trx if pw is not None else None, tr, dx, dres, dw,
                                  dpw, dg, ws, gate_rows or 1, scale)
    torch.cuda.synchronize()
    for c in (c0, c1, c2, c3, c4, c5):
        c()
    f = lambda t: None if t is None else t.cpu().numpy().astype(np.float64)   # noqa: E731
    return bf16_bits_to_f64(bits(dx)), bf16_bits_to_f64(bits(dres)), f(dw), f(dpw), f(dg)


def check_back(got, a, gate_rows, scale):
    dy, dh, x, h, pw, gate, w, rx, r = a
    m, k = dy.shape
    f = [None if v is None else bf16_bits_to_f64(v) for v in (dy, dh, x, h, pw, w)]
    dyv, dhv, xv, hv, pwv, wv = f
    gv = by_row(gate, gate_rows, m)
    rv, rxv = r.astype(np.float64), rx.astype(np.float64) if pw is not None else np.ones(m)
    s32 = float(np.float32(scale))
    d, dx, yn, vn, gn = X.sandwich_norm_backward(dyv, dhv, xv, hv, pwv, gv, wv, rxv, rv, s32)
    n, nx = np.abs(hv * rv[:, None]), np.abs(xv * rxv[:, None])
    an = np.abs(dyv * wv)
    mean = np.mean(an * n, axis=1, keepdims=True)
    ed = 8 * U * ((0 if dhv is None else np.abs(dhv)) + rv[:, None] * (an + n * mean)) + 64 * U * rv[:, None] * n * mean
    g1 = np.abs(s32 * (1 if gv is None else gv) * (1 if pwv is None else pwv)) * np.ones_like(d)
    eu, u = g1 * ed + 4 * U * g1 * np.abs(d), g1 * np.abs(d)
    edx = eu if pwv is None else rxv[:, None] * (eu + 8 * U * (u + nx * np.mean(u * nx, axis=1, keepdims=True))
                                                 + nx * np.mean((eu + 64 * U * u) * nx, axis=1, keepdims=True))
    tiny = 2.0 ** -133
    for name, v, ref, tol in (("dresidual", got[1], d, ed), ("dx", got[0], dx, edx)):
        bad = ~(np.abs(v - ref) <= 2.0 ** -8 * (np.abs(ref) + tol) + tol + tiny)
        assert not bad.any(), f"{name}: {bad.sum()} out of tolerance, first at {np.argwhere(bad)[0]}: {v[bad][0]} for {ref[bad][0]}"
    L = (m + 8) * U
    rows = lambda t: t.sum(axis=0)                                          # noqa: E731
    sums = [("dweight", got[2], rows(yn), L * rows(np.abs(yn)))]
    if pwv is not None:
        sums.append(("dpost_weight", got[3], rows(vn), L * rows(np.abs(vn)) + rows(np.abs(s32 * (1 if gv is None else gv)) * ed * nx)))
    if gv is not None:
        add = lambda t: np.add.reduceat(t, np.arange(0, m, gate_rows), axis=0)   # noqa: E731
        sums.append(("dgate", got[4], add(gn), L * add(np.abs(gn)) + add(np.abs(s32 * (1 if pwv is None else pwv)) * ed * nx)))
    for name, v, ref, tol in sums:
        bad = ~(np.abs(v - ref) <= tol + 2.0 ** -140)
        assert not bad.any(), f"{name}: {bad.sum()} out of tolerance, first at {np.argwhere(bad)[0]}: {v[bad][0]} for {ref[bad][0]} +- {tol[bad][0]}"


@pytest.mark.parametrize("m,k,gate_rows,post,with_dh", [
    (1, 128, 1, True, True), (3, 7168, 3, True, True), (130, 2048, 50, True, False), (33, 5120, 1, True, True),
    (2, 16384, 7, True, True), (300, 9216, 128, True, True), (1100, 384, 256, True, True), (1500, 512, 1, True, False),
    (2100, 2176, 9, True, True), (40, 640, 0, True, True), (40, 640, 0, False, True), (700, 1280, 37, False, False),
    (5000, 128, 4, True, True), (4100, 256, 1000, True, True)])
def test_sandwich_backward_shapes(dg, m, k, gate_rows, post, with_dh):
    a = back_inputs(m + k, m, k, gate_rows, post, with_dh)
    check_back(run_back(dg, a, gate_rows, 0.7), a, gate_rows, 0.7)


@pytest.mark.parametrize("over", [(0, 1), (1, 0), (2, 3), (3, 2), (0, 3)])
def test_sandwich_backward_in_place(dg, over):
    """dx and dresidual over two of dy, dh, x and h: the same results."""
    a = back_inputs(5, 300, 1280, 100)
    want, got = run_back(dg, a, 100, 0.7), run_back(dg, a, 100, 0.7, over)
    for w, g in zip(want, got):
        assert np.array_equal(w, g)


def test_sandwich_backward_edges(dg):
    """Zero rows of x and of dy, gates of zero, a scale of 0: gradients of zero where they are, finite everywhere."""
    a = list(back_inputs(7, 64, 512, 16))
    for i in (0, 1, 2):
        a[i][3] = 0
    a[0][5] = 0
    a[5][2] = 0
    a[7][3] = 1000.0                                           # 1 / sqrt(eps)
    check_back(run_back(dg, a, 16, 0.7), a, 16, 0.7)
    dx, dres, dw, dpw, dgate = run_back(dg, a, 16, 0.0)
    assert (dx == 0).all() and (dpw == 0).all() and (dgate == 0).all() and (dres != 0).any()


def test_sandwich_backward_repeats_bit_for_bit(dg):
    a = back_inputs(8, 1000, 1280, 130)
    want = run_back(dg, a, 130, 0.7)
    for _ in range(3):
        for w, g in zip(want, run_back(dg, a, 130, 0.7)):
            assert np.array_equal(w, g)


def test_sandwich_graph_and_streams(dg):
    """Forward and backward captured on a side stream; every replay, with eager work between, gives the eager results,
    and new inputs in the same buffers give theirs."""
    m, k, gr = 200, 1280, 70
    a = back_inputs(9, m, k, gr)
    _, res, _, _, _ = inputs(9, m, k, gr)
    dy, dh, x, _, pw, gate, w = [dev(v) for v in a[:7]]
    res = dev(res)
    ws = torch.empty(dg.dg_sandwich_norm_backward_workspace_bytes(m, k), dtype=torch.uint8, device="cuda")
    new = lambda *sh, dt=torch.float32: torch.empty(*sh, dtype=dt, device="cuda")   # noqa: E731
    h, q, sf, rx, r = new(m, k, dt=torch.bfloat16), new(m, k, dt=torch.uint8), new(k // 128, m), new(m), new(m)
    dx, dres, dw, dpw, dgate = new(m, k, dt=torch.bfloat16), new(m, k, dt=torch.bfloat16), new(k), new(k), new(-(-m // gr), k)
    outs = (h, q, sf, rx, r, dx, dres, dw, dpw, dgate)

    def both():
        dg.dg_sandwich_norm(x, res, pw, gate, w, h, q, sf, dg.QUANT_E4M3_F32, rx, r, gr, 0.7, 1e-6)
        dg.dg_sandwich_norm_backward(dy, dh, x, h, pw, gate, w, rx, r, dx, dres, dw, dpw, dgate, ws, gr, 0.7)

    both()
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        both()
    for rep in range(4):
        x.mul_(-0.5)
        both()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.view(torch.uint8).fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (t, v) in enumerate(zip(outs, want)):
            assert torch.equal(t.view(torch.uint8), v.view(torch.uint8)), f"replay {rep}, output {i}"
