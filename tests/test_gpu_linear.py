"""The MXFP4 linear layer (bias, activation, residual) and its activation's backward pass, against the float64 oracle.

Tolerances, e = 2^-23.  u is the GEMM's sum with one addition more (the bias): tests/test_gpu_mxfp4.py derives
Eu = (K/8 + 2) e (1 + 2^-8) S, S = sum |a b| + |bias|; z adds its rounding, 2^-8 |u|.  The activations are off by their
slope (at most 1.13) times Eu and by their own evaluation: an exponential whose argument w (u^2 / 2 for the erf form) is
rounded twice, an approximation of 4 e at most and some ten roundings, together (16 + 2 |w|) e of the value; below 2^-120
(an exponential past fp32's range) they may be 0.  Slopes likewise, of the sum of their terms' magnitudes.  The products
and sums behind them add 4 e of their terms, bf16 outputs 2^-8 of the value.
"""

import numpy as np
import pytest
import torch

from oracle import mx as X
from oracle.formats import bf16_bits_to_f64, f64_to_bf16_bits
from tests.helpers import bits, check_bit_exact
from tests.test_gpu_mxfp4 import SHAPES, guarded, rand_mx
from tests.test_gpu_norm import bf, dev

pytestmark = pytest.mark.gpu

E = 2.0 ** -23
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
GATED = 16


def exponent(u, act):
    """|w|, the exponential's argument."""
    if act in ("none", "relu"):
        return np.zeros_like(u)
    w = u * u / 2 if act == "gelu" else np.abs(u) if act == "silu" else 1.6 * np.abs(u + 0.044715 * u ** 3)
    return np.minimum(w, 200.0)


def run(dgm, a, sa, b, sb, bias, act, gated, res, want_z, over_residual=False):
    m, n = a.shape[0], b.shape[0]
    t = [torch.from_numpy(v).cuda() for v in (a, sa, b, sb)]
    out = (m, n // 2 if gated else n)
    d, c0 = guarded(out, torch.bfloat16)
    z, c1 = guarded((m, n), torch.bfloat16) if want_z else (None, lambda: None)
    r = dev(res)
    if over_residual:
        d = r
    dgm.dg_mxfp4_linear(*t, dev(bias), ACTS[act] | (GATED if gated else 0), r, z, d)
    torch.cuda.synchronize()
    c0()
    c1()
    return bits(d), None if z is None else bits(z)


def check(got, a, sa, b, sb, bias, act, gated, res):
    k = 2 * a.shape[1]
    av, bv = X.dequant_mxfp4(a, sa), X.dequant_mxfp4(b, sb)
    u, s = av @ bv.T, np.abs(av) @ np.abs(bv).T
    if bias is not None:
        u, s = u + bf16_bits_to_f64(bias), s + np.abs(bf16_bits_to_f64(bias))
    eu = (k / 8 + 2) * E * (1 + 2.0 ** -8) * s
    half = u.shape[1] // 2
    g, eg = (u[:, :half], eu[:, :half]) if gated else (u, eu)
    y = X.activation(g, act)[0]
    ey = 1.13 * eg + (16 + 2 * exponent(g, act)) * E * np.abs(y) + 2.0 ** -120
    if gated:
        up, eup = u[:, half:], eu[:, half:]
        y, ey = y * up, ey * (np.abs(up) + eup) + np.abs(y) * eup + 4 * E * np.abs(y * up)
    ref = y
    if res is not None:
        ref = y + bf16_bits_to_f64(res)
        ey = ey + 4 * E * (np.abs(y) + np.abs(bf16_bits_to_f64(res)))
    for name, v, r, e in (("d", got[0], ref, ey), ("z", got[1], u, eu)):
        if v is None:
            continue
        v = bf16_bits_to_f64(v)
        bad = ~(np.abs(v - r) <= 2.0 ** -8 * (np.abs(r) + e) + e)
        assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} out of tolerance, first at {np.argwhere(bad)[0]}: " \
                              f"{v[bad][0]} against {r[bad][0]} +- {e[bad][0]}"


def case(seed, m, n, k, with_bias, with_res, gated):
    rng = np.random.default_rng(seed)
    a, sa = rand_mx(rng, m, k, -5, 1)
    b, sb = rand_mx(rng, n, k, -6, 0)
    bias = bf(seed + 1, n) if with_bias else None
    return a, sa, b, sb, bias, bf(seed + 2, m, n // 2 if gated else n, scale=2.0) if with_res else None


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_linear_shapes(dg, m, n, k, gated):
    if gated:
        n = (n + 31) // 32 * 32
    i = m + n // 16 + k // 128
    act = list(ACTS)[i % 5]
    a, sa, b, sb, bias, res = case(i, m, n, k, i % 3 != 0, i % 2 == 0, gated)
    check(run(dg, a, sa, b, sb, bias, act, gated, res, i % 4 < 2), a, sa, b, sb, bias, act, gated, res)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("m", [5, 20, 150])
def test_linear_activations(dg, m, act, gated):
    a, sa, b, sb, bias, res = case(m, m, 288, 512, True, True, gated)
    got = run(dg, a, sa, b, sb, bias, act, gated, res, True)
    check(got, a, sa, b, sb, bias, act, gated, res)
    # the same without z, and over the residual
    again, _ = run(dg, a, sa, b, sb, bias, act, gated, res, False)
    over, _ = run(dg, a, sa, b, sb, bias, act, gated, res, True, over_residual=True)
    assert np.array_equal(again, got[0]) and np.array_equal(over, got[0])


def integers(seed, m, n, k):
    rng = np.random.default_rng(seed)
    ints = np.array([0, 2, 4, 6, 10, 12], dtype=np.uint8)                # 0, 1, 2, 4, -1, -2
    a, b = (X.pack_pairs(ints[rng.integers(0, 6, (r, k))]) for r in (m, n))
    sa, sb = (np.ascontiguousarray(X.pack_words((127 + rng.integers(0, 2, (r, k // 32))).astype(np.uint8)).T) for r in (m, n))
    return a, sa, b, sb, f64_to_bf16_bits(rng.integers(-100, 101, n).astype(np.float64)), rng


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kernel", [0, 1, 2, 3, 4, 5, 6, 7, 100, 101])
def test_linear_every_kernel(dg, kernel, gated, monkeypatch):
    """Each tile and each form for few rows pinned, over partial tiles, odd counts of K blocks, a split along K and (with
    the CU cap) several tiles per workgroup: integers whose sums, products and results are exact, so that d and z are the
    oracle's bf16 roundings bit for bit."""
    monkeypatch.setenv("DG_FORCE_MXFP4", str(kernel))
    rows = {100: (1, 16), 101: (17, 32)}.get(kernel, (1, 70, 200, 300))
    for m in rows:
        for n, k, cap in ((288, 128, 0), (544, 2176, 0), (416, 1152, 8)):
            dg.dg_set_num_cus(cap)
            try:
                a, sa, b, sb, bias, rng = integers(m + n, m, n, k)
                res = f64_to_bf16_bits(rng.integers(-100, 101, (m, n // 2 if gated else n)).astype(np.float64))
                u = X.mxfp4_gemm_nt(a, sa, b, sb) + bf16_bits_to_f64(bias)
                for act in ("none", "relu"):
                    d, z = run(dg, a, sa, b, sb, bias, act, gated, res, True)
                    check_bit_exact(z, u, f"z {m} {n} {k} {act}")
                    check_bit_exact(d, X.linear_epilogue(u, act, gated, bf16_bits_to_f64(res)), f"d {m} {n} {k} {act}")
            finally:
                dg.dg_set_num_cus(0)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m", [3, 150])
def test_linear_without_an_epilogue_is_the_gemm(dg, m, gated):
    """No bias, activation and residual: the GEMM's d (gated: z) bit for bit."""
    a, sa, b, sb, _, _ = case(7, m, 544, 1152, False, False, gated)
    t = [torch.from_numpy(v).cuda() for v in (a, sa, b, sb)]
    want = dg.mxfp4_gemm_nt(*t)
    if gated:
        _, got = dg.mxfp4_linear(*t, activation=dg.ACT_GATED, pre_activation=True)
    else:
        got = dg.mxfp4_linear(*t)
    assert torch.equal(got, want)


def test_linear_nonfinite(dg):
    """A NaN scale makes its row NaN, an infinite bias its column what the activation makes of it; no other place."""
    m, n, k = 40, 96, 256
    a, sa, b, sb, bias, _ = case(3, m, n, k, True, False, False)
    sa.view(np.uint8).reshape(k // 128, m, 4)[1, 7, 2] = 255
    a[7, 96:112] = 0
    bias[5], bias[6] = 0x7f80, 0xff80
    for act, plus, minus in (("none", np.inf, -np.inf), ("relu", np.inf, 0.0), ("silu", np.inf, np.nan), ("gelu", np.inf, np.nan),
                             ("gelu_tanh", np.inf, np.nan)):
        d, z = (bf16_bits_to_f64(v) for v in run(dg, a, sa, b, sb, bias, act, False, None, True))
        rest = np.delete(d, 7, axis=0)
        assert np.isnan(d[7]).all() and np.isnan(z[7]).all(), act
        assert np.array_equal(rest[:, 5], np.full(m - 1, plus), equal_nan=True), act
        assert np.array_equal(rest[:, 6], np.full(m - 1, minus), equal_nan=True), act
        assert np.isfinite(np.delete(rest, (5, 6), axis=1)).all(), act


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_linear_activation_over_its_range(dg, act):
    """u = bias alone, over every magnitude and sign of bf16: the activation itself."""
    n = 65280 // 16 * 16
    pats = np.arange(0x7f80, dtype=np.uint16)
    bias = np.concatenate([pats, pats | 0x8000])[:n]
    n = len(bias)
    a, sa = np.zeros((2, 64), np.uint8), np.full((1, 2), 0x7f7f7f7f, np.int32)
    b, sb = np.zeros((n, 64), np.uint8), np.full((1, n), 0x7f7f7f7f, np.int32)
    check(run(dg, a, sa, b, sb, bias, act, False, None, True), a, sa, b, sb, bias, act, False, None)


# ---------------------------------------------------------------------------- backward

def run_back(dgm, dy, z, act, gated, want=("dz", "rows", "cols", "bias"), inplace=None):
    m, n = (dy if z is None else z).shape
    mb = (m + 127) // 128
    ty, tz = dev(dy), dev(z)
    outs = dict(dz=((m, n), torch.bfloat16, "dz"), q=((m, n // 2), torch.uint8, "rows"), sf=((n // 128, m), torch.int32, "rows"),
                qt=((n, mb * 64), torch.uint8, "cols"), sft=((mb, n), torch.int32, "cols"), dbias=((n,), torch.float32, "bias"))
    made = {k: guarded(*v[:2]) for k, v in outs.items() if v[2] in want}
    t = {k: v[0] for k, v in made.items()}
    if inplace:
        t["dz"] = dict(z=tz, dy=ty)[inplace]
    nbytes = dgm.dg_activation_backward_workspace_bytes(m, n)
    ws, cw = guarded((nbytes,), torch.uint8) if nbytes else (None, lambda: None)
    dgm.dg_activation_backward(ty, tz, ACTS[act] | (GATED if gated else 0), **t, workspace=ws)
    torch.cuda.synchronize()
    cw()
    for _, c in made.values():
        c()
    return t


def check_back(dgm, got, dy, z, act, gated):
    dyv = bf16_bits_to_f64(dy)
    zv = bf16_bits_to_f64(z) if z is not None else np.zeros_like(dyv)
    ref = X.linear_epilogue_backward(dyv, zv, act, gated)
    half = zv.shape[1] // 2
    g = zv[:, :half] if gated else zv
    y, d = X.activation(g, act)
    _, pos = X.activation(np.abs(g), act)                               # s (or Phi) and the slope's other term, added up
    w = exponent(g, act)
    terms = np.abs(pos) + 2 * np.minimum(np.abs(g) * np.exp(-w) * (1 + g * g), 2.0) + 1
    # (the exponent's error counts in what the exponential scales: 2 |w| exp(-|w|) times it is below 8 everywhere)
    ed = E * (16 * np.minimum(terms * np.ones_like(g), 6.0) + 8) if act not in ("none", "relu") else np.zeros_like(g)
    ey = (16 + 2 * w) * E * np.abs(y) + 2.0 ** -120
    if gated:
        up = zv[:, half:]
        e = np.hstack([np.abs(dyv * up) * ed, np.abs(dyv) * ey]) + 4 * E * np.abs(ref)
    else:
        e = np.abs(dyv) * ed + 4 * E * np.abs(ref)
    if "dz" in got:
        v = bf16_bits_to_f64(bits(got["dz"]))
        bad = ~(np.abs(v - ref) <= 2.0 ** -8 * (np.abs(ref) + e) + e + 2.0 ** -133)
        assert not bad.any(), f"dz: {bad.sum()} out of tolerance, first at {np.argwhere(bad)[0]}: {v[bad][0]} for {ref[bad][0]} +- {e[bad][0]}"
        q, sf, qt, sft = dgm.quantize_mxfp4(got["dz"].view(torch.bfloat16), transposed=True)
        for name, t in dict(q=q, sf=sf, qt=qt, sft=sft).items():
            if name in got:
                assert torch.equal(got[name], t), name
    if "dbias" in got:
        m = len(ref)
        v = got["dbias"].cpu().numpy().astype(np.float64)
        tol = e.sum(axis=0) + (8 + 16 + (m + 127) // 128 + 4) * 2.0 ** -24 * np.abs(ref).sum(axis=0) + 2.0 ** -140
        bad = ~(np.abs(v - ref.sum(axis=0)) <= tol)
        assert not bad.any(), f"dbias: {bad.sum()} out of tolerance, first at {np.argwhere(bad)[0]}"


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("m,n", [(1, 256), (130, 512), (300, 1280)])
def test_backward_shapes(dg, m, n, act, gated):
    dy, z = bf(m, m, n // 2 if gated else n, scale=1e-2), bf(m + 1, m, n, scale=2.0)
    check_back(dg, run_back(dg, dy, z, act, gated), dy, z, act, gated)


@pytest.mark.parametrize("m,n", [(128, 128), (127, 384), (1000, 128), (5000, 256), (40000, 128)])
def test_backward_sizes(dg, m, n):
    dy, z = bf(m, m, n, scale=1e-2), bf(m + 1, m, n, scale=2.0)
    check_back(dg, run_back(dg, dy, z, "silu", False), dy, z, "silu", False)


@pytest.mark.parametrize("want", [("dz",), ("rows",), ("cols",), ("bias",), ("dz", "rows"), ("dz", "cols", "bias"), ("rows", "bias"),
                                  ("rows", "cols")])
def test_backward_output_sets(dg, want):
    """Any set of outputs is what all of them together are."""
    dy, z = bf(1, 200, 256, scale=1e-2), bf(2, 200, 512, scale=2.0)
    every = run_back(dg, dy, z, "gelu", True)
    for name, t in run_back(dg, dy, z, "gelu", True, want).items():
        assert torch.equal(t.view(torch.uint8), every[name].view(torch.uint8)), name


def test_backward_without_z(dg):
    dy = bf(3, 140, 256)
    got = run_back(dg, dy, None, "none", False)
    assert np.array_equal(bits(got["dz"]), dy)
    check_back(dg, got, dy, None, "none", False)


@pytest.mark.parametrize("inplace,gated", [("z", False), ("z", True), ("dy", False)])
def test_backward_in_place(dg, inplace, gated):
    dy, z = bf(1, 200, 256 if gated else 512, scale=1e-2), bf(2, 200, 512, scale=2.0)
    want = run_back(dg, dy, z, "silu", gated)
    got = run_back(dg, dy, z, "silu", gated, ("rows", "cols", "bias"), inplace)
    for name, t in got.items():
        assert torch.equal(t.view(torch.uint8), want[name].view(torch.uint8)), name


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
def test_backward_over_the_range_of_z(dg, act):
    """Every magnitude and sign of bf16 (its infinities and NaN: dz is NaN or finite, and no other place is touched)."""
    pats = np.arange(0x8000, dtype=np.uint16)
    z = np.concatenate([pats, pats | 0x8000]).reshape(-1, 256)
    dy = np.full_like(z, 0x3f80)
    finite = np.isfinite(bf16_bits_to_f64(z))
    got = run_back(dg, dy, z, act, False, ("dz",))
    v = bf16_bits_to_f64(bits(got["dz"]))
    assert np.isfinite(v[finite]).all()
    if act != "relu":
        assert np.isnan(v[np.isnan(bf16_bits_to_f64(z))]).all()
    zf = np.where(finite, z, 0).astype(np.uint16)
    check_back(dg, run_back(dg, dy, zf, act, False, ("dz",)), dy, zf, act, False)


def test_backward_repeats_bit_for_bit(dg):
    dy, z = bf(1, 3000, 256, scale=1e-2), bf(2, 3000, 512, scale=2.0)
    want = run_back(dg, dy, z, "silu", True)
    for _ in range(3):
        for name, t in run_back(dg, dy, z, "silu", True).items():
            assert torch.equal(t.view(torch.uint8), want[name].view(torch.uint8)), name


def test_training_step_gradients(dg):
    """Forward, activation_backward and the two products together: dx and dw against the oracle's products of the same
    operands, and a linear layer's bias gradient."""
    m, n, k = 200, 512, 384
    x, w, bias, dy = bf(1, m, k), bf(2, n, k, scale=k ** -0.5), bf(3, n, scale=0.1), bf(4, m, n // 2, scale=1e-2)
    tx, tw = dev(x), dev(w)
    xq, xsf, xqt, xsft = dg.quantize_mxfp4(tx, transposed=True)
    wq, wsf, wqt, wsft = dg.quantize_mxfp4(tw, transposed=True)
    act = dg.ACT_SILU | dg.ACT_GATED
    y, z = dg.mxfp4_linear(xq, xsf, wq, wsf, dev(bias), act, pre_activation=True)
    q, sf, qt, sft, dbias = dg.activation_backward(dev(dy), z, act)
    dx, dw = dg.mxfp4_gemm_nt(q, sf, wqt, wsft), dg.mxfp4_gemm_nt(qt, sft, xqt, xsft)
    torch.cuda.synchronize()
    c = lambda t: t.cpu().numpy()                                           # noqa: E731
    check((bits(y), bits(z)), c(xq), c(xsf), c(wq), c(wsf), bias, "silu", True, None)
    check_back(dg, dict(dbias=dbias), dy, bits(z), "silu", True)
    dz = X.linear_epilogue_backward(bf16_bits_to_f64(dy), bf16_bits_to_f64(bits(z)), "silu", True)
    for got, a, b, ref in ((dx, (q, sf), (wqt, wsft), dz @ bf16_bits_to_f64(w)), (dw, (qt, sft), (xqt, xsft), dz.T @ bf16_bits_to_f64(x))):
        assert np.array_equal(bits(got), bits(dg.mxfp4_gemm_nt(*a, *b)))
        v = bf16_bits_to_f64(bits(got))
        # E2M1 steps are a sixth of the block's largest value at most: an operand is off by some 10 % of itself at
        # random, their product's sum by 15 % of its size
        assert np.linalg.norm(v - ref) < 0.25 * np.linalg.norm(ref)


@pytest.mark.parametrize("m,n,k", [(70, 288, 4096), (300, 544, 1152), (20, 96, 512)])
def test_graph_replays_match_eager(dg, m, n, k):
    """Forward (a plan with partial tiles among them) and backward captured on a side stream: every replay on new inputs,
    with eager calls between that use workspaces of their own, gives the eager results."""
    n = n // 32 * 32
    a, sa, b, sb, bias, _ = case(m, m, n, k, True, False, True)
    ta, tsa, tb, tsb = (torch.from_numpy(v).cuda() for v in (a, sa, b, sb))
    nb = (n + 255) // 256 * 256                                       # the backward pass's columns
    zb, dy = dev(bf(1, m, nb, scale=2.0)), dev(bf(2, m, nb // 2))
    tbias, res = dev(bias), dev(bf(3, m, n // 2))
    new = lambda *sh, dt=torch.bfloat16: torch.empty(*sh, dtype=dt, device="cuda")   # noqa: E731
    ws = new(max(1, dg.dg_mxfp4_gemm_workspace_bytes(m, n, k)), dt=torch.uint8)
    ws2 = new(max(1, dg.dg_activation_backward_workspace_bytes(m, nb)), dt=torch.uint8)
    mb = (m + 127) // 128
    d, z = new(m, n // 2), new(m, n)
    q, sf, qt, sft, dbias = (new(m, nb // 2, dt=torch.uint8), new(nb // 128, m, dt=torch.int32), new(nb, mb * 64, dt=torch.uint8),
                             new(mb, nb, dt=torch.int32), new(nb, dt=torch.float32))
    outs = (d, z, q, sf, qt, sft, dbias)
    act = dg.ACT_GELU_TANH | dg.ACT_GATED

    def step():
        dg.dg_mxfp4_linear(ta, tsa, tb, tsb, tbias, act, res, z, d, ws)
        dg.dg_activation_backward(dy, zb, act, None, q, sf, qt, sft, dbias, ws2)

    step()
    torch.cuda.synchronize()
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for rep in range(4):
        ta.copy_(torch.from_numpy(np.roll(a, rep + 1, axis=0)))
        dy.mul_(-0.5)
        want_d, want_z = dg.mxfp4_linear(ta, tsa, tb, tsb, tbias, act, res, pre_activation=True)
        want = (want_d, want_z, *dg.activation_backward(dy, zb, act))
        for t in outs:
            t.view(torch.uint8).fill_(255)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (t, v) in enumerate(zip(outs, want)):
            assert torch.equal(t.view(torch.uint8), v.view(torch.uint8)), f"replay {rep}, output {i}"


def test_calls_on_two_streams(dg):
    """Calls in flight together on two streams, each with the workspace that the wrapper makes: what they give alone."""
    sets = []
    for seed, (m, n, k) in enumerate([(70, 544, 4096), (300, 1088, 1152)]):
        a, sa, b, sb, bias, _ = case(seed, m, n, k, True, False, True)
        t = [torch.from_numpy(v).cuda() for v in (a, sa, b, sb)] + [dev(bias), dg.ACT_SILU | dg.ACT_GATED]
        zb, dy = dev(bf(seed, m, 512)), dev(bf(seed + 9, m, 256))
        call = lambda t=t, zb=zb, dy=dy: (dg.mxfp4_linear(*t), *dg.activation_backward(dy, zb, dg.ACT_GELU | dg.ACT_GATED))   # noqa: E731
        sets.append((call, call()))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [[], []]
    for _ in range(8):
        for i, (call, _) in enumerate(sets):
            with torch.cuda.stream(streams[i]):
                got[i].append(call())
    torch.cuda.synchronize()
    for (_, want), many in zip(sets, got):
        for one in many:
            assert all(torch.equal(w.view(torch.uint8), g.view(torch.uint8)) for w, g in zip(want, one))
