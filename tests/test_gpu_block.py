"""The operators around a block's products in a row, as a model's layer runs them: norms with gate, gated projection,
quantisation, second projection, and the way back through all of them; once dense and once over experts.

Every product is quantised, so the results are compared twice: step by step with the oracle on the very operands that
the step read (the tolerances of each operator's own tests), and as a whole with the layer in float64 without any
quantisation, in the 2-norm.  E2M1 values are off by some 10 % of a block's size at random (steps of a sixth of its
largest value and more), a product of two quantised operands by 15 %, four products in a row, with what passes through
the norms and the activation between them, by less than 40 %.
"""

import numpy as np
import pytest
import torch

from oracle import mx as X
from oracle.formats import bf16_bits_to_f64
from tests.helpers import bits
from tests.test_gpu_linear import check as check_linear
from tests.test_gpu_linear import check_back as check_activation_back
from tests.test_gpu_norm import bf, check_norm, dev
from tests.test_gpu_sandwich import bf16_of_fp32, by_row, check_back as check_sandwich_back

pytestmark = pytest.mark.gpu

EPS, SCALE = 1e-6, 0.7


def f64(t):
    return bf16_bits_to_f64(bits(t))


def host(*ts):
    return [t.cpu().numpy() for t in ts]


def near(got, want, what, tol=0.4):
    off = np.linalg.norm(got - want) / np.linalg.norm(want)
    assert off < tol, f"{what}: {off:.3f} off the layer without quantisation"


def ffn64(xq, w1, b1, w2, res):
    u = xq @ w1.T + b1
    a = X.linear_epilogue(u, "silu", True)
    return u, a, a @ w2.T + (0 if res is None else res)


def test_feed_forward_block_and_its_way_back(dg):
    m, k, inter, gr = 300, 512, 384, 100
    x, res = bf(1, m, k, scale=2.0), bf(2, m, k)
    gate, pw, w = bf(3, 3, k), bf(4, k, scale=0.1), bf(5, k, scale=0.1)
    pw, w = (np.where(v & 0x8000, v ^ 0x8000, v) | 0x3f00 for v in (pw, w))            # about 0.5 .. 2
    pw, w = pw.astype(np.uint16), w.astype(np.uint16)
    w1, b1, w2 = bf(6, 2 * inter, k, scale=k ** -0.5), bf(7, 2 * inter, scale=0.1), bf(8, k, inter, scale=inter ** -0.5)
    t = dict(x=dev(x), res=dev(res), gate=dev(gate), pw=dev(pw), w=dev(w), b1=dev(b1))
    w1q, w1sf, w1qt, w1sft = dg.quantize_mxfp4(dev(w1), transposed=True)
    w2q, w2sf, w2qt, w2sft = dg.quantize_mxfp4(dev(w2), transposed=True)
    act = dg.ACT_SILU | dg.ACT_GATED

    # forward
    q, sf, h, rx, r = dg.sandwich_norm(t["x"], t["res"], t["pw"], t["gate"], t["w"], SCALE, gr, EPS, dg.QUANT_MXFP4)
    a, z = dg.mxfp4_linear(q, sf, w1q, w1sf, t["b1"], act, pre_activation=True)
    aq, asf, aqt, asft = dg.quantize_mxfp4(a, transposed=True)
    y = dg.mxfp4_linear(aq, asf, w2q, w2sf, None, dg.ACT_NONE, h)
    # back: dy arrives at y = h + ffn(norm(h)); the residual's share goes past the products
    dy = dev(bf(9, m, k, scale=1e-2))
    dyq, dysf, dyqt, dysft, _ = dg.activation_backward(dy, None, dg.ACT_NONE, bias=False)
    da, dw2 = dg.mxfp4_gemm_nt(dyq, dysf, w2qt, w2sft), dg.mxfp4_gemm_nt(dyqt, dysft, aqt, asft)
    zq, zsf, zqt, zsft, db1 = dg.activation_backward(da, z, act)
    dn = dg.mxfp4_gemm_nt(zq, zsf, w1qt, w1sft)
    n_bf = (h.float() * r[:, None] * t["w"].float()).bfloat16()
    nqt, nsft = dg.quantize_mxfp4(n_bf, transposed=True)[2:]
    dw1 = dg.mxfp4_gemm_nt(zqt, zsft, nqt, nsft)
    dx, dres, dw, dpw, dgate = dg.sandwich_norm_backward(dn, dy, t["x"], h, t["pw"], t["gate"], t["w"], rx, r, SCALE, gr)
    torch.cuda.synchronize()

    # step by step
    xv, rv, pwv, wv = (bf16_bits_to_f64(v) for v in (x, res, pw, w))
    gv = by_row(gate, gr, m)
    h64, rx64 = X.sandwich_norm(xv, rv, pwv, gv, SCALE, EPS)
    assert np.array_equal(bits(h), bf16_of_fp32(h64))
    check_norm((*host(q, sf), bits(h), r.cpu().numpy().astype(np.float64)), bits(h), None, w, 2, EPS)
    check_linear((bits(a), bits(z)), *host(q, sf, w1q, w1sf), b1, "silu", True, None)
    check_linear((bits(y), None), *host(aq, asf, w2q, w2sf), None, "none", False, bits(h))
    for got, want in zip((dyq, dysf, dyqt, dysft), dg.quantize_mxfp4(dy, transposed=True)):
        assert torch.equal(got, want)
    check_activation_back(dg, dict(dbias=db1), bits(da), bits(z), "silu", True)
    back = (bits(dn), bits(dy), x, bits(h), pw, gate, w, *host(rx, r))
    f = lambda v: v.cpu().numpy().astype(np.float64)                         # noqa: E731
    check_sandwich_back((f64(dx), f64(dres), f(dw), f(dpw), f(dgate)), back, gr, SCALE)

    # as a whole
    r64 = 1 / np.sqrt(np.mean(h64 * h64, axis=1) + EPS)
    n64 = h64 * r64[:, None] * wv
    w1v, w2v, b1v, dyv = (bf16_bits_to_f64(v) for v in (w1, w2, b1, bits(dy)))
    u64, a64, y64 = ffn64(n64, w1v, b1v, w2v, h64)
    dz64 = X.linear_epilogue_backward(dyv @ w2v, u64, "silu", True)
    dn64 = dz64 @ w1v
    d64, dx64, yn, vn, gn = X.sandwich_norm_backward(dn64, dyv, xv, h64, pwv, gv, wv, rx64, r64, SCALE)
    near(f64(y), y64, "y", 0.25)
    for name, got, want in (("dw2", f64(dw2), dyv.T @ a64), ("dw1", f64(dw1), dz64.T @ n64), ("db1", f(db1), dz64.sum(axis=0)),
                            ("dx", f64(dx), dx64), ("dresidual", f64(dres), d64), ("dweight", f(dw), yn.sum(axis=0)),
                            ("dpost_weight", f(dpw), vn.sum(axis=0)), ("dgate", f(dgate), np.add.reduceat(gn, [0, 100, 200]))):
        near(got, want, name)


def test_expert_layer_and_its_way_back(dg):
    """Rows sorted by expert, both projections over the experts with the gated activation between them, and every
    gradient."""
    ms, k, inter = [130, 0, 37, 200, 1], 256, 256
    m, G = sum(ms), len(ms)
    x, w1, w2 = bf(1, m, k), bf(2, G, 2 * inter, k, scale=k ** -0.5), bf(3, G, k, inter, scale=inter ** -0.5)
    dy = bf(4, m, k, scale=1e-2)
    tms = torch.tensor(ms, dtype=torch.int32, device="cuda")
    w1q, w1sf, w1qt, w1sft = dg.quantize_mxfp4(dev(w1), transposed=True)
    w2q, w2sf, w2qt, w2sft = dg.quantize_mxfp4(dev(w2), transposed=True)
    xq, xsf, xqt, xsft = dg.quantize_mxfp4_ragged(dev(x), tms)
    z = dg.m_grouped_mxfp4_gemm_nt_ragged(xq, xsf, w1q, w1sf, tms)
    zf = z.float()
    a = (zf[:, :inter] * torch.sigmoid(zf[:, :inter]) * zf[:, inter:]).bfloat16()
    aq, asf, aqt, asft = dg.quantize_mxfp4_ragged(a, tms)
    y = dg.m_grouped_mxfp4_gemm_nt_ragged(aq, asf, w2q, w2sf, tms)
    dyq, dysf, dyqt, dysft = dg.quantize_mxfp4_ragged(dev(dy), tms)
    da = dg.m_grouped_mxfp4_gemm_nt_ragged(dyq, dysf, w2qt, w2sft, tms)
    dw2 = dg.k_grouped_mxfp4_gemm_nt_ragged(dyqt, dysft, aqt, asft, tms)
    dz = torch.empty_like(z)
    dg.dg_activation_backward(da, z, dg.ACT_SILU | dg.ACT_GATED, dz)
    zq, zsf, zqt, zsft = dg.quantize_mxfp4_ragged(dz, tms)
    dx = dg.m_grouped_mxfp4_gemm_nt_ragged(zq, zsf, w1qt, w1sft, tms)
    dw1 = dg.k_grouped_mxfp4_gemm_nt_ragged(zqt, zsft, xqt, xsft, tms)
    torch.cuda.synchronize()
    xv, w1v, w2v, dyv = (bf16_bits_to_f64(v) for v in (x, w1, w2, dy))
    for g, (s, e) in enumerate(X.group_rows(ms, m)):
        if s == e:
            assert (f64(dw1)[g] == 0).all() and (f64(dw2)[g] == 0).all()
            continue
        u, a64, y64 = ffn64(xv[s:e], w1v[g], 0.0, w2v[g], None)
        dz64 = X.linear_epilogue_backward(dyv[s:e] @ w2v[g], u, "silu", True)
        for name, got, want in (("y", f64(y)[s:e], y64), ("dx", f64(dx)[s:e], dz64 @ w1v[g]), ("dw1", f64(dw1)[g], dz64.T @ xv[s:e]),
                                ("dw2", f64(dw2)[g], dyv[s:e].T @ a64)):
            near(got, want, f"{name} of group {g}")
