"""The activations' slopes in full, and a linear layer's gradients against the oracle's products of the very operands.

The slopes are read in fp32, before their rounding to bf16: dbias of a single row is that row of dz.  For u <= 0 a slope is
s + u s (1 - s) w' (sigmoid forms, s = 1 / (1 + exp(-w))) or Phi + u phi (erf), whose terms keep relative accuracy however
small they are: with e = 2^-23 the exponential's argument is off by five roundings of 2^-24 at most, 3 |w| e of the
terms, its value, reciprocal, approximation (4.7e-7, 4 e) and products by less than 24 e; below 2^-118 (an exponential past
fp32's range, times up to 100) they may be 0.  Likewise act(u) itself, which a gated layer's other half is scaled by."""

import numpy as np
import pytest
from scipy.special import ndtr

from oracle import mx as X
from oracle.formats import bf16_bits_to_f64
from tests.helpers import bits
from tests.test_gpu_linear import ACTS, E, GATED, exponent
from tests.test_gpu_norm import bf, dev

pytestmark = pytest.mark.gpu

NEGATIVE = np.arange(0x8000, 0xff80, dtype=np.uint16)   # every finite bf16 u <= 0: 255 * 128 of them


def terms(u, act):
    """Of act'(u): the sum of its two terms' magnitudes."""
    if act == "gelu":
        return ndtr(u) + np.abs(u) * np.exp(-np.minimum(u * u / 2, 700.0)) / np.sqrt(2 * np.pi)
    c = np.sqrt(2 / np.pi)
    dw = 1.0 if act == "silu" else 2 * c * (1 + 3 * 0.044715 * u ** 2)
    w = np.abs(u) if act == "silu" else 2 * c * np.abs(u + 0.044715 * u ** 3)
    s = 1 / (1 + np.exp(np.minimum(w, 700.0)))
    return s + np.abs(u) * s * (1 - s) * dw


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_slopes_of_the_negative_tail(dg, act):
    u = bf16_bits_to_f64(NEGATIVE)
    rel = (24 + 3 * np.minimum(exponent(u, act), 200.0)) * E
    one = dev(np.full((1, len(u)), 0x3f80, np.uint16))
    z = NEGATIVE[None]
    got = dg.activation_backward(one, dev(z), ACTS[act])[4].cpu().numpy().astype(np.float64)
    y, d = X.activation(u, act)
    off = np.abs(got - d) - (rel * terms(u, act) + 2.0 ** -118)
    assert (off <= 0).all(), f"slope of {u[off.argmax()]}: {got[off.argmax()]} for {d[off.argmax()]}"
    # gated: the gate's slope by an up of 1, and act(gate) for the other half
    got = dg.activation_backward(one, dev(np.hstack([z, np.full_like(z, 0x3f80)])), ACTS[act] | GATED)[4]
    got = got.cpu().numpy().astype(np.float64)
    n = len(u)
    assert (np.abs(got[:n] - d) <= rel * terms(u, act) + 2.0 ** -118).all()
    off = np.abs(got[n:] - y) - (rel * np.abs(y) + 2.0 ** -118)
    assert (off <= 0).all(), f"{act} of {u[off.argmax()]}: {got[n:][off.argmax()]} for {y[off.argmax()]}"


@pytest.mark.parametrize("act,gated", [("none", False), ("relu", True), ("silu", True), ("gelu", False), ("gelu_tanh", True)])
@pytest.mark.parametrize("m,n,k", [(1, 256, 128), (200, 512, 384), (333, 768, 640)])
def test_gradients_are_the_products_of_their_operands(dg, m, n, k, act, gated):
    """dx = q(dz) . qt(w)^T and dw = qt(dz) . qt(x)^T, each within the GEMM's bound of the oracle's product (tests/
    test_gpu_mxfp4.py: 2^-8 of the value and (K/8 + 1) e (1 + 2^-8) of the sum of magnitudes)."""
    x, w, bias, dy = bf(1, m, k), bf(2, n, k, scale=k ** -0.5), bf(3, n, scale=0.1), bf(4, m, n // 2 if gated else n, scale=1e-2)
    xq, xsf, xqt, xsft = dg.quantize_mxfp4(dev(x), transposed=True)
    wq, wsf, wqt, wsft = dg.quantize_mxfp4(dev(w), transposed=True)
    code = ACTS[act] | (GATED if gated else 0)
    z = dg.mxfp4_linear(xq, xsf, wq, wsf, dev(bias), code, pre_activation=True)[1]
    q, sf, qt, sft, _ = dg.activation_backward(dev(dy), z, code)
    for a, a_sf, b, b_sf in ((q, sf, wqt, wsft), (qt, sft, xqt, xsft)):
        got = bf16_bits_to_f64(bits(dg.mxfp4_gemm_nt(a, a_sf, b, b_sf)))
        av, bv = X.dequant_mxfp4(a.cpu().numpy(), a_sf.cpu().numpy()), X.dequant_mxfp4(b.cpu().numpy(), b_sf.cpu().numpy())
        ref, s = av @ bv.T, np.abs(av) @ np.abs(bv).T
        tol = 2.0 ** -8 * np.abs(ref) + (av.shape[1] / 8 + 1) * E * (1 + 2.0 ** -8) * s
        assert got.shape == ref.shape and (np.abs(got - ref) <= tol).all()
    # the operands are those of dz by the formula: E2M1 leaves some 10 % of them (steps of a sixth of a block's largest)
    ref = X.linear_epilogue_backward(bf16_bits_to_f64(dy), bf16_bits_to_f64(bits(z)), act, gated)
    for v in (X.dequant_mxfp4(q.cpu().numpy(), sf.cpu().numpy()), X.dequant_mxfp4(qt.cpu().numpy(), sft.cpu().numpy())[:, :m].T):
        assert np.linalg.norm(v - ref) < 0.2 * np.linalg.norm(ref)


@pytest.mark.parametrize("act,want", [("none", 1.0), ("relu", 0.0), ("silu", np.nan), ("gelu", np.nan), ("gelu_tanh", np.nan)])
def test_slopes_of_a_nan(dg, act, want):
    """As include/dg.h has them; a gated layer's other half takes act(NaN), which is a NaN in all of them."""
    z = bf(1, 1, 512)
    z[0, 7] = 0x7fc0
    z[0, 256:] = 0x3f80
    one = np.full((1, 256), 0x3f80, np.uint16)
    got = dg.activation_backward(dev(one), dev(z[:, :256].copy()), ACTS[act])[4].cpu().numpy()
    assert np.array_equal(got[7], want, equal_nan=True) and np.isfinite(np.delete(got, 7)).all()
    got = dg.activation_backward(dev(one), dev(z), ACTS[act] | GATED)[4].cpu().numpy()
    assert np.array_equal(got[7], want, equal_nan=True) and np.isnan(got[256 + 7])
    assert np.isfinite(np.delete(got, (7, 256 + 7))).all()
