"""Host-side checks of the operators around a block's products: every refusal comes before any HIP call, and the
binding checks its tensors (no compute is launched; these tests run without a GPU).  The oracle's gradients are held to
differences of its forward formulas here, too."""

import numpy as np
import pytest
import torch

import fp4_gemm_dense_amd as dgm
from oracle import mx as X

A = 0x10000      # a fake aligned address, never dereferenced on the host
OK = (0, 4)      # passed validation; without a gfx950 device the call stops at the device check
NAN, INF = float("nan"), float("inf")

no_gpu = pytest.mark.skipif(torch.cuda.is_available(), reason="fake addresses: only where no GPU is visible")


def expect(got, status):
    assert got in status if isinstance(status, tuple) else got == status


@no_gpu
@pytest.mark.parametrize("change,status", [
    ({}, OK), (dict(post_weight=0), OK), (dict(gate=0, gate_rows=0), OK), (dict(rstd_x=0, rstd=0), OK), (dict(fmt=2), OK),
    (dict(gate_rows=1 << 30), OK), (dict(scale=0.0), OK), (dict(scale=-3.0), OK), (dict(k=32768), OK),
    (dict(x=0), 1), (dict(residual=0), 1), (dict(weight=0), 1), (dict(h=0), 1), (dict(q=0), 1), (dict(sf=0), 1),
    (dict(fmt=3), 1), (dict(m=0), 1), (dict(k=0), 1), (dict(gate_rows=0), 1), (dict(gate_rows=-1), 1),
    (dict(scale=NAN), 1), (dict(scale=INF), 1), (dict(eps=0.0), 1), (dict(eps=NAN), 1),
    (dict(x=A + 8), 1), (dict(residual=A + 8), 1), (dict(post_weight=A + 8), 1), (dict(gate=A + 8), 1),
    (dict(weight=A + 8), 1), (dict(h=A + 8), 1), (dict(q=A + 8), 1), (dict(sf=A + 2), 1), (dict(rstd_x=A + 2), 1),
    (dict(rstd=A + 2), 1), (dict(k=192), 2), (dict(k=32768 + 128), 2), (dict(m=1 << 26, k=128), 2),
])
def test_sandwich_norm_refusals(change, status):
    v = dict(x=A, residual=A, post_weight=A, gate=A, weight=A, h=A, q=A, sf=A, fmt=0, rstd_x=A, rstd=A, m=8, k=256, gate_rows=3,
             scale=0.5, eps=1e-6)
    v.update(change)
    expect(dgm.lib().dg_sandwich_norm(*v.values(), None), status)


@no_gpu
@pytest.mark.parametrize("change,status", [
    ({}, OK), (dict(dh=0), OK), (dict(post_weight=0, dpost=0), OK), (dict(post_weight=0, dpost=0, rstd_x=0), OK),
    (dict(gate=0, dgate=0, gate_rows=0), OK), (dict(k=16384), OK), (dict(m=1 << 30, k=128, gate_rows=0x7fffffff), OK),
    (dict(dy=0), 1), (dict(x=0), 1), (dict(h=0), 1), (dict(weight=0), 1), (dict(rstd=0), 1), (dict(rstd_x=0), 1),
    (dict(dx=0), 1), (dict(dres=0), 1), (dict(dweight=0), 1), (dict(dpost=0), 1), (dict(post_weight=0), 1), (dict(gate=0), 1),
    (dict(dgate=0), 1), (dict(gate_rows=0), 1), (dict(m=0), 1), (dict(k=-128), 1), (dict(scale=INF), 1), (dict(scale=1e39), 1),
    (dict(dy=A + 8), 1), (dict(dh=A + 8), 1), (dict(x=A + 8), 1), (dict(h=A + 8), 1), (dict(dx=A + 8), 1),
    (dict(dres=A + 8), 1), (dict(dweight=A + 8), 1), (dict(dpost=A + 8), 1), (dict(dgate=A + 4), 1), (dict(ws=0), 1),
    (dict(ws=A + 8), 1), (dict(less=1), 1), (dict(k=200), 2), (dict(k=16384 + 128), 2), (dict(m=(1 << 30) + 1), 2),
])
def test_sandwich_norm_backward_refusals(change, status):
    v = dict(dy=A, dh=A, x=A, h=A, post_weight=A, gate=A, weight=A, rstd_x=A, rstd=A, dx=A, dres=A, dweight=A, dpost=A, dgate=A,
             m=8, k=256, gate_rows=3, scale=0.5, ws=A)
    less = change.get("less", 0)
    v.update({n: c for n, c in change.items() if n != "less"})
    need = dgm.dg_sandwich_norm_backward_workspace_bytes(v["m"], v["k"], bool(v["post_weight"]), bool(v["gate"]))
    expect(dgm.lib().dg_sandwich_norm_backward(*v.values(), need - less, None), status)


def test_sandwich_norm_backward_workspace_query():
    f = dgm.dg_sandwich_norm_backward_workspace_bytes
    assert f(0, 128) == f(8, 0) == f(8, 100) == f(8, 16384 + 128) == f((1 << 30) + 1, 128) == 0
    assert f(1, 128, False, False) == 512 and f(1, 128, True, False) == 1024 and f(1, 128, True, True) == 2048
    assert f(1 << 30, 16384) <= 128 << 20


def test_sandwich_binding_checks_tensors():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="x: must be a device tensor"):
        dgm.sandwich_norm(x, x, None, None, x[0].clone())
    with pytest.raises(ValueError, match="gate_rows: expected"):
        dgm.sandwich_norm(x, x, None, x, x[0].clone(), gate_rows=0)
    with pytest.raises(ValueError, match="dy: must be a device tensor"):
        dgm.sandwich_norm_backward(x, None, x, x, None, None, x[0].clone(), None, x[:, 0].float())


@pytest.mark.parametrize("post,gated", [(True, True), (False, True), (True, False), (False, False)])
def test_oracle_sandwich_gradients_are_those_of_differences(post, gated):
    """L = sum(dy * y) + sum(dh * h) without roundings: the oracle's gradients against central differences (error of
    order step^2: 1e-5 of the gradient's size for a step of 1e-4 with some margin for the third derivative)."""
    rng = np.random.default_rng(5)
    m, k, scale, eps = 4, 16, 0.7, 1e-3
    t = dict(x=rng.standard_normal((m, k)), res=rng.standard_normal((m, k)), pw=1 + 0.3 * rng.standard_normal(k),
             w=1 + 0.3 * rng.standard_normal(k), gate=rng.standard_normal((2, k)))
    dy, dh = rng.standard_normal((m, k)), rng.standard_normal((m, k))

    def parts(t):
        g = np.repeat(t["gate"], 2, axis=0) if gated else None
        h, rx = X.sandwich_norm(t["x"], t["res"], t["pw"] if post else None, g, scale, eps)
        return g, h, rx, 1 / np.sqrt(np.mean(h * h, axis=1) + eps)

    def loss(t):
        _, h, _, r = parts(t)
        return np.sum(dy * h * r[:, None] * t["w"]) + np.sum(dh * h)

    g, h, rx, r = parts(t)
    d, dx, yn, vn, gn = X.sandwich_norm_backward(dy, dh, t["x"], h, t["pw"] if post else None, g, t["w"], rx, r, scale)
    want = dict(x=dx, res=d, w=yn.sum(axis=0))
    if post:
        want["pw"] = vn.sum(axis=0)
    if gated:
        want["gate"] = gn.reshape(2, 2, k).sum(axis=1)
    for name, grad in want.items():
        for at in np.ndindex(*t[name].shape):
            up, dn = ({n: v.copy() for n, v in t.items()} for _ in range(2))
            up[name][at] += 1e-4
            dn[name][at] -= 1e-4
            assert abs((loss(up) - loss(dn)) / 2e-4 - grad[at]) < 1e-5 * (1 + np.abs(grad).max()), (name, at)


@no_gpu
@pytest.mark.parametrize("change,status", [
    ({}, OK), (dict(bias=0), OK), (dict(residual=0), OK), (dict(z=0), OK), (dict(act=2 | 16), OK), (dict(act=4), OK),
    (dict(m=1, n=16, k=128), OK),
    (dict(a=0), 1), (dict(a_sf=0), 1), (dict(b=0), 1), (dict(b_sf=0), 1), (dict(d=0), 1), (dict(act=5), 1), (dict(act=-1), 1),
    (dict(act=32), 1), (dict(act=21), 1), (dict(m=0), 1), (dict(n=0), 1), (dict(k=-1), 1),
    (dict(a=A + 8), 1), (dict(b=A + 8), 1), (dict(bias=A + 8), 1), (dict(residual=A + 8), 1), (dict(z=A + 8), 1),
    (dict(d=A + 8), 1), (dict(a_sf=A + 2), 1), (dict(b_sf=A + 2), 1),
    (dict(k=192), 2), (dict(n=24), 2), (dict(n=48, act=16), 2), (dict(m=1 << 22, k=2048), 2), (dict(m=1 << 16, n=(1 << 14) + 32, k=128), 2),
])
def test_linear_refusals(change, status):
    v = dict(a=A, a_sf=A, b=A, b_sf=A, bias=A, act=3, residual=A, z=A, d=A, m=8, n=256, k=256)
    v.update(change)
    need = dgm.lib().dg_mxfp4_gemm_workspace_bytes(v["m"], v["n"], v["k"], 256)
    expect(dgm.lib().dg_mxfp4_linear(*v.values(), A if need else None, need, None), status)


@no_gpu
@pytest.mark.parametrize("change,status", [
    ({}, OK), (dict(dz=0), OK), (dict(q=0, sf=0), OK), (dict(qt=0, sft=0), OK), (dict(dbias=0), OK), (dict(z=0, act=0), OK),
    (dict(act=18), OK), (dict(m=300, ws=A), OK), (dict(q=0, sf=0, qt=0, sft=0, dz=0), OK), (dict(m=300, dbias=0, ws=0, less=1), OK),
    (dict(dy=0), 1), (dict(z=0), 1), (dict(z=0, act=16), 1), (dict(q=0), 1), (dict(sf=0), 1), (dict(qt=0), 1), (dict(sft=0), 1),
    (dict(dz=0, q=0, sf=0, qt=0, sft=0, dbias=0), 1), (dict(act=7), 1), (dict(m=0), 1), (dict(n=-128), 1),
    (dict(m=300), 1), (dict(m=300, ws=A + 8), 1), (dict(m=300, ws=A, less=1), 1),
    (dict(dy=A + 8), 1), (dict(z=A + 8), 1), (dict(dz=A + 8), 1), (dict(q=A + 8), 1), (dict(qt=A + 8), 1), (dict(sf=A + 2), 1),
    (dict(sft=A + 2), 1), (dict(dbias=A + 8), 1),
    (dict(n=192), 2), (dict(n=128, act=18), 2), (dict(m=0x7fffffff - 126), 2), (dict(n=1 << 23), 2), (dict(n=(1 << 23) - 128), OK),
])
def test_activation_backward_refusals(change, status):
    v = dict(dy=A, z=A, act=3, dz=A, q=A, sf=A, qt=A, sft=A, dbias=A, m=8, n=256, ws=0)
    less = change.get("less", 0)
    v.update({n: c for n, c in change.items() if n != "less"})
    need = dgm.dg_activation_backward_workspace_bytes(v["m"], v["n"])
    expect(dgm.lib().dg_activation_backward(*v.values(), need - less, None), status)


def test_activation_backward_workspace_query():
    f = dgm.dg_activation_backward_workspace_bytes
    assert f(0, 128) == f(8, 0) == f(8, 100) == f(128, 256) == f(0x7fffffff, 128) == 0 and f(129, 256) == 5 * 256 * 4
    assert f(0x7fffffff - 127, (1 << 23) - 128) <= 1 << 30


def test_linear_binding_checks_tensors():
    q, sf = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="a: must be a device tensor"):
        dgm.mxfp4_linear(q, sf, q, sf)
    z = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="activation: expected"):
        dgm.activation_backward(z, z, 9)
    with pytest.raises(ValueError, match="dy: expected shape"):
        dgm.activation_backward(z, z, dgm.ACT_SILU | dgm.ACT_GATED)
    with pytest.raises(ValueError, match="dy: must be a device tensor"):
        dgm.activation_backward(z, z, dgm.ACT_SILU)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_oracle_activation_gradients_are_those_of_differences(act, gated):
    """The slope of sum(dy * d) against central differences, away from ReLU's kink."""
    rng = np.random.default_rng(1)
    z = rng.standard_normal((5, 16)) * 3
    z = np.where(np.abs(z) < 0.01, 0.5, z)
    dy = rng.standard_normal((5, 8 if gated else 16))
    dz = X.linear_epilogue_backward(dy, z, act, gated)
    for at in np.ndindex(*z.shape):
        up, dn = z.copy(), z.copy()
        up[at] += 1e-4
        dn[at] -= 1e-4
        slope = np.sum(dy * (X.linear_epilogue(up, act, gated) - X.linear_epilogue(dn, act, gated))) / 2e-4
        assert abs(slope - dz[at]) < 1e-6 * (1 + np.abs(dz).max())


RAGGED = [
    ({}, OK), (dict(m=1, n=16, k=128, groups=1), OK), (dict(groups=1024), OK),
    (dict(a=0), 1), (dict(a_sf=0), 1), (dict(b=0), 1), (dict(b_sf=0), 1), (dict(ms=0), 1), (dict(d=0), 1),
    (dict(m=0), 1), (dict(n=0), 1), (dict(k=0), 1), (dict(groups=0), 1), (dict(groups=-3), 1),
    (dict(a=A + 8), 1), (dict(b=A + 8), 1), (dict(d=A + 8), 1), (dict(a_sf=A + 2), 1), (dict(b_sf=A + 2), 1), (dict(ms=A + 2), 1),
    (dict(k=192), 2), (dict(n=24), 2), (dict(groups=1025), 2), (dict(m=1 << 22, k=2048), 2), (dict(n=1 << 22, k=2048), 2),
    (dict(m=1 << 16, n=(1 << 14) + 16, k=128), 2),
]


@no_gpu
@pytest.mark.parametrize("entry", ["dg_m_grouped_mxfp4_gemm_nt_ragged", "dg_k_grouped_mxfp4_gemm_nt_ragged"])
@pytest.mark.parametrize("change,status", RAGGED)
def test_ragged_gemm_refusals(entry, change, status):
    v = dict(a=A, a_sf=A, b=A, b_sf=A, ms=A, d=A, m=8, n=256, k=256, groups=4)
    v.update(change)
    expect(getattr(dgm.lib(), entry)(*v.values(), None), status)


@no_gpu
@pytest.mark.parametrize("change,status", [
    ({}, OK), (dict(q=0, sf=0), OK), (dict(x_type=1), OK), (dict(groups=1024), OK),
    (dict(x=0), 1), (dict(ms=0), 1), (dict(q=0), 1), (dict(sf=0), 1), (dict(qt=0), 1), (dict(sft=0), 1), (dict(x_type=2), 1),
    (dict(m=0), 1), (dict(k=0), 1), (dict(groups=0), 1), (dict(x=A + 8), 1), (dict(q=A + 8), 1), (dict(qt=A + 8), 1),
    (dict(sf=A + 2), 1), (dict(sft=A + 2), 1), (dict(ms=A + 1), 1), (dict(k=64), 2), (dict(groups=1025), 2),
    (dict(m=0x7fffffff - 126), 2),
])
def test_quantize_ragged_refusals(change, status):
    v = dict(x=A, x_type=0, ms=A, q=A, sf=A, qt=A, sft=A, m=8, k=256, groups=4)
    v.update(change)
    expect(dgm.lib().dg_quantize_mxfp4_ragged(*v.values(), None), status)


def test_ragged_blocks():
    f = dgm.dg_mxfp4_ragged_blocks
    assert f(0, 1) == f(1, 0) == f(1, 1025) == 0
    assert f(1, 1) == 1 and f(128, 1) == 1 and f(129, 1) == 2 and f(2, 2) == 2 and f(100, 100) == 100
    rng = np.random.default_rng(1)
    for _ in range(200):
        ms = rng.integers(0, 400, rng.integers(1, 9))
        assert sum(-(-int(r) // 128) for r in ms) <= f(max(int(ms.sum()), 1), len(ms))


def test_ragged_binding_checks_tensors():
    q, sf, ms = torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="ms: must be a device tensor"):
        dgm.m_grouped_mxfp4_gemm_nt_ragged(q, sf, q[None].repeat(2, 1, 1), sf[None].repeat(2, 1, 1), ms)
    with pytest.raises(ValueError, match="b: expected"):
        dgm.m_grouped_mxfp4_gemm_nt_ragged(q, sf, q, sf, ms)
    with pytest.raises(ValueError, match="x: must be a device tensor"):
        dgm.quantize_mxfp4_ragged(torch.zeros(4, 256), ms)
    with pytest.raises(ValueError, match="a: must be a device tensor"):
        dgm.k_grouped_mxfp4_gemm_nt_ragged(q, sf, q, sf, ms)
