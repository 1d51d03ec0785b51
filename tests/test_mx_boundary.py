"""Host-side checks of the quantisation, MXFP4 GEMM and norm entry points: every refusal comes before any HIP call,
and the binding checks its tensors (no compute is launched; these tests run without a GPU)."""

import ctypes
import os
import subprocess
import sys

import pytest
import torch

import fp4_gemm_dense_amd as dgm

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000      # a fake aligned address, never dereferenced on the host
BIG = 1 << 30
OK = (0, 4)      # passed validation; without a gfx950 device the call stops at the device check


@pytest.fixture(scope="module", autouse=True)
def _no_gpu():
    # a fake address must not reach a kernel
    if torch.cuda.is_available():
        pytest.skip("fake addresses: only where no GPU is visible")


@pytest.mark.parametrize("change,status", [
    ({}, OK), (dict(x_type=1), OK), (dict(qt=A, sft=A), OK), (dict(q=0, sf=0, values=A), OK),
    (dict(q=0, sf=0, qt=A, sft=A), OK), (dict(groups=3, m=1), OK),
    (dict(x=0), 1), (dict(q=0, sf=0), 1), (dict(sf=0), 1), (dict(q=0), 1), (dict(qt=A), 1), (dict(sft=A), 1),
    (dict(x_type=2), 1), (dict(x_type=-1), 1), (dict(m=0), 1), (dict(k=0), 1), (dict(groups=0), 1), (dict(m=-5), 1),
    (dict(x=A + 8), 1), (dict(q=A + 4), 1), (dict(sf=A + 2), 1), (dict(qt=A + 8, sft=A), 1), (dict(qt=A, sft=A + 1), 1),
    (dict(values=A + 2), 1), (dict(k=192), 2), (dict(k=64), 2), (dict(groups=1 << 16, m=1 << 15), 2),
    (dict(m=0x7fffffff), 2),
])
def test_quantize_refusals(change, status):
    v = dict(x=A, x_type=0, q=A, sf=A, qt=0, sft=0, values=0, groups=1, m=8, k=256)
    v.update(change)
    got = dgm.lib().dg_quantize_mxfp4(*v.values(), None)
    assert got in status if isinstance(status, tuple) else got == status


@pytest.mark.parametrize("change,status", [
    ({}, OK), (dict(c=A), OK), (dict(m=1, n=16, k=128), OK),
    (dict(a=0), 1), (dict(a_sf=0), 1), (dict(b=0), 1), (dict(b_sf=0), 1), (dict(d=0), 1),
    (dict(m=0), 1), (dict(n=-1), 1), (dict(k=0), 1),
    (dict(a=A + 8), 1), (dict(b=A + 8), 1), (dict(c=A + 8), 1), (dict(d=A + 8), 1), (dict(a_sf=A + 2), 1),
    (dict(b_sf=A + 2), 1),
    (dict(k=192), 2), (dict(n=24), 2), (dict(m=1 << 22, k=2048), 2), (dict(n=1 << 22, k=2048), 2),
    (dict(m=1 << 16, n=(1 << 14) + 16, k=128), 2),
])
def test_gemm_refusals(change, status):
    v = dict(a=A, a_sf=A, b=A, b_sf=A, c=0, d=A, m=8, n=256, k=256)
    v.update(change)
    need = dgm.lib().dg_mxfp4_gemm_workspace_bytes(v["m"], v["n"], v["k"], 256)
    got = dgm.lib().dg_mxfp4_gemm_nt(*v.values(), A if need else None, need, None)
    assert got in status if isinstance(status, tuple) else got == status


def test_gemm_workspace_query_is_host_only_and_zero_for_invalid_sizes():
    f = dgm.dg_mxfp4_gemm_workspace_bytes
    for bad in ((0, 256, 256), (8, 0, 256), (8, 256, 0), (8, 24, 256), (8, 256, 200)):
        assert f(*bad, 256) == 0
    for m in (1, 16, 64, 100, 300, 1111, 4096):
        for n, k in ((16, 128), (2112, 7168), (7168, 16384), (24576, 1536)):
            assert 0 <= f(m, n, k, 256) <= 256 << 20


@pytest.mark.parametrize("change,status", [
    ({}, OK), (dict(residual=0), OK), (dict(h=0), OK), (dict(rstd=0), OK), (dict(fmt=1), OK), (dict(fmt=2), OK),
    (dict(k=32768), OK),
    (dict(x=0), 1), (dict(weight=0), 1), (dict(q=0), 1), (dict(sf=0), 1), (dict(fmt=3), 1), (dict(fmt=-1), 1),
    (dict(m=0), 1), (dict(k=-128), 1), (dict(eps=0.0), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(x=A + 2), 1), (dict(residual=A + 8), 1), (dict(weight=A + 8), 1),
    (dict(h=A + 8), 1), (dict(q=A + 8), 1), (dict(sf=A + 2), 1), (dict(rstd=A + 2), 1),
    (dict(k=64), 2), (dict(k=320), 2), (dict(k=32768 + 128), 2),
    (dict(m=1 << 26, k=128), 2), (dict(m=1 << 22, k=32768), 2),
])
def test_norm_refusals(change, status):
    v = dict(x=A, residual=A, weight=A, h=A, q=A, sf=A, fmt=0, rstd=A, m=8, k=256, eps=1e-6)
    v.update(change)
    got = dgm.lib().dg_add_rms_norm(*v.values(), None)
    assert got in status if isinstance(status, tuple) else got == status


@pytest.mark.parametrize("change,status", [
    ({}, OK), (dict(dh=0), OK), (dict(m=5000, ws_bytes=BIG), OK),
    (dict(dy=0), 1), (dict(h=0), 1), (dict(weight=0), 1), (dict(rstd=0), 1), (dict(dx=0), 1), (dict(dweight=0), 1),
    (dict(m=5000, ws=0), 1), (dict(m=5000, ws=A + 8), 1), (dict(m=5000, ws_bytes=15), 1), (dict(ws=0), OK),
    (dict(m=0), 1), (dict(k=0), 1), (dict(dy=A + 8), 1),
    (dict(dh=A + 8), 1), (dict(dx=A + 2), 1), (dict(dweight=A + 4), 1), (dict(k=200), 2), (dict(k=32768 + 128), 2),
])
def test_norm_backward_refusals(change, status):
    v = dict(dy=A, dh=A, h=A, weight=A, rstd=A, dx=A, dweight=A, m=8, k=256, ws=A, ws_bytes=None)
    v.update(change)
    if v["ws_bytes"] is None:
        v["ws_bytes"] = dgm.dg_add_rms_norm_backward_workspace_bytes(v["m"], v["k"])
    got = dgm.lib().dg_add_rms_norm_backward(*v.values(), None)
    assert got in status if isinstance(status, tuple) else got == status


def test_norm_backward_workspace_query():
    f = dgm.dg_add_rms_norm_backward_workspace_bytes
    assert f(0, 128) == f(8, 0) == f(8, 100) == f(8, 32768 + 128) == 0
    assert f(1, 128) == f(1024, 7168) == 0 and f(1025, 128) >= 128 * 4 and f(1 << 30, 7168) <= 64 << 20


def test_binding_checks_tensors():
    """The binding names the argument at fault; CPU tensors are refused."""
    bf, u8, i32, f32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32
    x = torch.zeros(4, 256, dtype=bf)
    with pytest.raises(ValueError, match="x: must be a device tensor"):
        dgm.quantize_mxfp4(x)
    with pytest.raises(TypeError, match="x: expected"):
        dgm.quantize_mxfp4(x.half())
    with pytest.raises(ValueError, match="x: must be contiguous"):
        dgm.dg_quantize_mxfp4(torch.zeros(256, 4, dtype=bf).t(), None)
    with pytest.raises(ValueError, match=r"x: expected \[m, k\]"):
        dgm.dg_quantize_mxfp4(torch.zeros(256, dtype=bf))
    q, sf = torch.zeros(4, 128, dtype=u8), torch.zeros(2, 4, dtype=i32)
    with pytest.raises(ValueError, match="a: must be a device tensor"):
        dgm.mxfp4_gemm_nt(q, sf, q, sf)
    with pytest.raises(ValueError, match="x: must be a device tensor"):
        dgm.add_rms_norm(x, None, x[0].clone())
    with pytest.raises(ValueError, match="quant_format"):
        dgm.dg_add_rms_norm(x, None, x[0].clone(), None, q, sf, 1e-6, 7)
    with pytest.raises(ValueError, match="dy: must be a device tensor"):
        dgm.dg_add_rms_norm_backward(x, None, x, x[0].clone(), torch.zeros(4, dtype=f32), x, torch.zeros(256, dtype=f32),
                                     torch.zeros(8, dtype=u8))
    assert isinstance(dgm.lib(), ctypes.CDLL)


def test_norm_backward_refuses_rows_whose_successor_passes_int():
    """A workgroup steps from row to row by up to 1024: the last row it tests has to be an int."""
    def call(m):
        need = dgm.dg_add_rms_norm_backward_workspace_bytes(m, 128)
        return need, dgm.lib().dg_add_rms_norm_backward(A, A, A, A, A, A, A, m, 128, A, need, None)
    assert call(0x7fffffff) == (0, 2) and call(0x7fffffff - 1023) == (0, 2)
    need, status = call(0x7fffffff - 1024)
    assert need > 0 and status in OK


def test_host_only_uses_without_the_device_backend():
    """A torch built without the device backend has neither of the functions that the launching calls read the device and
    stream with: importing the binding, plans, workspace queries and refusals have to work there."""
    code = """
import torch
for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
import fp4_gemm_dense_amd as dgm
assert dgm.dg_mxfp4_gemm_workspace_bytes(512, 512, 8192, 256) >= 0
assert dgm.dg_add_rms_norm_backward_workspace_bytes(1025, 128) > 0
try:
    dgm.quantize_mxfp4(torch.zeros(4, 256, dtype=torch.bfloat16))
except ValueError as e:
    assert "must be a device tensor" in str(e)
else:
    raise AssertionError
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
