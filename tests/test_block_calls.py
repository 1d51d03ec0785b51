"""What the binding hands to the C entry points of the operators around a block, seen without a GPU: host tensors stand for
device ones, and the call is recorded instead of made."""

import ctypes
import sys

import pytest
import torch

import fp4_gemm_dense_amd as dgm


@pytest.fixture
def calls(monkeypatch):
    """The recorded calls, (entry point, arguments); tensors have to have the asked types and shapes."""
    made = []

    def arg(t, dtypes, shape, index, name):
        if t is None:
            return None
        assert t.dtype in dtypes and tuple(t.shape) == tuple(shape) and t.is_contiguous(), name
        return t.data_ptr()

    monkeypatch.setattr(dgm, "_arg", arg)
    monkeypatch.setattr(dgm, "_call", lambda name, index, *args: made.append((name, args)))
    return made


# the argument's place
GATE_ROWS = {"dg_sandwich_norm": 13, "dg_sandwich_norm_backward": 16}
HUGE = [8, 9, 1 << 30, (1 << 31) - 1, 1 << 31, 1 << 32, (1 << 32) + 3, (1 << 62) + 5, sys.maxsize]


@pytest.mark.parametrize("gate_rows", HUGE)
def test_one_gate_for_all_rows(calls, gate_rows):
    """gate_rows of m or more is one gate row, however large: the C call keeps 32 bits of it, and a smaller number there
    would be more gate rows than gate and dgate have."""
    m, k = 8, 128
    x, gate, w = torch.zeros(m, k, dtype=torch.bfloat16), torch.zeros(1, k, dtype=torch.bfloat16), torch.zeros(k, dtype=torch.bfloat16)
    r = torch.zeros(m)
    dgm.sandwich_norm(x, x, w, gate, w, gate_rows=gate_rows)
    dgm.dg_sandwich_norm(x, x, w, gate, w, torch.empty_like(x), torch.empty(m, k, dtype=torch.uint8), torch.empty(1, m), 0,
                         gate_rows=gate_rows)
    dgm.sandwich_norm_backward(x, None, x, x, w, gate, w, r, r, gate_rows=gate_rows)
    dgm.dg_sandwich_norm_backward(x, None, x, x, w, gate, w, r, r, torch.empty_like(x), torch.empty_like(x), torch.empty(k),
                                  torch.empty(k), torch.empty(1, k), torch.empty(1 << 16, dtype=torch.uint8), gate_rows=gate_rows)
    assert [name for name, _ in calls] == ["dg_sandwich_norm"] * 2 + ["dg_sandwich_norm_backward"] * 2
    for name, args in calls:
        got = ctypes.c_int(args[GATE_ROWS[name]]).value
        assert got >= m, f"{name}: {got}"


@pytest.mark.parametrize("fmt", [-1, 3, 1 << 32, (1 << 32) + 1, (1 << 32) + 2])
def test_unknown_formats_are_refused(calls, fmt):
    """Also those whose low 32 bits are a format's: codes and scales would be another format's than the tensors say."""
    x, w = torch.zeros(8, 512, dtype=torch.bfloat16), torch.zeros(512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="quant_format: expected"):
        dgm.sandwich_norm(x, x, None, None, w, quant_format=fmt)
    with pytest.raises(ValueError, match="quant_format: expected"):
        dgm.add_rms_norm(x, x, w, quant_format=fmt)
    assert not calls
