"""Python binding of the gfx950 fine-grained-scaled FP8 / FP8xFP4 GEMM library.

Argument marshalling only: every function here checks dtypes, shapes and
devices of torch tensors, then calls the C ABI of ``libdg.so`` (declared in
``include/dg.h``) with raw device pointers and torch's current HIP stream.
All arithmetic runs in the library's HIP kernels; there is no fallback path.
If the library is not built, ``load_library()`` raises.

The ``dg_*`` functions mirror the C entry points one to one (outputs are
caller-allocated).  ``fp8_gemm_nt`` etc. are convenience wrappers that allocate
the output, as in the pages' Python API (usage guide, 五、使用方法).
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdg.so")
_lib = None

DG_OK = 0
STATUS_NAMES = {0: "DG_OK", 1: "DG_ERR_INVALID_ARG", 2: "DG_ERR_UNSUPPORTED", 3: "DG_ERR_HIP",
                4: "DG_ERR_NO_DEVICE", 5: "DG_ERR_SCRATCH_LIMIT"}

_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t

_SIGNATURES = {
    "dg_fp8_gemm_nt": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "dg_m_grouped_fp8_gemm_nt_contiguous": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "dg_m_grouped_fp8_gemm_nt_masked": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _SZ, _P]),
    "dg_fp8_gemm_nn": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "dg_fp8_gemm_tn": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "dg_k_grouped_fp8_gemm_tn_contiguous": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "dg_fp8_gemm_tt": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "dg_m_grouped_fp8_gemm_nn_contiguous": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "dg_fp8_gemm_nt_ue8m0": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P, _SZ, _P]),
    "dg_m_grouped_fp8_gemm_nt_masked_ue8m0": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _SZ, _P]),
    "dg_m_grouped_fp8_fp4_gemm_nt_contiguous": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _P]),
    "dg_m_grouped_fp8_fp4_gemm_nt_masked": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P]),
    "dg_transform_fp4_weight_sf": (_I, [_P, _P, _I, _I, _I, _P]),
    "dg_fp8_fp4_expert_ffn_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I]),
    "dg_fp8_fp4_expert_ffn": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _SZ, _P]),
    "dg_fp8_gemm_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
    "dg_quantize_mxfp4": (_I, [_P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
    "dg_mxfp4_gemm_nt": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P, _SZ, _P]),
    "dg_mxfp4_gemm_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "dg_m_grouped_mxfp4_gemm_nt_ragged": (_I, [_P] * 6 + [_I] * 4 + [_P]),
    "dg_k_grouped_mxfp4_gemm_nt_ragged": (_I, [_P] * 6 + [_I] * 4 + [_P]),
    "dg_quantize_mxfp4_ragged": (_I, [_P, _I] + [_P] * 5 + [_I] * 3 + [_P]),
    "dg_mxfp4_ragged_blocks": (_I, [_I, _I]),
    "dg_mxfp4_linear": (_I, [_P] * 5 + [_I] + [_P] * 3 + [_I, _I, _I, _P, _SZ, _P]),
    "dg_activation_backward": (_I, [_P, _P, _I] + [_P] * 6 + [_I, _I, _P, _SZ, _P]),
    "dg_activation_backward_workspace_bytes": (_SZ, [_I, _I]),
    "dg_add_rms_norm": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _I, _I, ctypes.c_float, _P]),
    "dg_add_rms_norm_backward": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _P, _SZ, _P]),
    "dg_add_rms_norm_backward_workspace_bytes": (_SZ, [_I, _I]),
    "dg_sandwich_norm": (_I, [_P] * 8 + [_I, _P, _P, _I, _I, _I, ctypes.c_double, ctypes.c_float, _P]),
    "dg_sandwich_norm_backward": (_I, [_P] * 14 + [_I, _I, _I, ctypes.c_double, _P, _SZ, _P]),
    "dg_sandwich_norm_backward_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "dg_fp8_gemm_nt_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _P]),
    "dg_get_mk_alignment_for_contiguous_layout": (_I, []),
    "dg_set_num_cus": (_I, [_I]),
    "dg_get_num_cus": (_I, []),
    "dg_query_plan": (_I, [_I, _I, _I, _I, _I, _P]),
    "dg_query_plan_contiguous": (_I, [_I, _I, _I, _I, _I, _P]),
    "dg_query_plan_form": (_I, [_I, _I, _I, _I, _I, _I, _I, _P]),
    "dg_num_tiles": (_I, [_I, _I, _I, _I]),
    "dg_status_string": (ctypes.c_char_p, [_I]),
}


class DgPlan(ctypes.Structure):
    _fields_ = [("block_m", _I), ("block_n", _I), ("num_tiles", _I), ("num_workgroups", _I),
                ("kernel_id", _I), ("splits", _I), ("full_tiles", _I)]


class DgError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)} "
                         f"({_lib.dg_status_string(status).decode() if _lib else '?'})")


def load_library(path=LIB_PATH):
    """Load libdg.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m fp4_gemm_dense_amd.build` "
                           "(or __graft_entry__.build()); there is no fallback path")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def lib():
    return load_library()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _check(fn, status):
    if status != DG_OK:
        raise DgError(fn, status)


def _req(t, dtype, shape, name):
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a device tensor")


_U8 = torch.uint8
_BF = (torch.int16, torch.bfloat16, torch.uint16) if hasattr(torch, "uint16") else (torch.int16, torch.bfloat16)


def _req_bf16(t, shape, name):
    if t.dtype not in _BF:
        raise TypeError(f"{name}: expected bf16 (or its int16 bit view), got {t.dtype}")
    _req(t, t.dtype, shape, name)


def _nb(n):
    return (n + 127) // 128


# dg_gemm_form (include/dg.h): which FP8 GEMM entry point a workspace query is for
FORM_NT, FORM_NN, FORM_TN, FORM_TT, FORM_NT_UE8M0 = 0, 1, 2, 3, 4
FORM_CONTIGUOUS_NT, FORM_CONTIGUOUS_NN, FORM_CONTIGUOUS_NT_UE8M0 = 5, 6, 7
FORM_MASKED_NT, FORM_MASKED_NT_UE8M0 = 8, 9


def dg_fp8_gemm_workspace_bytes(form, m, n, k, num_groups=1, expected_m=0, num_cus=0):
    """Bytes of workspace the FP8 GEMM entry point `form` needs for these sizes (0: none)."""
    return int(lib().dg_fp8_gemm_workspace_bytes(int(form), m, n, k, num_groups, int(expected_m), int(num_cus)))


def _workspace(form, m, n, k, num_groups, expected_m, device, workspace):
    """(pointer, bytes) of the workspace for one call: the caller's uint8 tensor, or a
    new one from torch's caching allocator when none is given and the plan needs one."""
    if workspace is not None:
        _req(workspace, _U8, (workspace.numel(),), "workspace")
        return _ptr(workspace), workspace.numel(), workspace
    need = dg_fp8_gemm_workspace_bytes(form, m, n, k, num_groups, expected_m)
    if need == 0:
        return None, 0, None
    ws = torch.empty(need, dtype=_U8, device=device)
    return _ptr(ws), need, ws


# ----------------------------------------------------------------------------
# C entry points (caller-allocated outputs)
# ----------------------------------------------------------------------------

def dg_fp8_gemm_nt(a, sfa, b, sfb, c, d, workspace=None):
    """d = c + a . b^T (see include/dg.h).  a/b uint8 e4m3, sfa [K/128, M], sfb [ceil(N/128), K/128].
    workspace: optional uint8 device tensor for the split-K partials (allocated here when needed
    and not given)."""
    L = lib()
    M, K = a.shape
    N = b.shape[0]
    _req(a, _U8, (M, K), "a")
    _req(b, _U8, (N, K), "b")
    _req(sfa, torch.float32, (K // 128, M), "sfa")
    _req(sfb, torch.float32, (_nb(N), K // 128), "sfb")
    if c is not None:
        _req_bf16(c, (M, N), "c")
    _req_bf16(d, (M, N), "d")
    wp, wn, _keep = _workspace(FORM_NT, M, N, K, 1, 0, a.device, workspace)
    _check("dg_fp8_gemm_nt", L.dg_fp8_gemm_nt(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(c), _ptr(d),
                                              M, N, K, wp, wn, _stream(a)))
    return d


def dg_fp8_gemm_nt_noalloc(a, sfa, b, sfb, c, d):
    """d = c + a . b^T like dg_fp8_gemm_nt, with the split-K partials in the library's static
    per-GPU scratch buffer (24 MiB): the call allocates nothing.  Calls that overlap in time
    on one GPU race on that buffer."""
    L = lib()
    M, K = a.shape
    N = b.shape[0]
    _req(a, _U8, (M, K), "a")
    _req(b, _U8, (N, K), "b")
    _req(sfa, torch.float32, (K // 128, M), "sfa")
    _req(sfb, torch.float32, (_nb(N), K // 128), "sfb")
    if c is not None:
        _req_bf16(c, (M, N), "c")
    _req_bf16(d, (M, N), "d")
    _check("dg_fp8_gemm_nt_noalloc", L.dg_fp8_gemm_nt_noalloc(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(c),
                                                              _ptr(d), M, N, K, _stream(a)))
    return d


def dg_m_grouped_fp8_gemm_nt_contiguous(a, sfa, b, sfb, m_indices, d, workspace=None):
    L = lib()
    M, K = a.shape
    G, N = b.shape[0], b.shape[1]
    _req(a, _U8, (M, K), "a")
    _req(b, _U8, (G, N, K), "b")
    _req(sfa, torch.float32, (K // 128, M), "sfa")
    _req(sfb, torch.float32, (G, _nb(N), K // 128), "sfb")
    _req(m_indices, torch.int32, (M,), "m_indices")
    _req_bf16(d, (M, N), "d")
    wp, wn, _keep = _workspace(FORM_CONTIGUOUS_NT, M, N, K, G, 0, a.device, workspace)
    _check("dg_m_grouped_fp8_gemm_nt_contiguous",
           L.dg_m_grouped_fp8_gemm_nt_contiguous(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(m_indices),
                                                 _ptr(d), M, N, K, G, wp, wn, _stream(a)))
    return d


def dg_m_grouped_fp8_gemm_nt_masked(a, sfa, b, sfb, masked_m, d, expected_m=0, workspace=None):
    L = lib()
    G, max_m, K = a.shape
    N = b.shape[1]
    _req(a, _U8, (G, max_m, K), "a")
    _req(b, _U8, (G, N, K), "b")
    _req(sfa, torch.float32, (G, K // 128, max_m), "sfa")
    _req(sfb, torch.float32, (G, _nb(N), K // 128), "sfb")
    _req(masked_m, torch.int32, (G,), "masked_m")
    _req_bf16(d, (G, max_m, N), "d")
    wp, wn, _keep = _workspace(FORM_MASKED_NT, max_m, N, K, G, expected_m, a.device, workspace)
    _check("dg_m_grouped_fp8_gemm_nt_masked",
           L.dg_m_grouped_fp8_gemm_nt_masked(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(masked_m), _ptr(d),
                                             G, max_m, N, K, int(expected_m), wp, wn, _stream(a)))
    return d


def dg_fp8_gemm_nn(a, sfa, b, sfb, c, d, workspace=None):
    """d = c + a . b with b stored [K, N] (NN layout)."""
    L = lib()
    M, K = a.shape
    N = b.shape[1]
    _req(a, _U8, (M, K), "a")
    _req(b, _U8, (K, N), "b")
    _req(sfa, torch.float32, (K // 128, M), "sfa")
    _req(sfb, torch.float32, (_nb(N), K // 128), "sfb")
    if c is not None:
        _req_bf16(c, (M, N), "c")
    _req_bf16(d, (M, N), "d")
    wp, wn, _keep = _workspace(FORM_NN, M, N, K, 1, 0, a.device, workspace)
    _check("dg_fp8_gemm_nn", L.dg_fp8_gemm_nn(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(c), _ptr(d),
                                              M, N, K, wp, wn, _stream(a)))
    return d


def _dense_layout(name, form, a, sfa, b, sfb, c, d, a_km, b_kn, workspace):
    L = lib()
    if a_km:
        K, M = a.shape
    else:
        M, K = a.shape
    N = b.shape[1] if b_kn else b.shape[0]
    _req(a, _U8, (K, M) if a_km else (M, K), "a")
    _req(b, _U8, (K, N) if b_kn else (N, K), "b")
    _req(sfa, torch.float32, (K // 128, M), "sfa")
    _req(sfb, torch.float32, (_nb(N), K // 128), "sfb")
    if c is not None:
        _req_bf16(c, (M, N), "c")
    _req_bf16(d, (M, N), "d")
    wp, wn, _keep = _workspace(form, M, N, K, 1, 0, a.device, workspace)
    _check(name, getattr(L, name)(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(c), _ptr(d), M, N, K, wp, wn,
                                  _stream(a)))
    return d


def dg_fp8_gemm_tn(a, sfa, b, sfb, c, d, workspace=None):
    """d = c + a^T b with a stored [K, M] and b stored [K, N] (TN layout)."""
    return _dense_layout("dg_fp8_gemm_tn", FORM_TN, a, sfa, b, sfb, c, d, True, True, workspace)


def dg_fp8_gemm_tt(a, sfa, b, sfb, c, d, workspace=None):
    """d = c + a^T b^T with a stored [K, M] and b stored [N, K] (TT layout)."""
    return _dense_layout("dg_fp8_gemm_tt", FORM_TT, a, sfa, b, sfb, c, d, True, False, workspace)


def dg_k_grouped_fp8_gemm_tn_contiguous(a, sfa, b, sfb, ks, d):
    """d[g] = a[rows of g]^T . b[rows of g] with a stored [K, M], b [K, N], groups along K (ks on the device)."""
    L = lib()
    K, M = a.shape
    N = b.shape[1]
    G = ks.shape[0]
    _req(a, _U8, (K, M), "a")
    _req(sfa, torch.float32, (K // 128, M), "sfa")
    _req(b, _U8, (K, N), "b")
    _req(sfb, torch.float32, (_nb(N), K // 128), "sfb")
    _req(ks, torch.int32, (G,), "ks")
    _req_bf16(d, (G, M, N), "d")
    _check("dg_k_grouped_fp8_gemm_tn_contiguous",
           L.dg_k_grouped_fp8_gemm_tn_contiguous(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(ks), _ptr(d),
                                                 M, N, K, G, _stream(a)))
    return d


def dg_m_grouped_fp8_gemm_nn_contiguous(a, sfa, b, sfb, m_indices, d, workspace=None):
    """Contiguous grouped form with each group's b stored [K, N]."""
    L = lib()
    M, K = a.shape
    G, N = b.shape[0], b.shape[2]
    _req(a, _U8, (M, K), "a")
    _req(sfa, torch.float32, (K // 128, M), "sfa")
    _req(b, _U8, (G, K, N), "b")
    _req(sfb, torch.float32, (G, _nb(N), K // 128), "sfb")
    _req(m_indices, torch.int32, (M,), "m_indices")
    _req_bf16(d, (M, N), "d")
    wp, wn, _keep = _workspace(FORM_CONTIGUOUS_NN, M, N, K, G, 0, a.device, workspace)
    _check("dg_m_grouped_fp8_gemm_nn_contiguous",
           L.dg_m_grouped_fp8_gemm_nn_contiguous(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(m_indices), _ptr(d),
                                                 M, N, K, G, wp, wn, _stream(a)))
    return d


def _kw(K):
    return (K // 128 + 3) // 4


def dg_fp8_gemm_nt_ue8m0(a, sfa, b, sfb, c, d, workspace=None):
    L = lib()
    M, K = a.shape
    N = b.shape[0]
    _req(a, _U8, (M, K), "a")
    _req(sfa, torch.int32, (M, _kw(K)), "sfa")
    _req(b, _U8, (N, K), "b")
    _req(sfb, torch.int32, (_nb(N), _kw(K)), "sfb")
    if c is not None:
        _req_bf16(c, (M, N), "c")
    _req_bf16(d, (M, N), "d")
    wp, wn, _keep = _workspace(FORM_NT_UE8M0, M, N, K, 1, 0, a.device, workspace)
    _check("dg_fp8_gemm_nt_ue8m0",
           L.dg_fp8_gemm_nt_ue8m0(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(c),
                                  _ptr(d), M, N, K, wp, wn, _stream(a)))
    return d


def dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0(a, sfa, b, sfb, m_indices, d, workspace=None):
    L = lib()
    M, K = a.shape
    G, N = b.shape[0], b.shape[1]
    _req(a, _U8, (M, K), "a")
    _req(sfa, torch.int32, (M, _kw(K)), "sfa")
    _req(b, _U8, (G, N, K), "b")
    _req(sfb, torch.int32, (G, _nb(N), _kw(K)), "sfb")
    _req(m_indices, torch.int32, (M,), "m_indices")
    _req_bf16(d, (M, N), "d")
    wp, wn, _keep = _workspace(FORM_CONTIGUOUS_NT_UE8M0, M, N, K, G, 0, a.device, workspace)
    _check("dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0",
           L.dg_m_grouped_fp8_gemm_nt_contiguous_ue8m0(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(m_indices),
                                                       _ptr(d), M, N, K, G, wp, wn, _stream(a)))
    return d


def dg_m_grouped_fp8_gemm_nt_masked_ue8m0(a, sfa, b, sfb, masked_m, d, expected_m=0, workspace=None):
    L = lib()
    G, max_m, K = a.shape
    N = b.shape[1]
    _req(a, _U8, (G, max_m, K), "a")
    _req(sfa, torch.int32, (G, max_m, _kw(K)), "sfa")
    _req(b, _U8, (G, N, K), "b")
    _req(sfb, torch.int32, (G, _nb(N), _kw(K)), "sfb")
    _req(masked_m, torch.int32, (G,), "masked_m")
    _req_bf16(d, (G, max_m, N), "d")
    wp, wn, _keep = _workspace(FORM_MASKED_NT_UE8M0, max_m, N, K, G, expected_m, a.device, workspace)
    _check("dg_m_grouped_fp8_gemm_nt_masked_ue8m0",
           L.dg_m_grouped_fp8_gemm_nt_masked_ue8m0(_ptr(a), _ptr(sfa), _ptr(b), _ptr(sfb), _ptr(masked_m),
                                                   _ptr(d), G, max_m, N, K, int(expected_m), wp, wn, _stream(a)))
    return d


def dg_m_grouped_fp8_fp4_gemm_nt_contiguous(a, a_sf, b, b_sf, m_indices, d):
    L = lib()
    M, K = a.shape
    G, N = b.shape[0], b.shape[1]
    _req(a, _U8, (M, K), "a")
    _req(a_sf, torch.int32, (M, (K // 128 + 3) // 4), "a_sf")
    _req(b, _U8, (G, N, K // 2), "b")
    _req(b_sf, torch.int32, (G, K // 128, N), "b_sf")
    _req(m_indices, torch.int32, (M,), "m_indices")
    _req_bf16(d, (M, N), "d")
    _check("dg_m_grouped_fp8_fp4_gemm_nt_contiguous",
           L.dg_m_grouped_fp8_fp4_gemm_nt_contiguous(_ptr(a), _ptr(a_sf), _ptr(b), _ptr(b_sf), _ptr(m_indices),
                                                     _ptr(d), M, N, K, G, _stream(a)))
    return d


def dg_m_grouped_fp8_fp4_gemm_nt_masked(a, a_sf, b, b_sf, masked_m, d, expected_m=0):
    L = lib()
    G, max_m, K = a.shape
    N = b.shape[1]
    _req(a, _U8, (G, max_m, K), "a")
    _req(a_sf, torch.int32, (G, max_m, (K // 128 + 3) // 4), "a_sf")
    _req(b, _U8, (G, N, K // 2), "b")
    _req(b_sf, torch.int32, (G, K // 128, N), "b_sf")
    _req(masked_m, torch.int32, (G,), "masked_m")
    _req_bf16(d, (G, max_m, N), "d")
    _check("dg_m_grouped_fp8_fp4_gemm_nt_masked",
           L.dg_m_grouped_fp8_fp4_gemm_nt_masked(_ptr(a), _ptr(a_sf), _ptr(b), _ptr(b_sf), _ptr(masked_m),
                                                 _ptr(d), G, max_m, N, K, int(expected_m), _stream(a)))
    return d


def dg_transform_fp4_weight_sf(sf, sf_t=None):
    """Packed UE8M0 weight-scale words [G, N, K/128] -> K-block-major [G, K/128, N] (new tensor
    unless sf_t is given)."""
    G, N, KB = sf.shape
    _req(sf, torch.int32, (G, N, KB), "sf")
    if sf_t is None:
        sf_t = torch.empty(G, KB, N, dtype=torch.int32, device=sf.device)
    _req(sf_t, torch.int32, (G, KB, N), "sf_t")
    _check("dg_transform_fp4_weight_sf",
           lib().dg_transform_fp4_weight_sf(_ptr(sf), _ptr(sf_t), G, N, KB * 128, _stream(sf)))
    return sf_t


def dg_fp8_fp4_expert_ffn_workspace_bytes(num_tokens, num_topk, num_local_experts, hidden, intermediate):
    return int(lib().dg_fp8_fp4_expert_ffn_workspace_bytes(num_tokens, num_topk, num_local_experts,
                                                            hidden, intermediate))


def dg_fp8_fp4_expert_ffn(x, x_sf, topk_idx, topk_w, w1, w1_sf, w2, w2_sf, y, expert_offset, workspace):
    L = lib()
    T, H = x.shape
    k = topk_idx.shape[1]
    E, I2 = w1.shape[0], w1.shape[1]
    I = I2 // 2
    _req(x, _U8, (T, H), "x")
    _req(x_sf, torch.int32, (T, H // 512), "x_sf")
    _req(topk_idx, torch.int32, (T, k), "topk_idx")
    _req(topk_w, torch.float32, (T, k), "topk_w")
    _req(w1, _U8, (E, 2 * I, H // 2), "w1")
    _req(w1_sf, torch.int32, (E, H // 128, 2 * I), "w1_sf")
    _req(w2, _U8, (E, H, I // 2), "w2")
    _req(w2_sf, torch.int32, (E, I // 128, H), "w2_sf")
    _req_bf16(y, (T, H), "y")
    _req(workspace, _U8, (workspace.numel(),), "workspace")
    _check("dg_fp8_fp4_expert_ffn",
           L.dg_fp8_fp4_expert_ffn(_ptr(x), _ptr(x_sf), _ptr(topk_idx), _ptr(topk_w), _ptr(w1), _ptr(w1_sf),
                                   _ptr(w2), _ptr(w2_sf), _ptr(y), T, k, E, int(expert_offset), H, I,
                                   _ptr(workspace), workspace.numel(), _stream(x)))
    return y


# dg_dtype and dg_quant_format (include/dg.h)
_X_TYPES = {**{t: 0 for t in _BF}, torch.float32: 1}
QUANT_E4M3_F32, QUANT_E4M3_UE8M0, QUANT_MXFP4 = 0, 1, 2


def _call(name, index, *args):
    """The C entry point on device `index` and torch's current stream there.  (A decode step makes many calls of a few
    microseconds: these wrappers read the raw stream and device index, and pass addresses as plain integers.  A torch
    without the device backend has neither of the two, so they are looked up here.)"""
    f, c = getattr(_lib or load_library(), name), torch._C
    if index == c._cuda_getDevice():
        st = f(*args, c._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            st = f(*args, c._cuda_getCurrentRawStream(index))
    if st:
        raise DgError(name, st)


def _arg(t, dtypes, shape, index, name):
    """Checks one tensor argument (None passes; index: the device it has to be on) and returns its address."""
    if t is None:
        return None
    if t.dtype in dtypes and t.shape == shape and t.is_contiguous() and t.get_device() == index >= 0:
        return t.data_ptr()
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.get_device() < 0 or index < 0:
        raise ValueError(f"{name}: must be a device tensor")
    raise ValueError(f"{name}: on device {t.get_device()}, expected {index}")


def _req_given(t, dtypes, shape, index, name):
    """_arg for an argument that cannot be None."""
    if t is None:
        raise TypeError(f"{name}: expected a tensor, got None")
    return _arg(t, dtypes, shape, index, name)


_empty = torch.empty_strided


def _new(shape, dtype, dev):
    """A new contiguous 1-D or 2-D tensor (the quickest of torch's constructors)."""
    return _empty(shape, (shape[1], 1) if len(shape) == 2 else (1,), dtype=dtype, device=dev)


_U8S, _I32S, _F32S = (_U8,), (torch.int32,), (torch.float32,)


def _matrix_dims(x):
    if x.dim() not in (2, 3):
        raise ValueError(f"x: expected [m, k] or [G, m, k], got {tuple(x.shape)}")
    return x.shape if x.dim() == 3 else (1, *x.shape)


def dg_quantize_mxfp4(x, q=None, sf=None, qt=None, sft=None, values=None):
    """x [m, k] or [G, m, k] (bf16 or fp32) -> MXFP4 (see include/dg.h).  Blocks along k: q [.., m, k/2] uint8 and
    sf [.., k/128, m] int32; blocks along m, transposed: qt [.., k, mp/2] and sft [.., mp/128, k], mp = m rounded up
    to 128; values [.., m, k] bf16: what q and sf stand for.  Outputs that are None are not computed."""
    G, m, k = _matrix_dims(x)
    lead, mb, dev = x.shape[:-2], (m + 127) // 128, x.get_device()
    xp = _arg(x, _X_TYPES, x.shape, dev, "x")
    _call("dg_quantize_mxfp4", dev, xp, _X_TYPES[x.dtype], _arg(q, _U8S, (*lead, m, k // 2), dev, "q"),
          _arg(sf, _I32S, (*lead, k // 128, m), dev, "sf"), _arg(qt, _U8S, (*lead, k, mb * 64), dev, "qt"),
          _arg(sft, _I32S, (*lead, mb, k), dev, "sft"), _arg(values, _BF, x.shape, dev, "values"), G, m, k)


def dg_mxfp4_gemm_workspace_bytes(m, n, k, num_cus=0):
    """Bytes of workspace dg_mxfp4_gemm_nt needs for these sizes (0: none)."""
    return int(lib().dg_mxfp4_gemm_workspace_bytes(m, n, k, int(num_cus)))


def _mxfp4_operands(a, a_sf, b, b_sf):
    """Checks the operands of an MXFP4 GEMM; returns (m, n, k, device index)."""
    m, kh = a.shape
    n, k, index = b.shape[0], 2 * kh, a.get_device()
    kb = k // 128
    if not (a.dtype is b.dtype is _U8 and a_sf.dtype is b_sf.dtype is torch.int32 and b.shape == (n, kh)
            and a_sf.shape == (kb, m) and b_sf.shape == (kb, n) and a.is_contiguous() and a_sf.is_contiguous()
            and b.is_contiguous() and b_sf.is_contiguous()
            and 0 <= index == a_sf.get_device() == b.get_device() == b_sf.get_device()):
        for t, dtypes, shape, name in ((a, _U8S, (m, kh), "a"), (a_sf, _I32S, (kb, m), "a_sf"), (b, _U8S, (n, kh), "b"),
                                       (b_sf, _I32S, (kb, n), "b_sf")):
            _arg(t, dtypes, shape, index, name)
    return m, n, k, index


def dg_mxfp4_gemm_nt(a, a_sf, b, b_sf, c, d, workspace=None):
    """d = c + a . b^T, both operands MXFP4: a [M, K/2] uint8, a_sf [K/128, M] int32, b [N, K/2], b_sf [K/128, N].
    workspace: optional uint8 device tensor (allocated here when needed and not given)."""
    m, n, k, index = _mxfp4_operands(a, a_sf, b, b_sf)
    cp, dp = _arg(c, _BF, (m, n), index, "c"), _arg(d, _BF, (m, n), index, "d")
    if workspace is None:
        nbytes, wp = (_lib or load_library()).dg_mxfp4_gemm_workspace_bytes(m, n, k, 0), None
        if nbytes:
            workspace = _new((nbytes,), _U8, a.device)
            wp = workspace.data_ptr()
    else:
        nbytes = workspace.numel()
        wp = _arg(workspace, _U8S, (nbytes,), index, "workspace")
    _call("dg_mxfp4_gemm_nt", index, a.data_ptr(), a_sf.data_ptr(), b.data_ptr(), b_sf.data_ptr(), cp, dp, m, n, k, wp,
          nbytes)
    return d


def dg_mxfp4_ragged_blocks(m, num_groups):
    """Blocks of 128 rows that any m rows in num_groups ragged groups need at most."""
    return int(lib().dg_mxfp4_ragged_blocks(m, num_groups))


def _groups(ms, index):
    """Checks the groups' row counts; returns their number and address."""
    if ms.dim() != 1:
        raise ValueError(f"ms: expected [num_groups], got {tuple(ms.shape)}")
    return ms.shape[0], _arg(ms, _I32S, ms.shape, index, "ms")


def dg_quantize_mxfp4_ragged(x, ms, q=None, sf=None, qt=None, sft=None):
    """x [m, k] (bf16 or fp32), its rows in groups of ms [G] int32 -> MXFP4 (see include/dg.h): qt [k, 64 B] and sft
    [B, k] in blocks along each group's rows, B = dg_mxfp4_ragged_blocks(m, G); q [m, k/2] and sf [k/128, m] or None."""
    m, k = x.shape
    dev = x.get_device()
    xp = _arg(x, _X_TYPES, x.shape, dev, "x")
    G, mp = _groups(ms, dev)
    blocks = dg_mxfp4_ragged_blocks(m, G)
    _call("dg_quantize_mxfp4_ragged", dev, xp, _X_TYPES[x.dtype], mp, _arg(q, _U8S, (m, k // 2), dev, "q"),
          _arg(sf, _I32S, (k // 128, m), dev, "sf"), _arg(qt, _U8S, (k, blocks * 64), dev, "qt"),
          _arg(sft, _I32S, (blocks, k), dev, "sft"), m, k, G)


def _ragged_operands(a, a_sf, b, b_sf, ms):
    """Checks the operands of dg_m_grouped_mxfp4_gemm_nt_ragged; returns (m, n, k, G, device index, ms' address)."""
    if b.dim() != 3:
        raise ValueError(f"b: expected [num_groups, n, k/2], got {tuple(b.shape)}")
    (m, kh), index = a.shape, a.get_device()
    G, mp = _groups(ms, index)
    n, kb = b.shape[1], kh // 64
    for t, dtypes, shape, name in ((a, _U8S, (m, kh), "a"), (a_sf, _I32S, (kb, m), "a_sf"), (b, _U8S, (G, n, kh), "b"),
                                   (b_sf, _I32S, (G, kb, n), "b_sf")):
        _arg(t, dtypes, shape, index, name)
    return m, n, 2 * kh, G, index, mp


def dg_m_grouped_mxfp4_gemm_nt_ragged(a, a_sf, b, b_sf, ms, d):
    """d[r] = a[r] . b[g]^T for the rows r of group g, ms [G] int32 rows a group one behind another; a [M, K/2],
    a_sf [K/128, M], b [G, N, K/2], b_sf [G, K/128, N], d [M, N] bf16 (rows behind the last group's are left)."""
    m, n, k, G, index, mp = _ragged_operands(a, a_sf, b, b_sf, ms)
    _call("dg_m_grouped_mxfp4_gemm_nt_ragged", index, a.data_ptr(), a_sf.data_ptr(), b.data_ptr(), b_sf.data_ptr(), mp,
          _req_given(d, _BF, (m, n), index, "d"), m, n, k, G)
    return d


def dg_k_grouped_mxfp4_gemm_nt_ragged(a, a_sf, b, b_sf, ms, d):
    """d[g] = a . b^T over the K blocks of group g: a [M, K/2] and b [N, K/2] with a_sf and b_sf as
    dg_quantize_mxfp4_ragged's qt and sft, ms [G] int32 the rows that they were made with; d [G, M, N] bf16."""
    m, n, k, index = _mxfp4_operands(a, a_sf, b, b_sf)
    G, mp = _groups(ms, index)
    _call("dg_k_grouped_mxfp4_gemm_nt_ragged", index, a.data_ptr(), a_sf.data_ptr(), b.data_ptr(), b_sf.data_ptr(), mp,
          _req_given(d, _BF, (G, m, n), index, "d"), m, n, k, G)
    return d


# dg_activation (include/dg.h); ACT_GATED is or-ed in
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACT_GATED = 0, 1, 2, 3, 4, 16


def _activation_columns(activation, n):
    """Columns of the output of a layer whose product has n."""
    if activation & ~ACT_GATED not in (ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH):
        raise ValueError(f"activation: expected one of the ACT_ values, ACT_GATED or-ed in or not, got {activation}")
    if not activation & ACT_GATED:
        return n
    if n % 2:
        raise ValueError(f"activation: a gated one halves the columns, got {n}")
    return n // 2


def dg_mxfp4_linear(a, a_sf, b, b_sf, bias, activation, residual, z, d, workspace=None):
    """d = residual + act(a . b^T + bias) (see include/dg.h): operands as dg_mxfp4_gemm_nt; bias [N] bf16 or None;
    residual, d [M, N] bf16 (gated: [M, N/2]), residual None or given; z [M, N] bf16, the pre-activation, or None.
    workspace: optional uint8 device tensor (allocated here when needed and not given)."""
    m, n, k, index = _mxfp4_operands(a, a_sf, b, b_sf)
    out = (m, _activation_columns(activation, n))
    ptrs = (_arg(bias, _BF, (n,), index, "bias"), activation, _arg(residual, _BF, out, index, "residual"),
            _arg(z, _BF, (m, n), index, "z"), _arg(d, _BF, out, index, "d"))
    if workspace is None:
        nbytes, wp = (_lib or load_library()).dg_mxfp4_gemm_workspace_bytes(m, n, k, 0), None
        if nbytes:
            workspace = _new((nbytes,), _U8, a.device)
            wp = workspace.data_ptr()
    else:
        nbytes = workspace.numel()
        wp = _arg(workspace, _U8S, (nbytes,), index, "workspace")
    _call("dg_mxfp4_linear", index, a.data_ptr(), a_sf.data_ptr(), b.data_ptr(), b_sf.data_ptr(), *ptrs, m, n, k, wp, nbytes)
    return d


def dg_activation_backward_workspace_bytes(m, n):
    return int(lib().dg_activation_backward_workspace_bytes(m, n))


def dg_activation_backward(dy, z, activation, dz=None, q=None, sf=None, qt=None, sft=None, dbias=None, workspace=None):
    """dz = dy * act'(z) (see include/dg.h) in the forms that are given: dz [m, n] bf16, q [m, n/2] and sf [n/128, m],
    qt [n, mp/2] and sft [mp/128, n] (mp = m rounded up to 128), and its column sums dbias [n] fp32.  dy [m, n] (gated:
    [m, n/2]), z [m, n] bf16 (None with ACT_NONE).  workspace: uint8 device tensor of at least
    dg_activation_backward_workspace_bytes(m, n) bytes (None where that is 0 or dbias is None)."""
    m, n = (dy if z is None else z).shape
    index, mb = dy.get_device(), (m + 127) // 128
    nbytes = 0 if workspace is None else workspace.numel()
    _call("dg_activation_backward", index, _arg(dy, _BF, (m, _activation_columns(activation, n)), index, "dy"),
          _arg(z, _BF, (m, n), index, "z"), activation, _arg(dz, _BF, (m, n), index, "dz"),
          _arg(q, _U8S, (m, n // 2), index, "q"), _arg(sf, _I32S, (n // 128, m), index, "sf"),
          _arg(qt, _U8S, (n, mb * 64), index, "qt"), _arg(sft, _I32S, (mb, n), index, "sft"),
          _arg(dbias, _F32S, (n,), index, "dbias"), m, n, _arg(workspace, _U8S, (nbytes,), index, "workspace"), nbytes)


def _check_format(quant_format):
    if quant_format not in (QUANT_E4M3_F32, QUANT_E4M3_UE8M0, QUANT_MXFP4):
        raise ValueError(f"quant_format: expected QUANT_E4M3_F32, QUANT_E4M3_UE8M0 or QUANT_MXFP4, got {quant_format}")


def dg_add_rms_norm(x, residual, weight, h, q, sf, eps, quant_format, rstd=None):
    """h = x + residual; q, sf = quantised h / rms(h) * weight (see include/dg.h).  x, residual, h [m, k] bf16 (residual
    and h may be None), weight [k]; q [m, k] uint8 and sf [k/128, m] fp32 (QUANT_E4M3_F32) or [m, ceil(k/512)] int32
    (QUANT_E4M3_UE8M0), or q [m, k/2] and sf [k/128, m] int32 (QUANT_MXFP4); rstd [m] fp32 or None."""
    m, k = x.shape
    _check_format(quant_format)
    shape, dev = (m, k), x.get_device()
    sf_shape = (m, _kw(k)) if quant_format == QUANT_E4M3_UE8M0 else (k // 128, m)
    _call("dg_add_rms_norm", dev, _arg(x, _BF, shape, dev, "x"), _arg(residual, _BF, shape, dev, "residual"),
          _arg(weight, _BF, (k,), dev, "weight"), _arg(h, _BF, shape, dev, "h"),
          _arg(q, _U8S, (m, k // 2) if quant_format == QUANT_MXFP4 else shape, dev, "q"),
          _arg(sf, _F32S if quant_format == QUANT_E4M3_F32 else _I32S, sf_shape, dev, "sf"), quant_format,
          _arg(rstd, _F32S, (m,), dev, "rstd"), m, k, eps)


def dg_add_rms_norm_backward_workspace_bytes(m, k):
    return int(lib().dg_add_rms_norm_backward_workspace_bytes(m, k))


def dg_add_rms_norm_backward(dy, dh, h, weight, rstd, dx, dweight, workspace=None):
    """dx [m, k] bf16 and dweight [k] fp32 from dy, dh (or None), h [m, k] bf16, weight [k] bf16 and the forward
    pass's rstd [m] (see include/dg.h).  workspace: uint8 device tensor of at least
    dg_add_rms_norm_backward_workspace_bytes(m, k) bytes (None where that is 0)."""
    m, k = dy.shape
    shape, dev = (m, k), dy.get_device()
    nbytes = 0 if workspace is None else workspace.numel()
    _call("dg_add_rms_norm_backward", dev, _arg(dy, _BF, shape, dev, "dy"), _arg(dh, _BF, shape, dev, "dh"),
          _arg(h, _BF, shape, dev, "h"), _arg(weight, _BF, (k,), dev, "weight"), _arg(rstd, _F32S, (m,), dev, "rstd"),
          _arg(dx, _BF, shape, dev, "dx"), _arg(dweight, _F32S, (k,), dev, "dweight"), m, k,
          _arg(workspace, _U8S, (nbytes,), dev, "workspace"), nbytes)


def _gate_shape(gate, gate_rows, m, k):
    """The gate's shape, and gate_rows as the C call takes it: an int there, so that m stands for every number beyond
    (their low 32 bits would be another number of gate rows)."""
    if gate is None:
        return None, 1
    if gate_rows < 1:
        raise ValueError(f"gate_rows: expected 1 or more, got {gate_rows}")
    gate_rows = min(gate_rows, max(m, 1))
    return ((m + gate_rows - 1) // gate_rows, k), gate_rows


def dg_sandwich_norm(x, residual, post_weight, gate, weight, h, q, sf, quant_format, rstd_x=None, rstd=None, gate_rows=1,
                     scale=1.0, eps=1e-6):
    """h = residual + scale * gate * norm(x) * post_weight; q, sf = quantised h / rms(h) * weight (see include/dg.h).
    x, residual, h [m, k] bf16; post_weight, weight [k] and gate [ceil(m / gate_rows), k] bf16 (post_weight and gate may
    be None); q, sf as dg_add_rms_norm; rstd_x, rstd [m] fp32 or None."""
    m, k = x.shape
    _check_format(quant_format)
    shape, dev, (gshape, gate_rows) = (m, k), x.get_device(), _gate_shape(gate, gate_rows, m, k)
    sf_shape = (m, _kw(k)) if quant_format == QUANT_E4M3_UE8M0 else (k // 128, m)
    _call("dg_sandwich_norm", dev, _arg(x, _BF, shape, dev, "x"), _arg(residual, _BF, shape, dev, "residual"),
          _arg(post_weight, _BF, (k,), dev, "post_weight"), _arg(gate, _BF, gshape, dev, "gate"),
          _arg(weight, _BF, (k,), dev, "weight"), _arg(h, _BF, shape, dev, "h"),
          _arg(q, _U8S, (m, k // 2) if quant_format == QUANT_MXFP4 else shape, dev, "q"),
          _arg(sf, _F32S if quant_format == QUANT_E4M3_F32 else _I32S, sf_shape, dev, "sf"), quant_format,
          _arg(rstd_x, _F32S, (m,), dev, "rstd_x"), _arg(rstd, _F32S, (m,), dev, "rstd"), m, k, gate_rows, scale, eps)


def dg_sandwich_norm_backward_workspace_bytes(m, k, with_post_weight=True, with_gate=True):
    return int(lib().dg_sandwich_norm_backward_workspace_bytes(m, k, int(with_post_weight), int(with_gate)))


def dg_sandwich_norm_backward(dy, dh, x, h, post_weight, gate, weight, rstd_x, rstd, dx, dresidual, dweight, dpost_weight,
                              dgate, workspace, gate_rows=1, scale=1.0):
    """dx, dresidual [m, k] bf16, dweight and dpost_weight [k] and dgate [ceil(m / gate_rows), k] fp32 of dg_sandwich_norm
    (see include/dg.h); dh may be None, post_weight, rstd_x and dpost_weight together, and gate and dgate.  workspace:
    uint8 device tensor of at least dg_sandwich_norm_backward_workspace_bytes(...) bytes."""
    m, k = dy.shape
    shape, dev, (gshape, gate_rows) = (m, k), dy.get_device(), _gate_shape(gate, gate_rows, m, k)
    nbytes = workspace.numel()
    _call("dg_sandwich_norm_backward", dev, _arg(dy, _BF, shape, dev, "dy"), _arg(dh, _BF, shape, dev, "dh"),
          _arg(x, _BF, shape, dev, "x"), _arg(h, _BF, shape, dev, "h"), _arg(post_weight, _BF, (k,), dev, "post_weight"),
          _arg(gate, _BF, gshape, dev, "gate"), _arg(weight, _BF, (k,), dev, "weight"),
          _arg(rstd_x, _F32S, (m,), dev, "rstd_x"), _arg(rstd, _F32S, (m,), dev, "rstd"), _arg(dx, _BF, shape, dev, "dx"),
          _arg(dresidual, _BF, shape, dev, "dresidual"), _arg(dweight, _F32S, (k,), dev, "dweight"),
          _arg(dpost_weight, _F32S, (k,), dev, "dpost_weight"), _arg(dgate, _F32S, gshape, dev, "dgate"), m, k, gate_rows,
          scale, _arg(workspace, _U8S, (nbytes,), dev, "workspace"), nbytes)


def dg_get_mk_alignment_for_contiguous_layout():
    return int(lib().dg_get_mk_alignment_for_contiguous_layout())


def dg_set_num_cus(n):
    _check("dg_set_num_cus", lib().dg_set_num_cus(int(n)))


def dg_get_num_cus():
    return int(lib().dg_get_num_cus())


def dg_query_plan(m, n, k, num_groups=1, num_cus=0):
    p = DgPlan()
    _check("dg_query_plan", lib().dg_query_plan(m, n, k, num_groups, num_cus, ctypes.byref(p)))
    return {f: getattr(p, f) for f, _ in DgPlan._fields_}


def dg_query_plan_contiguous(m, n, k, num_groups, num_cus=0):
    p = DgPlan()
    _check("dg_query_plan_contiguous",
           lib().dg_query_plan_contiguous(m, n, k, num_groups, num_cus, ctypes.byref(p)))
    return {f: getattr(p, f) for f, _ in DgPlan._fields_}


def dg_query_plan_form(form, m, n, k, num_groups=1, expected_m=0, num_cus=0):
    """The plan of a call of the given form (FORM_* constant)."""
    p = DgPlan()
    _check("dg_query_plan_form",
           lib().dg_query_plan_form(form, m, n, k, num_groups, expected_m, num_cus, ctypes.byref(p)))
    return {f: getattr(p, f) for f, _ in DgPlan._fields_}


def dg_num_tiles(m, n, block_m, block_n):
    return int(lib().dg_num_tiles(m, n, block_m, block_n))


# ----------------------------------------------------------------------------
# allocating conveniences (the pages' Python-style API)
# ----------------------------------------------------------------------------

def fp8_gemm_nt(a, sfa, b, sfb, c=None):
    """Returns a new bf16 tensor d = c + a . b^T."""
    d = torch.empty(a.shape[0], b.shape[0], dtype=torch.bfloat16, device=a.device)
    if c is not None and c.dtype == torch.int16:
        d = d.view(torch.int16)
    return dg_fp8_gemm_nt(a, sfa, b, sfb, c, d)


def m_grouped_fp8_gemm_nt_contiguous(a, sfa, b, sfb, m_indices, out=None):
    d = out if out is not None else torch.empty(a.shape[0], b.shape[1], dtype=torch.bfloat16, device=a.device)
    return dg_m_grouped_fp8_gemm_nt_contiguous(a, sfa, b, sfb, m_indices, d)


def m_grouped_fp8_gemm_nt_masked(a, sfa, b, sfb, masked_m, expected_m=0, out=None):
    d = out if out is not None else torch.empty(a.shape[0], a.shape[1], b.shape[1], dtype=torch.bfloat16,
                                                device=a.device)
    return dg_m_grouped_fp8_gemm_nt_masked(a, sfa, b, sfb, masked_m, d, expected_m)


def transform_weights_for_expert_ffn(l1_weights, l2_weights):
    """(w1, w1_sf), (w2, w2_sf) with row-major scale words -> the same pairs with the scale
    words K-block-major, the layout dg_fp8_fp4_expert_ffn reads; the E2M1 bytes are unchanged."""
    (w1, w1_sf), (w2, w2_sf) = l1_weights, l2_weights
    return (w1, dg_transform_fp4_weight_sf(w1_sf)), (w2, dg_transform_fp4_weight_sf(w2_sf))


def fp8_fp4_expert_ffn(x, x_sf, topk_idx, topk_w, w1, w1_sf, w2, w2_sf, expert_offset=0, workspace=None):
    T, H = x.shape
    E, I2 = w1.shape[0], w1.shape[1]
    nbytes = dg_fp8_fp4_expert_ffn_workspace_bytes(T, topk_idx.shape[1], E, H, I2 // 2)
    if workspace is None or workspace.numel() < nbytes:
        workspace = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=x.device)
    y = torch.empty(T, H, dtype=torch.bfloat16, device=x.device)
    return dg_fp8_fp4_expert_ffn(x, x_sf, topk_idx, topk_w, w1, w1_sf, w2, w2_sf, y, expert_offset, workspace)


# (The outputs made here need no checks: these call the C entry points themselves.)

def quantize_mxfp4(x, transposed=False, values=False):
    """MXFP4 of x [m, k] or [G, m, k] (bf16 or fp32): (q, sf), the operand whose products sum over k; with transposed,
    (q, sf, qt, sft), qt and sft the transposed operand, whose products sum over m; with values, also the bf16 values
    that q and sf stand for, as the last item."""
    shape = x.shape
    grouped = len(shape) != 2
    G, m, k = _matrix_dims(x) if grouped else (1, *shape)
    index, dev = x.get_device(), x.device
    xp = _arg(x, _X_TYPES, shape, index, "x")
    q, sf = _new((G * m, k // 2), _U8, dev), _new((G * (k // 128), m), torch.int32, dev)
    qt = sft = v = qtp = sftp = vp = None
    if transposed:
        mb = (m + 127) // 128
        qt, sft = _new((G * k, mb * 64), _U8, dev), _new((G * mb, k), torch.int32, dev)
        qtp, sftp = qt.data_ptr(), sft.data_ptr()
    if values:
        v = torch.empty_like(x, dtype=torch.bfloat16)
        vp = v.data_ptr()
    _call("dg_quantize_mxfp4", index, xp, _X_TYPES[x.dtype], q.data_ptr(), sf.data_ptr(), qtp, sftp, vp, G, m, k)
    out = (q, sf, qt, sft) if transposed else (q, sf)
    if grouped:
        out = tuple(t.view(G, -1, t.shape[1]) for t in out)
    return out if v is None else (*out, v)


def mxfp4_gemm_nt(a, a_sf, b, b_sf, c=None):
    """Returns a new bf16 tensor d = c + a . b^T, both operands MXFP4."""
    m, n, k, index = _mxfp4_operands(a, a_sf, b, b_sf)
    cp, dev = _arg(c, _BF, (m, n), index, "c"), a.device
    d = _new((m, n), torch.bfloat16, dev)
    nbytes, wp = (_lib or load_library()).dg_mxfp4_gemm_workspace_bytes(m, n, k, 0), None
    if nbytes:
        ws = _new((nbytes,), _U8, dev)
        wp = ws.data_ptr()
    _call("dg_mxfp4_gemm_nt", index, a.data_ptr(), a_sf.data_ptr(), b.data_ptr(), b_sf.data_ptr(), cp, d.data_ptr(), m, n,
          k, wp, nbytes)
    return d


def quantize_mxfp4_ragged(x, ms):
    """(q, sf, qt, sft) of x [m, k] (bf16 or fp32), whose rows lie in groups of ms [G] int32 (on the device): q and sf the
    operand of m_grouped_mxfp4_gemm_nt_ragged, qt and sft that of k_grouped_mxfp4_gemm_nt_ragged."""
    (m, k), index, dev = x.shape, x.get_device(), x.device
    xp = _arg(x, _X_TYPES, x.shape, index, "x")
    G, mp = _groups(ms, index)
    blocks = (_lib or load_library()).dg_mxfp4_ragged_blocks(m, G)
    q, sf = _new((m, k // 2), _U8, dev), _new((k // 128, m), torch.int32, dev)
    qt, sft = _new((k, blocks * 64), _U8, dev), _new((blocks, k), torch.int32, dev)
    _call("dg_quantize_mxfp4_ragged", index, xp, _X_TYPES[x.dtype], mp, q.data_ptr(), sf.data_ptr(), qt.data_ptr(),
          sft.data_ptr(), m, k, G)
    return q, sf, qt, sft


def m_grouped_mxfp4_gemm_nt_ragged(a, a_sf, b, b_sf, ms, out=None):
    """d [M, N] bf16 (a new tensor unless out is given): d[r] = a[r] . b[g]^T for the rows r of group g, ms [G] int32 rows
    a group.  Rows behind the last group's are left as they are (in a new tensor: undefined)."""
    m, n, k, G, index, mp = _ragged_operands(a, a_sf, b, b_sf, ms)
    d = _new((m, n), torch.bfloat16, a.device) if out is None else out
    dp = d.data_ptr() if out is None else _arg(out, _BF, (m, n), index, "out")
    _call("dg_m_grouped_mxfp4_gemm_nt_ragged", index, a.data_ptr(), a_sf.data_ptr(), b.data_ptr(), b_sf.data_ptr(), mp, dp,
          m, n, k, G)
    return d


def k_grouped_mxfp4_gemm_nt_ragged(a, a_sf, b, b_sf, ms, out=None):
    """d [G, M, N] bf16 (a new tensor unless out is given): d[g] = a . b^T over the rows of group g that qt and sft of
    quantize_mxfp4_ragged (of dy as a, of x as b, both with this ms) hold."""
    m, n, k, index = _mxfp4_operands(a, a_sf, b, b_sf)
    G, mp = _groups(ms, index)
    d = torch.empty(G, m, n, dtype=torch.bfloat16, device=a.device) if out is None else out
    dp = d.data_ptr() if out is None else _arg(out, _BF, (G, m, n), index, "out")
    _call("dg_k_grouped_mxfp4_gemm_nt_ragged", index, a.data_ptr(), a_sf.data_ptr(), b.data_ptr(), b_sf.data_ptr(), mp, dp,
          m, n, k, G)
    return d


def mxfp4_linear(a, a_sf, b, b_sf, bias=None, activation=ACT_NONE, residual=None, pre_activation=False):
    """Returns a new bf16 tensor d = residual + act(a . b^T + bias), both operands MXFP4 (activation: an ACT_ value,
    gated with ACT_GATED or-ed in); with pre_activation, (d, z), z = bf16(a . b^T + bias) for activation_backward."""
    m, n, k, index = _mxfp4_operands(a, a_sf, b, b_sf)
    out, dev = (m, _activation_columns(activation, n)), a.device
    bp, rp = _arg(bias, _BF, (n,), index, "bias"), _arg(residual, _BF, out, index, "residual")
    d, z = _new(out, torch.bfloat16, dev), _new((m, n), torch.bfloat16, dev) if pre_activation else None
    nbytes, wp = (_lib or load_library()).dg_mxfp4_gemm_workspace_bytes(m, n, k, 0), None
    if nbytes:
        ws = _new((nbytes,), _U8, dev)
        wp = ws.data_ptr()
    _call("dg_mxfp4_linear", index, a.data_ptr(), a_sf.data_ptr(), b.data_ptr(), b_sf.data_ptr(), bp, activation, rp,
          None if z is None else z.data_ptr(), d.data_ptr(), m, n, k, wp, nbytes)
    return d if z is None else (d, z)


def activation_backward(dy, z, activation, bias=True):
    """(q, sf, qt, sft, dbias): the gradient of a linear layer's pre-activation z from dy, quantised to MXFP4 along the
    rows and along the columns of the transposed operand, and its sums over the rows (fp32; None without bias).  z may be
    None with ACT_NONE."""
    m, n = (dy if z is None else z).shape
    index, dev, mb = dy.get_device(), dy.device, (m + 127) // 128
    yp = _arg(dy, _BF, (m, _activation_columns(activation, n)), index, "dy")
    zp = _arg(z, _BF, (m, n), index, "z")
    q, sf = _new((m, n // 2), _U8, dev), _new((n // 128, m), torch.int32, dev)
    qt, sft = _new((n, mb * 64), _U8, dev), _new((mb, n), torch.int32, dev)
    dbias, bp, nbytes, wp = None, None, 0, None
    if bias:
        dbias = _new((n,), torch.float32, dev)
        bp = dbias.data_ptr()
        nbytes = (_lib or load_library()).dg_activation_backward_workspace_bytes(m, n)
        if nbytes:
            ws = _new((nbytes,), _U8, dev)
            wp = ws.data_ptr()
    _call("dg_activation_backward", index, yp, zp, activation, None, q.data_ptr(), sf.data_ptr(), qt.data_ptr(),
          sft.data_ptr(), bp, m, n, wp, nbytes)
    return q, sf, qt, sft, dbias


def add_rms_norm(x, residual, weight, eps=1e-6, quant_format=QUANT_E4M3_F32):
    """(q, sf, h, rstd): the quantised norm of h = x + residual (residual None: h is x itself), with h and
    rstd = 1 / rms(h) for the residual stream and the backward pass."""
    m, k = x.shape
    _check_format(quant_format)
    shape, index, dev = (m, k), x.get_device(), x.device
    xp, rp = _arg(x, _BF, shape, index, "x"), _arg(residual, _BF, shape, index, "residual")
    wp = _arg(weight, _BF, (k,), index, "weight")
    q = _new((m, k // 2) if quant_format == QUANT_MXFP4 else shape, _U8, dev)
    if quant_format == QUANT_E4M3_UE8M0:
        sf = _new((m, _kw(k)), torch.int32, dev)
    else:
        sf = _new((k // 128, m), torch.float32 if quant_format == QUANT_E4M3_F32 else torch.int32, dev)
    rstd = _new((m,), torch.float32, dev)
    h, hp = x, None
    if residual is not None:
        h = torch.empty_like(x)
        hp = h.data_ptr()
    _call("dg_add_rms_norm", index, xp, rp, wp, hp, q.data_ptr(), sf.data_ptr(), quant_format, rstd.data_ptr(), m, k, eps)
    return q, sf, h, rstd


def add_rms_norm_backward(dy, dh, h, weight, rstd):
    """(dx, dweight) of add_rms_norm: dx bf16 is the gradient of x and of residual alike, dweight fp32."""
    m, k = dy.shape
    shape, index, dev = (m, k), dy.get_device(), dy.device
    ins = (_arg(dy, _BF, shape, index, "dy"), _arg(dh, _BF, shape, index, "dh"), _arg(h, _BF, shape, index, "h"),
           _arg(weight, _BF, (k,), index, "weight"), _arg(rstd, _F32S, (m,), index, "rstd"))
    dx, dweight = torch.empty_like(dy), _new((k,), torch.float32, dev)
    nbytes = (_lib or load_library()).dg_add_rms_norm_backward_workspace_bytes(m, k)
    wp = None
    if nbytes:
        ws = _new((nbytes,), _U8, dev)
        wp = ws.data_ptr()
    _call("dg_add_rms_norm_backward", index, *ins, dx.data_ptr(), dweight.data_ptr(), m, k, wp, nbytes)
    return dx, dweight


def sandwich_norm(x, residual, post_weight, gate, weight, scale=1.0, gate_rows=None, eps=1e-6,
                  quant_format=QUANT_E4M3_F32):
    """(q, sf, h, rstd_x, rstd): h = residual + scale * gate * norm(x) * post_weight and its quantised norm.  gate:
    [ceil(m / gate_rows), k] (gate_rows None: one row for all rows of x), or None; post_weight None: x is not normed, and
    rstd_x None."""
    m, k = x.shape
    _check_format(quant_format)
    shape, index, dev = (m, k), x.get_device(), x.device
    gshape, gate_rows = _gate_shape(gate, max(m, 1) if gate_rows is None else gate_rows, m, k)
    ins = (_arg(x, _BF, shape, index, "x"), _req_given(residual, _BF, shape, index, "residual"),
           _arg(post_weight, _BF, (k,), index, "post_weight"), _arg(gate, _BF, gshape, index, "gate"),
           _req_given(weight, _BF, (k,), index, "weight"))
    q = _new((m, k // 2) if quant_format == QUANT_MXFP4 else shape, _U8, dev)
    if quant_format == QUANT_E4M3_UE8M0:
        sf = _new((m, _kw(k)), torch.int32, dev)
    else:
        sf = _new((k // 128, m), torch.float32 if quant_format == QUANT_E4M3_F32 else torch.int32, dev)
    h, rstd = torch.empty_like(x), _new((m,), torch.float32, dev)
    rstd_x = None if post_weight is None else _new((m,), torch.float32, dev)
    _call("dg_sandwich_norm", index, *ins, h.data_ptr(), q.data_ptr(), sf.data_ptr(), quant_format,
          None if rstd_x is None else rstd_x.data_ptr(), rstd.data_ptr(), m, k, gate_rows, scale, eps)
    return q, sf, h, rstd_x, rstd


def sandwich_norm_backward(dy, dh, x, h, post_weight, gate, weight, rstd_x, rstd, scale=1.0, gate_rows=None):
    """(dx, dresidual, dweight, dpost_weight, dgate) of sandwich_norm: dx and dresidual bf16, the others fp32
    (dpost_weight and dgate None where post_weight and gate are)."""
    m, k = dy.shape
    shape, index, dev = (m, k), dy.get_device(), dy.device
    gshape, gate_rows = _gate_shape(gate, max(m, 1) if gate_rows is None else gate_rows, m, k)
    ins = (_arg(dy, _BF, shape, index, "dy"), _arg(dh, _BF, shape, index, "dh"), _req_given(x, _BF, shape, index, "x"),
           _req_given(h, _BF, shape, index, "h"), _arg(post_weight, _BF, (k,), index, "post_weight"),
           _arg(gate, _BF, gshape, index, "gate"), _req_given(weight, _BF, (k,), index, "weight"),
           _arg(rstd_x, _F32S, (m,), index, "rstd_x"), _req_given(rstd, _F32S, (m,), index, "rstd"))
    dx, dresidual, dweight = torch.empty_like(dy), torch.empty_like(dy), _new((k,), torch.float32, dev)
    dpost = None if post_weight is None else _new((k,), torch.float32, dev)
    dgate = None if gate is None else _new(gshape, torch.float32, dev)
    nbytes = (_lib or load_library()).dg_sandwich_norm_backward_workspace_bytes(m, k, dpost is not None, dgate is not None)
    ws = _new((nbytes,), _U8, dev)
    _call("dg_sandwich_norm_backward", index, *ins, dx.data_ptr(), dresidual.data_ptr(), dweight.data_ptr(),
          None if dpost is None else dpost.data_ptr(), None if dgate is None else dgate.data_ptr(), m, k, gate_rows, scale,
          ws.data_ptr(), nbytes)
    return dx, dresidual, dweight, dpost, dgate


def dg_status_string(status):
    return lib().dg_status_string(int(status)).decode()
