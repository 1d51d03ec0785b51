"""MXFP4 quantisation and GEMM on the GPU against the float64 oracle.

Quantisation is defined exactly (an exponent from comparisons, a rounding to nearest even), so its outputs must equal
the oracle's bit for bit.  GEMM tolerance, per element: the bf16 rounding, 2^-8 of the result, and the fp32
accumulation: an instruction adds its products in groups of eight (exact for E2M1 values of one scale: integers below
2^11 quarters), so a sum over K makes K/8 additions (and one for C), each off by at most 2^-23 of the partial sum's
magnitude, itself at most S = sum |a b| + |c|:  |D - ref| <= 2^-8 |ref| + (K/8 + 1) 2^-23 (1 + 2^-8) S.
"""

import numpy as np
import pytest
import torch

from oracle import mx as X
from oracle.formats import bf16_bits_to_f64, f64_to_bf16_bits
from tests.helpers import bits, check_bit_exact, sentinel_like

pytestmark = pytest.mark.gpu

GUARD = 64


def guarded(shape, dtype):
    """A tensor of shape inside a larger buffer filled with 0x5A; returns (tensor, check)."""
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((n + 2 * GUARD,), 0x5A, dtype=torch.uint8, device="cuda")

    def check():
        b = buf.cpu().numpy()
        assert (b[:GUARD] == 0x5A).all() and (b[GUARD + n:] == 0x5A).all(), "written outside the output"
    return buf[GUARD:GUARD + n].view(dtype).view(shape), check


def values(seed, *shape):
    """Normal values with channels of different size and rows of zeros, tiny and large magnitudes."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape, dtype=np.float32) * np.exp(rng.standard_normal(shape[-1], dtype=np.float32))
    flat = x.reshape(-1, shape[-1])
    for i, f in ((1, 0.0), (2, 1e-30), (3, 1e30), (4, 2.0 ** -125), (5, 2.0 ** -133)):
        if len(flat) > i:
            flat[i] *= f
    return x


def to_dev(x, dtype):
    t = torch.from_numpy(x).to(dtype)
    return t.cuda(), t.double().numpy()


def oracle_quantize(x3):
    """[G, m, k] float64 -> q, sf, values, qt, sft stacked over the groups."""
    parts = [X.quantize_mxfp4(g) + X.quantize_mxfp4_transposed(g) for g in x3]
    return [np.stack(p) for p in zip(*parts)]


def check_quantize(dgm, x, x64, want=("rows", "cols", "values")):
    shape = x.shape if x.dim() == 3 else (1, *x.shape)
    G, m, k = shape
    lead = x.shape[:-2]
    mb = (m + 127) // 128
    outs = dict(q=((*lead, m, k // 2), torch.uint8), sf=((*lead, k // 128, m), torch.int32),
                qt=((*lead, k, mb * 64), torch.uint8), sft=((*lead, mb, k), torch.int32),
                values=(tuple(x.shape), torch.bfloat16))
    keep = dict(q="rows", sf="rows", qt="cols", sft="cols", values="values")
    made = {n: guarded(*o) for n, o in outs.items() if keep[n] in want}
    dgm.dg_quantize_mxfp4(x, **{n: t for n, (t, _) in made.items()})
    torch.cuda.synchronize()
    q, sf, v, qt, sft = oracle_quantize(x64.reshape(shape))
    ref = dict(q=q, sf=sf, qt=qt, sft=sft)
    for n, (t, check) in made.items():
        check()
        if n == "values":
            got = bits(t).reshape(v.shape)
            nan = np.isnan(v)
            assert np.isnan(bf16_bits_to_f64(got[nan])).all()
            check_bit_exact(got[~nan], v[~nan], "values")
        else:
            got = t.cpu().numpy().reshape(ref[n].shape)
            assert np.array_equal(got, ref[n]), f"{n}: {np.count_nonzero(got != ref[n])} of {got.size} differ"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 128), (5, 7168), (130, 384), (128, 128), (2, 33, 256), (3, 257, 640), (300, 1664)])
def test_quantize_shapes(dg, shape, dtype):
    x, x64 = to_dev(values(sum(shape), *shape), dtype)
    check_quantize(dg, x, x64)


@pytest.mark.parametrize("want", [("rows",), ("cols",), ("values",), ("rows", "values"), ("cols", "values"),
                                  ("rows", "cols")])
def test_quantize_output_sets(dg, want):
    x, x64 = to_dev(values(3, 2, 70, 256), torch.bfloat16)
    check_quantize(dg, x, x64, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_edges(dg, dtype):
    """Midpoints between codes, borders of the exponent, all-zero blocks, signed zeros, infinities and NaN."""
    row = np.zeros(256, dtype=np.float32)
    mids = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    row[:15] = [6.0] + mids + [-m for m in mids]
    row[32:36] = [-0.0, 0.0, -1e-38, 1e-38]
    row[64], row[96], row[128] = 6.0, 6.03125, 2.0 ** -126
    x = np.stack([row * np.float32(2.0) ** s for s in (0, -3, 5, 90, -100)] * 26)      # 130 rows
    x[7, 3], x[8, 40], x[9, 200], x[129, 255] = np.nan, np.inf, -np.inf, np.nan
    t, x64 = to_dev(x, dtype)
    check_quantize(dg, t, x64)


def rand_mx(rng, r, k, lo=-3, hi=3):
    """Random codes and scale words (exponents lo..hi around 1)."""
    q = rng.integers(0, 256, (r, k // 2)).astype(np.uint8)
    byte = (127 + rng.integers(lo, hi + 1, (r, k // 32))).astype(np.uint8)
    return q, np.ascontiguousarray(X.pack_words(byte).T)


def run_gemm(dgm, a, sa, b, sb, c=None):
    m, n = a.shape[0], b.shape[0]
    t = [torch.from_numpy(v).cuda() for v in (a, sa, b, sb)]
    ct = None if c is None else torch.from_numpy(c.view(np.int16)).cuda().view(torch.bfloat16)
    d, check = guarded((m, n), torch.bfloat16)
    dgm.dg_mxfp4_gemm_nt(*t, ct, d)
    torch.cuda.synchronize()
    check()
    return bits(d)


def check_gemm(dgm, a, sa, b, sb, c=None):
    got = bf16_bits_to_f64(run_gemm(dgm, a, sa, b, sb, c))
    k = 2 * a.shape[1]
    av, bv = X.dequant_mxfp4(a, sa), X.dequant_mxfp4(b, sb)
    ref, s = av @ bv.T, np.abs(av) @ np.abs(bv).T
    if c is not None:
        cv = bf16_bits_to_f64(c)
        ref, s = ref + cv, s + np.abs(cv)
    bound = 2.0 ** -8 * np.abs(ref) + (k / 8 + 1) * 2.0 ** -23 * (1 + 2.0 ** -8) * s
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), f"{bad.sum()} of {bad.size} out of tolerance, first at {np.argwhere(bad)[0]}: " \
                          f"{got[bad][0]} against {ref[bad][0]} +- {bound[bad][0]}"


# sizes around every tile and split: one row to several tiles, partial tiles of both kinds, one K block to many (odd too)
SHAPES = [(1, 16, 128), (1, 4096, 1024), (3, 48, 384), (16, 272, 640), (17, 96, 2176), (33, 512, 896), (64, 1040, 512),
          (65, 128, 1280), (128, 256, 256), (130, 144, 384), (200, 528, 1152), (256, 512, 768), (257, 272, 1408),
          (300, 2112, 7168), (511, 784, 2048), (513, 1024, 128), (1030, 1296, 640)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm_shapes(dg, m, n, k):
    rng = np.random.default_rng(m * 7 + n + k)
    a, sa = rand_mx(rng, m, k)
    b, sb = rand_mx(rng, n, k)
    c = f64_to_bf16_bits(rng.standard_normal((m, n)) * 50) if (m + n // 16) % 2 else None
    check_gemm(dg, a, sa, b, sb, c)


@pytest.mark.parametrize("m,n,k", [(1, 272, 512), (40, 96, 1024), (130, 400, 512), (300, 512, 640), (700, 1040, 384)])
def test_gemm_exact_integers(dg, m, n, k):
    """Scales 1, codes of small integers and C an integer: every sum is an integer below 2^24 and D its bf16 rounding,
    bit for bit, whatever the order; one element of each row of A is marked so that a moved row or K index shows."""
    rng = np.random.default_rng(k + m)
    ints = np.array([0, 2, 4, 6, 10, 12], dtype=np.uint8)                # 0, 1, 2, 4, -1, -2
    ca, cb = (ints[rng.integers(0, 6, (r, k))] for r in (m, n))
    ca[np.arange(m), np.arange(m) * 37 % k] = 7                           # 6
    one = lambda r: np.full((k // 128, r), 0x7f7f7f7f, dtype=np.int32)    # noqa: E731
    c = f64_to_bf16_bits(rng.integers(-100, 101, (m, n)).astype(np.float64))
    a, b = X.pack_pairs(ca), X.pack_pairs(cb)
    check_bit_exact(run_gemm(dg, a, one(m), b, one(n), c), X.mxfp4_gemm_nt(a, one(m), b, one(n), c), "exact")


@pytest.mark.parametrize("kernel", [0, 1, 2, 3, 4, 5, 6, 7, 100, 101])
def test_gemm_every_kernel(dg, kernel, monkeypatch):
    """Each tile and each form for few rows pinned, over partial tiles, odd counts of K blocks, a split along K and
    (where units exceed the workgroups, with the CU cap) several tiles per workgroup; exact integers with C."""
    monkeypatch.setenv("DG_FORCE_MXFP4", str(kernel))
    ints = np.array([0, 2, 4, 6, 10, 12], dtype=np.uint8)
    rows = {100: (1, 16), 101: (17, 32)}.get(kernel, (1, 70, 200, 300))
    for m in rows:
        for n, k, cap in ((272, 128, 0), (528, 2176, 0), (400, 1152, 8)):
            dg.dg_set_num_cus(cap)
            try:
                rng = np.random.default_rng(m + n)
                ca, cb = (ints[rng.integers(0, 6, (r, k))] for r in (m, n))
                byte = [(127 + rng.integers(0, 2, (r, k // 32))).astype(np.uint8) for r in (m, n)]
                a, b = X.pack_pairs(ca), X.pack_pairs(cb)
                sa, sb = (np.ascontiguousarray(X.pack_words(v).T) for v in byte)
                c = f64_to_bf16_bits(rng.integers(-100, 101, (m, n)).astype(np.float64))
                check_bit_exact(run_gemm(dg, a, sa, b, sb, c), X.mxfp4_gemm_nt(a, sa, b, sb, c), f"{m} {n} {k}")
            finally:
                dg.dg_set_num_cus(0)


@pytest.mark.parametrize("m,n,k", [(3, 128, 512), (100, 272, 640), (600, 1040, 768)])
def test_gemm_every_scale_byte_counts(dg, m, n, k):
    """Codes 1.0 everywhere: D is the sum over 32-blocks of 32 * 2^(ea + eb); a power of two apart from block to
    block, so a scale taken from another row, block or byte changes the result."""
    rng = np.random.default_rng(n)
    one = lambda r: np.full((r, k // 2), 0x22, dtype=np.uint8)            # noqa: E731
    ba = (127 + rng.integers(-2, 3, (m, k // 32))).astype(np.uint8)
    bb = (127 + rng.integers(-2, 3, (n, k // 32))).astype(np.uint8)
    sa, sb = (np.ascontiguousarray(X.pack_words(v).T) for v in (ba, bb))
    check_bit_exact(run_gemm(dg, one(m), sa, one(n), sb), X.mxfp4_gemm_nt(one(m), sa, one(n), sb), "scales")


@pytest.mark.parametrize("m,n,k", [(2, 64, 1024), (140, 272, 512), (530, 528, 384)])
def test_gemm_nan_scales(dg, m, n, k):
    """An exponent byte 255 (codes 0, as the quantiser writes them) gives NaN in its row or column of D, no other."""
    rng = np.random.default_rng(1)
    a, sa = rand_mx(rng, m, k)
    b, sb = rand_mx(rng, n, k)
    i, j = m - 1, n - 3
    sa.view(np.uint8).reshape(k // 128, m, 4)[k // 128 - 1, i, 2] = 255
    a[i, k // 2 - 32:k // 2 - 16] = 0
    sb.view(np.uint8).reshape(k // 128, n, 4)[0, j, 0] = 255
    b[j, :16] = 0
    got = bf16_bits_to_f64(run_gemm(dg, a, sa, b, sb))
    nan = np.zeros((m, n), dtype=bool)
    nan[i], nan[:, j] = True, True
    assert np.array_equal(np.isnan(got), nan)


def test_gemm_extreme_exponents(dg):
    """Scales near the ends of the range whose products are ordinary numbers, and products past bf16's range."""
    rng = np.random.default_rng(2)
    a, sa = rand_mx(rng, 20, 256, 100, 110)
    b, sb = rand_mx(rng, 48, 256, -112, -100)
    check_gemm(dg, a, sa, b, sb)
    got = bf16_bits_to_f64(run_gemm(dg, np.full((4, 128), 0x77, np.uint8), np.full((2, 4), -0x01010102, np.int32),
                                    np.full((16, 128), 0x77, np.uint8), np.full((2, 16), 0x7f7f7f7f, np.int32)))
    assert np.isposinf(got).all()


def test_gemm_results_below_fp32_normals_are_zero(dg):
    """The matrix cores flush sums below 2^-126; just above it they are exact."""
    one = np.full((20, 128), 0x22, np.uint8)
    sf = lambda r, e: np.ascontiguousarray(X.pack_words(np.full((r, 8), 127 + e, np.uint8)).T)      # noqa: E731
    for ea, eb, want in ((-60, -74, 2.0 ** -126), (-60, -90, 0.0), (-127, -127, 0.0)):               # 256 * 2^(ea + eb)
        got = bf16_bits_to_f64(run_gemm(dg, one, sf(20, ea), one[:16], sf(16, eb)))
        assert (got == want).all(), (ea, eb, got[0, 0])


def test_gemm_in_place_c(dg):
    rng = np.random.default_rng(4)
    for m, n, k in ((5, 256, 1024), (300, 528, 512)):
        a, sa = rand_mx(rng, m, k)
        b, sb = rand_mx(rng, n, k)
        t = [torch.from_numpy(v).cuda() for v in (a, sa, b, sb)]
        c = torch.randn(m, n, device="cuda").to(torch.bfloat16)
        want = dg.mxfp4_gemm_nt(*t, c)
        dg.dg_mxfp4_gemm_nt(*t, c, c)
        assert torch.equal(c, want)


@pytest.mark.parametrize("m,n,k,kernel", [(1, 4096, 7168, None), (64, 2112, 7168, None), (200, 4096, 2048, None),
                                          (512, 512, 8192, "2"), (300, 7168, 16384, "3")])
def test_gemm_repeats_bit_for_bit_and_graph_replays(dg, m, n, k, kernel, monkeypatch):
    if kernel:                                            # a tile that splits along K at this size
        monkeypatch.setenv("DG_FORCE_MXFP4", kernel)
        assert kernel == "3" or dg.dg_mxfp4_gemm_workspace_bytes(m, n, k) > 0
    rng = np.random.default_rng(9)
    t = [torch.from_numpy(v).cuda() for v in rand_mx(rng, m, k) + rand_mx(rng, n, k)]
    want = dg.mxfp4_gemm_nt(*t)
    need = dg.dg_mxfp4_gemm_workspace_bytes(m, n, k)
    ws = torch.full((max(need, 1),), 0xff, dtype=torch.uint8, device="cuda")   # its contents on entry are ignored
    d = torch.empty_like(want)
    dg.dg_mxfp4_gemm_nt(*t, None, d, ws)
    assert torch.equal(d, want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        dg.dg_mxfp4_gemm_nt(*t, None, d, ws)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dg.dg_mxfp4_gemm_nt(*t, None, d, ws)
    for i in range(4):
        d.fill_(float("nan"))
        ws.fill_(i)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, want), f"replay {i}"


def test_gemm_refuses_a_small_workspace(dg, monkeypatch):
    monkeypatch.setenv("DG_FORCE_MXFP4", "2")             # 16 tiles of 128x128, split along K
    m, n, k = 512, 512, 8192
    need = dg.dg_mxfp4_gemm_workspace_bytes(m, n, k)
    assert need > 0
    t = [torch.from_numpy(v).cuda() for v in rand_mx(np.random.default_rng(0), m, k) + rand_mx(np.random.default_rng(1), n, k)]
    d = sentinel_like((m, n)).view(torch.bfloat16)
    with pytest.raises(dg.DgError):
        dg.dg_mxfp4_gemm_nt(*t, None, d, torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert (bits(d) == 0xFFFF).all()


def test_two_streams_at_once(dg):
    """Two calls in flight together, each with a workspace of its own."""
    rng = np.random.default_rng(12)
    shapes = [(256, 1024, 4096), (64, 4096, 4096)]
    ts = [[torch.from_numpy(v).cuda() for v in rand_mx(rng, m, k) + rand_mx(rng, n, k)] for m, n, k in shapes]
    want = [dg.mxfp4_gemm_nt(*t) for t in ts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for _ in range(5):
        for t, s in zip(ts, streams):
            with torch.cuda.stream(s):
                got.append(dg.mxfp4_gemm_nt(*t))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        assert torch.equal(g, want[i % 2])


def test_training_step_of_a_linear_layer(dg):
    """y, dx and dw of one layer from the quantiser's operands, against the oracle's quantisation and products."""
    T, N, K = 150, 256, 384
    x, x64 = to_dev(values(21, T, K) * 0 + np.random.default_rng(1).standard_normal((T, K), dtype=np.float32), torch.bfloat16)
    w, w64 = to_dev(np.random.default_rng(2).standard_normal((N, K), dtype=np.float32), torch.bfloat16)
    dy, dy64 = to_dev(np.random.default_rng(3).standard_normal((T, N), dtype=np.float32), torch.bfloat16)
    xq, xs, xqt, xst = dg.quantize_mxfp4(x, transposed=True)
    wq, ws, wqt, wst = dg.quantize_mxfp4(w, transposed=True)
    yq, ys, yqt, yst = dg.quantize_mxfp4(dy, transposed=True)
    qv = lambda v: X.quantize_mxfp4(v)[2]                                                  # noqa: E731
    qt = lambda v: X.dequant_mxfp4(*X.quantize_mxfp4_transposed(v))                        # noqa: E731
    for got, a, b, k in ((dg.mxfp4_gemm_nt(xq, xs, wq, ws), qv(x64), qv(w64), K),
                         (dg.mxfp4_gemm_nt(yq, ys, wqt, wst), qv(dy64), qt(w64), N),
                         (dg.mxfp4_gemm_nt(yqt, yst, xqt, xst), qt(dy64), qt(x64), 256)):
        ref, s = a @ b.T, np.abs(a) @ np.abs(b).T
        err = np.abs(bf16_bits_to_f64(bits(got)) - ref)
        assert (err <= 2.0 ** -8 * np.abs(ref) + (k / 8 + 1) * 2.0 ** -23 * (1 + 2.0 ** -8) * s).all()


def test_quantized_weights_feed_the_expert_ffn(dg):
    """q and sf of expert weights are what the FP8 x FP4 entry points read: the FFN's result is bit for bit that on
    the generator's operands."""
    import synth
    E, H, I, T, topk = 2, 512, 256, 24, 2
    g = synth.gen_ffn(T=T, H=H, I=I, num_local=E, num_experts=4, topk=topk, seed=31)
    rng = np.random.default_rng(31)
    w1 = torch.from_numpy(rng.standard_normal((E, 2 * I, H), dtype=np.float32))
    w2 = torch.from_numpy(rng.standard_normal((E, H, I), dtype=np.float32))
    t = [g[n].cuda() for n in ("x", "x_sf", "topk_idx", "topk_w")]
    own = [v for w in (w1, w2) for v in dg.quantize_mxfp4(w.cuda())]
    gen = []
    for w in (w1, w2):
        p, s = zip(*[synth.quant_fp4_1x32(e) for e in w])
        gen += [torch.stack(p).cuda(), dg.dg_transform_fp4_weight_sf(torch.stack(s).cuda())]
    assert all(torch.equal(a, b) for a, b in zip(own, gen))
    assert torch.equal(dg.fp8_fp4_expert_ffn(*t, *own), dg.fp8_fp4_expert_ffn(*t, *gen))


@pytest.mark.parametrize("k", [2 ** 31 - 512, 2 ** 31 - 384, 2 ** 31 - 128])
def test_quantize_longest_row(dg, k):
    """The longest rows: codes and scales equal those of the row quantised piece by piece."""
    x = torch.randn(k // 16, device="cuda").to(torch.bfloat16).repeat(16).view(1, k)
    x[0, k - 77] = 1000.0
    q, sf = dg.quantize_mxfp4(x)
    step = 1 << 27
    for a in range(0, k, step):
        b = min(a + step, k)
        pq, psf = dg.quantize_mxfp4(x[:, a:b])
        assert torch.equal(q[:, a // 2:b // 2], pq) and torch.equal(sf[a // 128:b // 128], psf), a


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantize_near_the_largest_number(dg, dtype):
    """Blocks with a magnitude above 1.5 * 2^127 have the exponent 126; from 1.75 * 2^127 on the nearest code is 4, which
    stands for 2^128: infinity in the bf16 values, the largest finite exponent in the scale."""
    x = values(17, 40, 256)
    top = np.float32(2.0) ** 127
    for i, f in enumerate((1.5, 1.5078125, 1.7421875, 1.75, 1.7578125, 1.9921875)):
        x[i, 32 * i] = f * top
        x[i + 10, 32 * i + 5] = -f * top
    x[30, 3] = np.finfo(np.float32).max if dtype == torch.float32 else 1.9921875 * top
    t, x64 = to_dev(x, dtype)
    assert np.isfinite(x64).all()
    check_quantize(dg, t, x64)
    v = dg.quantize_mxfp4(t, values=True)[2].double().cpu().numpy()
    assert np.array_equal(np.isinf(v), np.abs(x64) >= 1.75 * 2.0 ** 127) and not np.isnan(v).any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("want", [("rows",), ("cols",), ("values",), ("rows", "values"), ("rows", "cols", "values")])
@pytest.mark.parametrize("shape", [(3, 257, 640), (1500, 1152), (2, 40, 4224)])
def test_quantize_more_tiles_than_workgroups(dg, shape, want, dtype):
    """Several tiles per workgroup: the LDS areas are used again and later tiles' groups, rows and columns decoded."""
    x, x64 = to_dev(values(sum(shape), *shape), dtype)
    dg.dg_set_num_cus(1)                                  # 8 workgroups of tiles, 64 of row blocks
    try:
        check_quantize(dg, x, x64, want)
    finally:
        dg.dg_set_num_cus(0)
