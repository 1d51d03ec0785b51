"""The operators around the block-scaled GEMMs, as cases that can be timed and compared.

Four operators: quantisation to MXFP4 (E2M1 codes with a power-of-two scale per 32 values), the MXFP4 x MXFP4
GEMM, RMS norm with the residual's addition and a quantised output, and that norm's backward pass.  ``run`` computes
a case either in plain torch operations (``own`` false) or with the library's kernels (``own`` true).

Formats (those of ``include/dg.h``):
  E2M1 pairs     uint8 [..., K/2], element 2i in the low nibble of byte i; magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6
  MX scales      int32 [..., K/128, rows], byte i of a word is the UE8M0 exponent (bias 127) of values 32i .. 32i+31
                 of that 128-wide K block; the smallest exponent e with 6 * 2^e >= amax, 0 where amax is 0
  e4m3, fp32     one scale amax / 448 per row and 128-wide block, fp32 [K/128, rows]
  e4m3, UE8M0    the smallest power of two with 448 * 2^e >= amax, bytes [rows, 4 * ceil(K/512)]
"""

import math

import torch

own = False

EPS = 1e-6
DEV = "cuda"


# ----------------------------------------------------------------------------
# the cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # the activations of a few decoded tokens rounded to MXFP4 and back (quantisation-aware evaluation)
        dict(name="quantize_tokens", op="quantize", groups=1, m=5, k=7168, fp32=False),
        # two experts' first weights, fp32 masters, quantised before a serving run; the values for the QAT forward pass
        dict(name="quantize_weights", op="quantize", groups=2, m=4096, k=7168, fp32=True),
        # one decoded token through a 4-bit linear layer: the smallest call, bound by latency and the weight stream
        dict(name="linear_1", op="linear", m=1, n=4096, k=7168, with_c=False),
        # a decode batch over a wide projection with a short K
        dict(name="linear_64", op="linear", m=64, n=24576, k=1536, with_c=False),
        # an odd number of prompt tokens, a width that is no multiple of 128, added onto an output that is there
        dict(name="linear_ragged", op="linear", m=1111, n=2112, k=7168, with_c=True),
        # a long prompt through the largest layer: bound by the matrix cores
        dict(name="linear_4096", op="linear", m=4096, n=7168, k=16384, with_c=False),
        # one training step of a linear layer: forward, input gradient, weight gradient, each operand quantised along
        # the axis that its product sums over
        dict(name="linear_train", op="train", m=4001, n=4096, k=7168),
        # the norm in front of a decode step's FP8 GEMM (fp32 scales)
        dict(name="norm_3", op="norm", m=3, k=7168, scales="f32", residual=True),
        # the norm in front of a prompt's expert layer (packed power-of-two scales)
        dict(name="norm_8192", op="norm", m=8192, k=7168, scales="ue8m0", residual=True),
        # norm, 4-bit activations and 4-bit weights in a row, as a layer of a prompt runs them
        dict(name="norm_linear", op="norm_linear", m=200, n=4096, k=7168),
        # the norm's backward pass in a training step
        dict(name="norm_back_4096", op="norm_back", m=4096, k=7168, with_dh=True),
        # the same for a short sequence, without a gradient from the residual branch
        dict(name="norm_back_130", op="norm_back", m=130, k=2048, with_dh=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "train", "norm", "norm_linear", "norm_back"])
    k = 128 * _log(rng, 1, 64)
    m = _log(rng, 1, 6000)
    if op == "quantize":
        return dict(op=op, groups=rng.randint(1, 3), m=m, k=k, fp32=rng.random() < 0.5)
    if op == "linear":
        return dict(op=op, m=m, n=16 * _log(rng, 1, 800), k=k, with_c=rng.random() < 0.5)
    if op == "train":
        return dict(op=op, m=m, n=128 * _log(rng, 1, 40), k=128 * _log(rng, 1, 56))
    if op == "norm":
        return dict(op=op, m=m, k=k, scales=rng.choice(["f32", "ue8m0"]), residual=rng.random() < 0.7)
    if op == "norm_linear":
        return dict(op=op, m=m, n=16 * _log(rng, 1, 512), k=k)
    return dict(op=op, m=m, k=k, with_dh=rng.random() < 0.7)


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    if op == "quantize":      # values in; codes, scales and the bf16 values they stand for out
        e = case["groups"] * m * k
        return dict(bytes=e * (4 if case["fp32"] else 2) + e * (0.5 + 1 / 32 + 2), flops=0)
    if op == "linear":        # bf16 rows in, 4-bit weights in, bf16 out
        n = case["n"]
        return dict(bytes=2 * m * k + n * k * (0.5 + 1 / 32) + 2 * m * n * (2 if case["with_c"] else 1),
                    flops=2 * m * n * k)
    if op == "train":         # x, w, dy in; y, dx, dw out
        n = case["n"]
        return dict(bytes=4 * (m * k + n * k + m * n), flops=6 * m * n * k)
    if op == "norm":          # x, residual in; h, codes, scales, 1/rms out
        r = case["residual"]
        return dict(bytes=m * k * (2 + (4 if r else 0) + 1) + m * k // 128 * (4 if case["scales"] == "f32" else 1)
                    + 4 * m + 2 * k, flops=0)
    if op == "norm_linear":
        n = case["n"]
        return dict(bytes=6 * m * k + 2 * k + n * k * (0.5 + 1 / 32) + 2 * m * n, flops=2 * m * n * k)
    return dict(bytes=m * k * (8 if case["with_dh"] else 6) + 6 * k + 4 * m, flops=0)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _activations(g, *shape):
    """Normal values whose channels differ in size (a few of them by much), as a residual stream's do."""
    scale = torch.exp(0.5 * torch.randn(shape[-1], generator=g, device=DEV))
    scale = torch.where(torch.rand(shape[-1], generator=g, device=DEV) < 0.005, scale * 12, scale)
    return torch.randn(*shape, generator=g, device=DEV) * scale


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op, m, k = case["op"], case["m"], case["k"]
    s = dict(case)
    if op == "quantize":
        w = _activations(g, case["groups"], m, k)
        s["x"] = w if case["fp32"] else w.to(torch.bfloat16)
        return s
    if op in ("linear", "norm_linear"):
        n = case["n"]
        # the layer's weights, quantised once when they were loaded
        s["wq"], s["wsf"] = _quantize(0.02 * torch.randn(n, k, generator=g, device=DEV))[:2]
    if op == "linear":
        s["x"] = _activations(g, m, k).to(torch.bfloat16)
        s["c"] = torch.randn(m, n, generator=g, device=DEV).to(torch.bfloat16) if case["with_c"] else None
    elif op == "train":
        n = case["n"]
        s["x"] = _activations(g, m, k).to(torch.bfloat16)
        s["w"] = (0.02 * torch.randn(n, k, generator=g, device=DEV)).to(torch.bfloat16)
        s["dy"] = (1e-3 * _activations(g, m, n)).to(torch.bfloat16)
    elif op in ("norm", "norm_linear"):
        s["x"] = _activations(g, m, k).to(torch.bfloat16)
        s["residual"] = _activations(g, m, k).to(torch.bfloat16) if case.get("residual", True) else None
        s["weight"] = (1 + 0.2 * torch.randn(k, generator=g, device=DEV)).to(torch.bfloat16)
    elif op == "norm_back":
        s["dy"] = (1e-3 * torch.randn(m, k, generator=g, device=DEV)).to(torch.bfloat16)
        s["dh"] = (1e-3 * torch.randn(m, k, generator=g, device=DEV)).to(torch.bfloat16) if case["with_dh"] else None
        s["h"] = _activations(g, m, k).to(torch.bfloat16)
        s["weight"] = (1 + 0.2 * torch.randn(k, generator=g, device=DEV)).to(torch.bfloat16)
        # kept by the forward pass
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(dim=1) + EPS)
    return s


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------

def _exponent(amax, qmax):
    """The smallest e with qmax * 2^e >= amax, within UE8M0's -127 .. 127; 0 where amax is 0, 128 where it is not finite."""
    f, x = torch.frexp(amax)
    fq, xq = math.frexp(qmax)
    e = torch.where(f <= fq, x - xq, x - xq + 1).clamp(-127, 127)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    return torch.where(torch.isfinite(amax), e, torch.full_like(e, 128))


def _pow2(e):
    """2^e in fp32 (e = 128: NaN, the value of exponent byte 255)."""
    v = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e.clamp(max=127))
    return torch.where(e > 127, torch.full_like(v, float("nan")), v)


def _round_e2m1(v):
    """fp32 -> the nearest E2M1 value, ties to the even code (the grid steps by .5, 1 and 2)."""
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, v)


def _nibble(q):
    """E2M1 value -> its 4-bit code."""
    a = q.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.int32)
    return code + 8 * torch.signbit(q)


def _quantize(x):
    """[..., rows, K] -> E2M1 pairs, scale words [..., K/128, rows], and the values they stand for (fp32)."""
    rows, k = x.shape[-2:]
    b = x.float().view(*x.shape[:-1], k // 32, 32)
    e = _exponent(b.abs().amax(dim=-1), 6.0)
    ok = (e < 128)[..., None]
    q = torch.where(ok, _round_e2m1(torch.ldexp(b, -e[..., None])), 0.0)
    values = (q * _pow2(e)[..., None]).view(x.shape)
    code = _nibble(q).view(*x.shape[:-1], k // 2, 2)
    packed = (code[..., 0] | code[..., 1] << 4).to(torch.uint8)
    return packed, _words((e + 127).view(*x.shape[:-1], k // 128, 4)).transpose(-1, -2).contiguous(), values


def _words(byte):
    """Exponent bytes [..., 4] -> int32 words, byte i from the least significant end."""
    return byte[..., 0] | byte[..., 1] << 8 | byte[..., 2] << 16 | byte[..., 3] << 24


def _dequantize(q, sf):
    """E2M1 pairs [rows, K/2] and words [K/128, rows] -> fp32 [rows, K]."""
    rows, k = q.shape[0], 2 * q.shape[1]
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=q.device)
    v = table[torch.stack([q & 15, q >> 4], dim=-1).int()].view(rows, k // 32, 32)
    byte = torch.stack([sf >> (8 * i) & 255 for i in range(4)], dim=-1)          # [K/128, rows, 4]
    e = byte.transpose(0, 1).reshape(rows, k // 32, 1) - 127
    return (v * _pow2(e)).view(rows, k)


def _rms(h, weight):
    rstd = torch.rsqrt(h.square().mean(dim=-1) + EPS)
    return rstd, h * rstd[:, None] * weight.float()


def _add(s):
    if s["residual"] is None:
        return s["x"]
    return (s["x"].float() + s["residual"].float()).to(torch.bfloat16)


def _quantize_e4m3(y, scales):
    """fp32 [rows, K] -> e4m3 codes and their scales."""
    rows, k = y.shape
    b = y.view(rows, k // 128, 128)
    amax = b.abs().amax(dim=-1)
    if scales == "f32":
        sf = torch.where(amax > 0, (amax / 448.0).clamp(min=2.0 ** -126), 1.0)
        return (b / sf[..., None]).to(torch.float8_e4m3fn).view(rows, k), sf.t().contiguous()
    e = _exponent(amax, 448.0)
    q = torch.ldexp(b, -e[..., None]).to(torch.float8_e4m3fn).view(rows, k)
    e = torch.cat([e, e.new_zeros(rows, -e.shape[1] % 4)], dim=1)                # the last word's unused bytes: 2^0
    return q, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _run_plain(s):
    op = s["op"]
    if op == "quantize":
        q, sf, values = _quantize(s["x"])
        return dict(q=q, sf=sf, values=values.to(torch.bfloat16))
    if op == "linear":
        y = _quantize(s["x"])[2] @ _dequantize(s["wq"], s["wsf"]).t()
        return (y if s["c"] is None else y + s["c"].float()).to(torch.bfloat16)
    if op == "train":
        x, w, dy = s["x"], s["w"], s["dy"]
        pad = -s["m"] % 128                                                      # whole blocks along the tokens
        xt, dyt = (torch.nn.functional.pad(t, (0, 0, 0, pad)).t().contiguous() for t in (x, dy))
        y = _quantize(x)[2] @ _quantize(w)[2].t()
        dx = _quantize(dy)[2] @ _quantize(w.t().contiguous())[2].t()
        dw = _quantize(dyt)[2] @ _quantize(xt)[2].t()
        return tuple(t.to(torch.bfloat16) for t in (y, dx, dw))
    if op == "norm":
        h = _add(s)
        rstd, y = _rms(h.float(), s["weight"])
        q, sf = _quantize_e4m3(y, s["scales"])
        return dict(q=q, sf=sf, h=h, rstd=rstd)
    if op == "norm_linear":
        h = _add(s)
        _, y = _rms(h.float(), s["weight"])
        return dict(h=h, y=(_quantize(y)[2] @ _dequantize(s["wq"], s["wsf"]).t()).to(torch.bfloat16))
    dy, n = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
    gr = dy * s["weight"].float()
    dx = s["rstd"][:, None] * (gr - n * (gr * n).mean(dim=1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return dict(dx=dx.to(torch.bfloat16), dweight=(dy * n).sum(dim=0))


# ----------------------------------------------------------------------------
# the library's calls
# ----------------------------------------------------------------------------

def _run_own(s):
    import fp4_gemm_dense_amd as dg
    op = s["op"]
    if op == "quantize":
        q, sf, values = dg.quantize_mxfp4(s["x"], values=True)
        return dict(q=q, sf=sf, values=values)
    if op == "linear":
        q, sf = dg.quantize_mxfp4(s["x"])
        return dg.mxfp4_gemm_nt(q, sf, s["wq"], s["wsf"], s["c"])
    if op == "train":
        xq, xsf, xqt, xsft = dg.quantize_mxfp4(s["x"], transposed=True)
        wq, wsf, wqt, wsft = dg.quantize_mxfp4(s["w"], transposed=True)
        dyq, dysf, dyqt, dysft = dg.quantize_mxfp4(s["dy"], transposed=True)
        return (dg.mxfp4_gemm_nt(xq, xsf, wq, wsf), dg.mxfp4_gemm_nt(dyq, dysf, wqt, wsft),
                dg.mxfp4_gemm_nt(dyqt, dysft, xqt, xsft))
    if op == "norm":
        fmt = dg.QUANT_E4M3_F32 if s["scales"] == "f32" else dg.QUANT_E4M3_UE8M0
        q, sf, h, rstd = dg.add_rms_norm(s["x"], s["residual"], s["weight"], EPS, fmt)
        if s["scales"] != "f32":
            sf = sf.view(torch.float8_e8m0fnu)
        return dict(q=q.view(torch.float8_e4m3fn), sf=sf, h=h, rstd=rstd)
    if op == "norm_linear":
        q, sf, h, _ = dg.add_rms_norm(s["x"], s["residual"], s["weight"], EPS, dg.QUANT_MXFP4)
        return dict(h=h, y=dg.mxfp4_gemm_nt(q, sf, s["wq"], s["wsf"]))
    dx, dweight = dg.add_rms_norm_backward(s["dy"], s["dh"], s["h"], s["weight"], s["rstd"])
    return dict(dx=dx, dweight=dweight)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------

def _snap64(x, block, grid):
    """float64 [rows, K] -> the nearest points of grid * 2^e, e the least integer for which the block's largest
    magnitude is on or below grid's largest; ties to the even place in the grid."""
    rows, k = x.shape
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    out = torch.empty_like(x)
    for r in range(0, rows, 512):
        b = x[r:r + 512].reshape(-1, block)
        big = b.abs().amax(dim=1, keepdim=True)
        e = torch.ceil(torch.log2(torch.where(big > 0, big, 1.0) / grid[-1]))
        e = torch.where(grid[-1] * torch.exp2(e - 1) >= big, e - 1, e)           # log2 may be off by a rounding
        e = torch.where(grid[-1] * torch.exp2(e) < big, e + 1, e)
        unit = torch.exp2(torch.where(big > 0, e, 0.0).clamp(-127, 127))
        a = b.abs() / unit
        up = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
        dn = (up - 1).clamp(min=0)
        over, under = grid[up] - a, a - grid[dn]
        near = torch.where((over < under) | ((over == under) & (up % 2 == 0)), grid[up], grid[dn])
        out[r:r + 512] = (torch.sign(b) * near * unit).view(-1, k)
    return out


_E2M1 = [0, .5, 1, 1.5, 2, 3, 4, 6]
_E4M3 = [m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def _mx64(x):
    return _snap64(x.double(), 32, _E2M1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"]
        return dict(q=None, sf=None, values=_mx64(x.reshape(-1, x.shape[-1])).view(x.shape))
    if op == "linear":
        y = _mx64(s["x"]) @ _unpack64(s["wq"], s["wsf"]).t()
        return y if s["c"] is None else y + s["c"].double()
    if op == "train":
        x, w, dy = s["x"].double(), s["w"].double(), s["dy"].double()
        full = (s["m"] + 127) // 128 * 128
        xt, dyt = x.new_zeros(case["k"], full), x.new_zeros(case["n"], full)
        xt[:, :s["m"]], dyt[:, :s["m"]] = x.t(), dy.t()
        return _mx64(x) @ _mx64(w).t(), _mx64(dy) @ _mx64(w.t().contiguous()).t(), _mx64(dyt) @ _mx64(xt).t()
    if op == "norm_back":
        h, dy, w, r = (s[t].double() for t in ("h", "dy", "weight", "rstd"))
        inner = torch.einsum("ij,j,ij->i", dy, w, h) / case["k"]
        dx = r[:, None] * dy * w - (r ** 3 * inner)[:, None] * h
        return dict(dx=dx if s["dh"] is None else dx + s["dh"].double(), dweight=torch.einsum("ij,ij,i->j", dy, h, r))
    # h is stored in bf16, and what follows reads the stored one
    h = s["x"].double() if s["residual"] is None else (s["x"].double() + s["residual"].double()).to(torch.bfloat16).double()
    rstd = 1 / torch.sqrt((h * h).sum(dim=1) / case["k"] + EPS)
    y = h * rstd[:, None] * s["weight"].double()
    if op == "norm_linear":
        return dict(h=h, y=_mx64(y) @ _unpack64(s["wq"], s["wsf"]).t())
    rows, blocks = case["m"], case["k"] // 128
    if case["scales"] == "f32":
        b = y.view(rows, blocks, 128)
        sf = b.abs().amax(dim=2) / 448
        sf = torch.where(sf > 0, sf.clamp(min=2.0 ** -126), 1.0)
        code = (b / sf[..., None]).clamp(-448, 448)
        grid = torch.tensor(_E4M3, dtype=torch.float64, device=y.device)
        up = torch.searchsorted(grid, code.abs()).clamp(max=len(grid) - 1)
        dn = (up - 1).clamp(min=0)
        over, under = grid[up] - code.abs(), code.abs() - grid[dn]
        near = torch.where((over < under) | ((over == under) & (up % 2 == 0)), grid[up], grid[dn])
        return dict(q=(torch.sign(code) * near).view(rows, -1), sf=sf.t().contiguous(), h=h, rstd=rstd)
    amax = y.view(rows, blocks, 128).abs().amax(dim=2)
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, 1.0) / 448))
    e = torch.where(448 * torch.exp2(e - 1) >= amax, e - 1, e)
    e = torch.where(448 * torch.exp2(e) < amax, e + 1, e)
    sf = torch.exp2(torch.where(amax > 0, e, 0.0))
    values = _snap64(y, 128, _E4M3)
    full = torch.ones(rows, (blocks + 3) // 4 * 4, dtype=torch.float64, device=y.device)
    full[:, :blocks] = sf
    return dict(q=(values.view(rows, blocks, 128) / sf[..., None]).view(rows, -1), sf=full, h=h, rstd=rstd)


def _unpack64(q, sf):
    """The 4-bit weights' values, read nibble by nibble."""
    rows, k = q.shape[0], 2 * q.shape[1]
    v = torch.empty(rows, k, dtype=torch.float64, device=q.device)
    for half, code in ((0, (q & 15).long()), (1, (q >> 4).long())):
        mag = torch.tensor(_E2M1, dtype=torch.float64, device=q.device)[code & 7]
        v[:, half::2] = torch.where(code >= 8, -mag, mag)
    for i in range(4):
        unit = torch.exp2(((sf.long() >> (8 * i)) & 255).double() - 127).t()       # [rows, K/128]
        v.view(rows, k // 128, 4, 32)[:, :, i] *= unit[..., None]
    return v
