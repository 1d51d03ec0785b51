"""The operators of a transformer block whose linear layers run in MXFP4, as cases that can be timed and compared.

Three families: the MXFP4 linear layer with bias, activation (gated or not) and residual in its epilogue, and the
gradient of its activation; the MXFP4 products grouped by expert with ragged sizes, in every direction of a training
step; and the norms behind and in front of a block with the block's gate, residual scale and quantised output, forward
and backward.  ``run`` computes a case either in plain torch operations (``own`` false) or with the library's kernels.

Formats (those of ``include/dg.h``):
  E2M1 pairs     uint8 [..., K/2], element 2i in the low nibble of byte i; magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6
  MX scales      int32 [..., K/128, rows], byte i of a word is the UE8M0 exponent (bias 127) of values 32i .. 32i+31
                 of that 128-wide K block; the smallest exponent e with 6 * 2^e >= amax, 0 where amax is 0
  e4m3, fp32     one scale amax / 448 per row and 128-wide block, fp32 [K/128, rows]
  e4m3, UE8M0    the smallest power of two with 448 * 2^e >= amax, bytes [rows, 4 * ceil(K/512)]
"""

import math
import random

import torch

own = False

EPS = 1e-6
DEV = "cuda"


# ----------------------------------------------------------------------------
# the cases
# ----------------------------------------------------------------------------

def listed():
    return [
        # one decoded token through a projection with a bias: the smallest call
        dict(name="linear_1", op="linear", m=1, n=4096, k=7168, act="gelu_tanh", gated=False, residual=False, z=False),
        # an odd number of prompt tokens through a block's last projection, added onto the residual stream
        dict(name="linear_ragged", op="linear", m=1111, n=2112, k=7168, act="none", gated=False, residual=True, z=False),
        # the gated first projection of a long prompt's feed-forward block: bound by the matrix cores
        dict(name="linear_gated_4096", op="linear", m=4096, n=16384, k=7168, act="silu", gated=True, residual=False, z=True),
        # a training step's way back through a linear layer with an erf GELU and a bias
        dict(name="linear_back_2001", op="linear_back", m=2001, n=4096, k=7168, act="gelu", gated=False),
        # the same of a gated projection, for a short sequence
        dict(name="linear_back_130", op="linear_back", m=130, n=4096, k=2048, act="silu", gated=True),
        # a decode batch's rows over an expert layer, a few each and some experts with none: the weights' stream
        dict(name="experts_decode", op="experts", m=64, n=4096, k=7168, groups=32, skew=1.0),
        # a prompt's rows over the experts
        dict(name="experts_prompt", op="experts", m=8192, n=4096, k=7168, groups=8, skew=0.3),
        # a training step of an expert layer: forward, input gradient and every expert's weight gradient
        dict(name="experts_train", op="experts_train", m=4000, n=4096, k=2048, groups=8, skew=0.5),
        # the norms between two blocks of a decode step, in front of an FP8 GEMM
        dict(name="sandwich_3", op="sandwich", m=3, k=7168, scales="f32", gate_rows=1 << 30),
        # the same for a prompt of four sequences with a gate each
        dict(name="sandwich_8192", op="sandwich", m=8192, k=7168, scales="ue8m0", gate_rows=2048),
        # their backward pass in a training step, a gate for each sequence
        dict(name="sandwich_back_4096", op="sandwich_back", m=4096, k=7168, gate_rows=1024),
        # the same for a short sequence and one gate for all rows
        dict(name="sandwich_back_130", op="sandwich_back", m=130, k=2048, gate_rows=1 << 30),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_back", "experts", "experts", "experts_train", "sandwich", "sandwich_back"])
    m, k = _log(rng, 1, 4096), 128 * _log(rng, 1, 56)
    act, gated = rng.choice(["none", "relu", "silu", "gelu", "gelu_tanh"]), rng.random() < 0.4
    if op == "linear":
        return dict(op=op, m=m, n=32 * _log(rng, 1, 512), k=k, act=act, gated=gated, residual=rng.random() < 0.5,
                    z=rng.random() < 0.3)
    if op == "linear_back":
        return dict(op=op, m=m, n=256 * _log(rng, 1, 28), k=k, act=act, gated=gated)
    if op == "experts":
        return dict(op=op, m=_log(rng, 1, 8192), n=16 * _log(rng, 1, 256), k=k, groups=rng.randint(1, 40),
                    skew=rng.uniform(0, 2))
    if op == "experts_train":
        return dict(op=op, m=m, n=128 * _log(rng, 1, 32), k=128 * _log(rng, 1, 16), groups=rng.randint(1, 12),
                    skew=rng.uniform(0, 2))
    gate_rows = rng.choice([1, _log(rng, 2, 1024), 1 << 30])
    if op == "sandwich":
        return dict(op=op, m=m, k=k, scales=rng.choice(["f32", "ue8m0"]), gate_rows=gate_rows)
    return dict(op=op, m=m, k=k, gate_rows=gate_rows)


def _gates(case):
    return -(-case["m"] // case["gate_rows"])


def work(case):
    op, m, k = case["op"], case["m"], case["k"]
    q = 0.5 + 1 / 32                                                             # bytes of an MXFP4 value
    if op == "linear":        # 4-bit rows and weights, bias and residual in; d and the pre-activation out
        n, out = case["n"], case["n"] // 2 if case["gated"] else case["n"]
        return dict(bytes=(m + n) * k * q + 2 * n + 2 * m * out * (2 if case["residual"] else 1) + (2 * m * n if case["z"] else 0),
                    flops=2 * m * n * k)
    if op == "linear_back":   # dy, z and the saved 4-bit operands in; dx, dw, dbias out
        n, out = case["n"], case["n"] // 2 if case["gated"] else case["n"]
        return dict(bytes=2 * m * (out + n) + (m * k + n * k) * q + 2 * (m * k + n * k) + 4 * n, flops=4 * m * n * k)
    if op == "experts":       # the weights of the experts that have rows (at most one for each row)
        n = case["n"]
        return dict(bytes=(m + min(m, case["groups"]) * n) * k * q + 2 * m * n, flops=2 * m * n * k)
    if op == "experts_train":  # x, w, dy in; y, dx, dw out
        n = case["n"]
        return dict(bytes=4 * (m * k + case["groups"] * n * k + m * n), flops=6 * m * n * k)
    if op == "sandwich":      # x, residual in; h, codes, scales, both 1/rms out
        return dict(bytes=m * k * (6 + 1) + m * k // 128 * (4 if case["scales"] == "f32" else 1) + 8 * m
                    + 2 * k * (2 + _gates(case)), flops=0)
    # dy, dh, x, h in; dx, dresidual and three weight gradients out
    return dict(bytes=12 * m * k + 8 * m + 12 * k + 6 * k * _gates(case), flops=0)


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------

def _activations(g, *shape):
    """Normal values whose channels differ in size (a few of them by much), as a residual stream's do."""
    scale = torch.exp(0.5 * torch.randn(shape[-1], generator=g, device=DEV))
    scale = torch.where(torch.rand(shape[-1], generator=g, device=DEV) < 0.005, scale * 12, scale)
    return torch.randn(*shape, generator=g, device=DEV) * scale


def _weights(g, *shape):
    return shape[-1] ** -0.5 * torch.randn(*shape, generator=g, device=DEV)


def _sizes(case, seed):
    """Rows of each expert: unequal shares of m, some of them none."""
    rng = random.Random(seed)
    p = [math.exp(case["skew"] * rng.gauss(0, 1)) for _ in range(case["groups"])]
    ends = [round(case["m"] * sum(p[:g + 1]) / sum(p)) for g in range(case["groups"])]
    return [e - b for b, e in zip([0] + ends, ends)]


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op, m, k = case["op"], case["m"], case["k"]
    bf = torch.bfloat16
    s = dict(case)
    if op in ("linear", "linear_back"):
        n = case["n"]
        out = n // 2 if case["gated"] else n
        x, w = _activations(g, m, k), _weights(g, n, k)
    if op == "linear":
        # the weights, quantised when they were loaded, and the rows as the norm in front left them
        s["wq"], s["wsf"] = _quantize(w)[:2]
        s["xq"], s["xsf"] = _quantize(x)[:2]
        s["bias"] = (0.2 * torch.randn(n, generator=g, device=DEV)).to(bf)
        s["res"] = _activations(g, m, out).to(bf) if case["residual"] else None
    elif op == "linear_back":
        # what the forward pass keeps: the transposed operands and the pre-activation
        s["wqt"], s["wsft"] = _quantize(w.t().contiguous())[:2]
        s["xqt"], s["xsft"] = _quantize(_padded(x).t().contiguous())[:2]
        s["z"] = (1.5 * torch.randn(m, n, generator=g, device=DEV)).to(bf)
        s["dy"] = (1e-3 * _activations(g, m, out)).to(bf)
    elif op in ("experts", "experts_train"):
        n, groups = case["n"], case["groups"]
        s["sizes"] = _sizes(case, seed)
        s["ms"] = torch.tensor(s["sizes"], dtype=torch.int32, device=DEV)
        x = _activations(g, m, k)
        if op == "experts":
            s["xq"], s["xsf"] = _quantize(x)[:2]
            s["wq"] = torch.empty(groups, n, k // 2, dtype=torch.uint8, device=DEV)
            s["wsf"] = torch.empty(groups, k // 128, n, dtype=torch.int32, device=DEV)
            for e in range(groups):
                s["wq"][e], s["wsf"][e] = _quantize(_weights(g, n, k))[:2]
        else:
            s["x"], s["w"] = x.to(bf), _weights(g, groups, n, k).to(bf)
            s["dy"] = (1e-3 * _activations(g, m, n)).to(bf)
    else:
        s["gate_rows"] = min(case["gate_rows"], m)
        s["scale"] = 0.7
        s["x"] = _activations(g, m, k).to(bf)
        s["residual"] = _activations(g, m, k).to(bf)
        s["post_weight"] = (1 + 0.2 * torch.randn(k, generator=g, device=DEV)).to(bf)
        s["weight"] = (1 + 0.2 * torch.randn(k, generator=g, device=DEV)).to(bf)
        s["gate"] = torch.tanh(torch.randn(_gates(case), k, generator=g, device=DEV)).to(bf)
        if op == "sandwich_back":
            # kept by the forward pass
            s["h"] = _block_output(s)[1]
            s["rstd_x"] = torch.rsqrt(s["x"].float().square().mean(dim=1) + EPS)
            s["rstd"] = torch.rsqrt(s["h"].float().square().mean(dim=1) + EPS)
            s["dy"] = (1e-3 * torch.randn(m, k, generator=g, device=DEV)).to(bf)
            s["dh"] = (1e-3 * torch.randn(m, k, generator=g, device=DEV)).to(bf)
    return s


# ----------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------

def _exponent(amax, qmax):
    """The smallest e with qmax * 2^e >= amax, within UE8M0's -127 .. 127; 0 where amax is 0."""
    f, x = torch.frexp(amax)
    fq, xq = math.frexp(qmax)
    e = torch.where(f <= fq, x - xq, x - xq + 1).clamp(-127, 127)
    return torch.where(amax > 0, e, torch.zeros_like(e))


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
    """[rows, K] -> E2M1 pairs, scale words [K/128, rows], and the values they stand for (fp32)."""
    rows, k = x.shape
    b = x.float().view(rows, k // 32, 32)
    e = _exponent(b.abs().amax(dim=-1), 6.0)
    q = _round_e2m1(torch.ldexp(b, -e[..., None]))
    code = _nibble(q).view(rows, k // 2, 2)
    byte = (e + 127).view(rows, k // 128, 4)
    words = byte[..., 0] | byte[..., 1] << 8 | byte[..., 2] << 16 | byte[..., 3] << 24
    return (code[..., 0] | code[..., 1] << 4).to(torch.uint8), words.t().contiguous(), torch.ldexp(q, e[..., None]).view(rows, k)


def _dequantize(q, sf):
    """E2M1 pairs [rows, K/2] and words [K/128, rows] -> fp32 [rows, K]."""
    rows, k = q.shape[0], 2 * q.shape[1]
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=q.device)
    v = table[torch.stack([q & 15, q >> 4], dim=-1).int()].view(rows, k // 32, 32)
    byte = torch.stack([sf >> (8 * i) & 255 for i in range(4)], dim=-1)          # [K/128, rows, 4]
    return torch.ldexp(v, byte.transpose(0, 1).reshape(rows, k // 32, 1) - 127).view(rows, k)


def _padded(x):
    """Rows to whole blocks of 128, with zeros."""
    return torch.nn.functional.pad(x, (0, 0, 0, -x.shape[0] % 128))


_TANH = math.sqrt(2 / math.pi)


def _act(u, act):
    if act == "relu":
        return u.clamp(min=0)
    if act == "silu":
        return u / (1 + torch.exp(-u))
    if act == "gelu":
        return 0.5 * u * torch.erfc(-u / math.sqrt(2))
    if act == "gelu_tanh":
        return u / (1 + torch.exp(-2 * _TANH * (u + 0.044715 * u * u * u)))
    return u


def _act_gradient(u, act):
    if act == "relu":
        return (u > 0).float()
    if act == "silu":
        s = 1 / (1 + torch.exp(-u))
        return s * (1 + u * (1 - s))
    if act == "gelu":
        return 0.5 * torch.erfc(-u / math.sqrt(2)) + u * torch.exp(-0.5 * u * u) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        s = 1 / (1 + torch.exp(-2 * _TANH * (u + 0.044715 * u * u * u)))
        return s + u * s * (1 - s) * 2 * _TANH * (1 + 3 * 0.044715 * u * u)
    return torch.ones_like(u)


def _rms(h, weight):
    rstd = torch.rsqrt(h.square().mean(dim=-1) + EPS)
    return rstd, h * rstd[:, None] * weight.float()


def _gate_of_rows(s, gate):
    return gate.repeat_interleave(s["gate_rows"], dim=0)[:s["m"]]


def _block_output(s):
    """1/rms of x, and h = residual + scale * gate * norm(x); in 64 bits, for h next to a border of bf16."""
    rstd, y = _rms(s["x"].double(), s["post_weight"])
    h = s["residual"].double() + s["scale"] * _gate_of_rows(s, s["gate"].double()) * y
    return rstd.float(), h.to(torch.bfloat16)


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
    op, bf = s["op"], torch.bfloat16
    if op == "linear":
        u = _dequantize(s["xq"], s["xsf"]) @ _dequantize(s["wq"], s["wsf"]).t() + s["bias"].float()
        half = s["n"] // 2
        y = _act(u[:, :half], s["act"]) * u[:, half:] if s["gated"] else _act(u, s["act"])
        y = (y if s["res"] is None else y + s["res"].float()).to(bf)
        return dict(y=y, z=u.to(bf)) if s["z"] else dict(y=y)
    if op == "linear_back":
        dy, z, half = s["dy"].float(), s["z"].float(), s["n"] // 2
        if s["gated"]:
            gate, up = z[:, :half], z[:, half:]
            dz = torch.cat([dy * up * _act_gradient(gate, s["act"]), dy * _act(gate, s["act"])], dim=1)
        else:
            dz = dy * _act_gradient(z, s["act"])
        dzb = dz.to(bf)
        dx = _quantize(dzb)[2] @ _dequantize(s["wqt"], s["wsft"]).t()
        dw = _quantize(_padded(dzb).t().contiguous())[2] @ _dequantize(s["xqt"], s["xsft"]).t()
        return dict(dx=dx.to(bf), dw=dw.to(bf), dbias=dz.sum(dim=0))
    if op == "experts":
        x = _dequantize(s["xq"], s["xsf"])
        return torch.cat([xe @ _dequantize(wq, wsf).t() for xe, wq, wsf in
                          zip(x.split(s["sizes"]), s["wq"], s["wsf"]) if len(xe)]).to(bf)
    if op == "experts_train":
        parts = [_expert_step(*t) for t in zip(s["x"].split(s["sizes"]), s["w"], s["dy"].split(s["sizes"]))]
        y, dx, dw = zip(*parts)
        return dict(y=torch.cat(y).to(bf), dx=torch.cat(dx).to(bf), dw=torch.stack(dw).to(bf))
    if op == "sandwich":
        rstd_x, h = _block_output(s)
        rstd, y = _rms(h.float(), s["weight"])
        q, sf = _quantize_e4m3(y, s["scales"])
        return dict(q=q, sf=sf, h=h, rstd_x=rstd_x, rstd=rstd)
    dy, dh, w, pw = (s[t].float() for t in ("dy", "dh", "weight", "post_weight"))
    nh, nx = s["h"].float() * s["rstd"][:, None], s["x"].float() * s["rstd_x"][:, None]
    gr = dy * w
    dres = dh + s["rstd"][:, None] * (gr - nh * (gr * nh).mean(dim=1, keepdim=True))
    v = dres * s["scale"] * _gate_of_rows(s, s["gate"].float())
    gr = v * pw
    dx = s["rstd_x"][:, None] * (gr - nx * (gr * nx).mean(dim=1, keepdim=True))
    share = s["scale"] * dres * nx * pw
    share = torch.nn.functional.pad(share, (0, 0, 0, -s["m"] % s["gate_rows"]))   # whole groups of gate_rows
    dgate = share.view(len(s["gate"]), s["gate_rows"], -1).sum(dim=1)
    return dict(dx=dx.to(bf), dresidual=dres.to(bf), dweight=(dy * nh).sum(dim=0), dpost_weight=(v * nx).sum(dim=0),
                dgate=dgate)


def _expert_step(x, w, dy):
    """One expert's y, dx and dw, each product's operands quantised along the axis that it sums over."""
    wq, wqt = _quantize(w)[2], _quantize(w.t().contiguous())[2]
    xt, dyt = (_quantize(_padded(t).t().contiguous())[2] if len(t) else t.t().float() for t in (x, dy))
    return _quantize(x)[2] @ wq.t(), _quantize(dy)[2] @ wqt.t(), dyt @ xt.t()


# ----------------------------------------------------------------------------
# the library's calls
# ----------------------------------------------------------------------------

def _run_own(s):
    import fp4_gemm_dense_amd as dg
    op = s["op"]
    if op in ("linear", "linear_back"):
        act = dict(none=dg.ACT_NONE, relu=dg.ACT_RELU, silu=dg.ACT_SILU, gelu=dg.ACT_GELU, gelu_tanh=dg.ACT_GELU_TANH)[s["act"]]
        act |= dg.ACT_GATED if s["gated"] else 0
    if op == "linear":
        if s["z"]:
            y, z = dg.mxfp4_linear(s["xq"], s["xsf"], s["wq"], s["wsf"], s["bias"], act, s["res"], pre_activation=True)
            return dict(y=y, z=z)
        return dict(y=dg.mxfp4_linear(s["xq"], s["xsf"], s["wq"], s["wsf"], s["bias"], act, s["res"]))
    if op == "linear_back":
        q, sf, qt, sft, dbias = dg.activation_backward(s["dy"], s["z"], act)
        return dict(dx=dg.mxfp4_gemm_nt(q, sf, s["wqt"], s["wsft"]), dw=dg.mxfp4_gemm_nt(qt, sft, s["xqt"], s["xsft"]),
                    dbias=dbias)
    if op == "experts":
        return dg.m_grouped_mxfp4_gemm_nt_ragged(s["xq"], s["xsf"], s["wq"], s["wsf"], s["ms"])
    if op == "experts_train":
        ms = s["ms"]
        wq, wsf, wqt, wsft = dg.quantize_mxfp4(s["w"], transposed=True)
        xq, xsf, xqt, xsft = dg.quantize_mxfp4_ragged(s["x"], ms)
        dyq, dysf, dyqt, dysft = dg.quantize_mxfp4_ragged(s["dy"], ms)
        return dict(y=dg.m_grouped_mxfp4_gemm_nt_ragged(xq, xsf, wq, wsf, ms),
                    dx=dg.m_grouped_mxfp4_gemm_nt_ragged(dyq, dysf, wqt, wsft, ms),
                    dw=dg.k_grouped_mxfp4_gemm_nt_ragged(dyqt, dysft, xqt, xsft, ms))
    if op == "sandwich":
        fmt = dg.QUANT_E4M3_F32 if s["scales"] == "f32" else dg.QUANT_E4M3_UE8M0
        q, sf, h, rstd_x, rstd = dg.sandwich_norm(s["x"], s["residual"], s["post_weight"], s["gate"], s["weight"], s["scale"],
                                                  s["gate_rows"], EPS, fmt)
        if s["scales"] != "f32":
            sf = sf.view(torch.float8_e8m0fnu)
        return dict(q=q.view(torch.float8_e4m3fn), sf=sf, h=h, rstd_x=rstd_x, rstd=rstd)
    dx, dres, dweight, dpost, dgate = dg.sandwich_norm_backward(
        s["dy"], s["dh"], s["x"], s["h"], s["post_weight"], s["gate"], s["weight"], s["rstd_x"], s["rstd"], s["scale"],
        s["gate_rows"])
    return dict(dx=dx, dresidual=dres, dweight=dweight, dpost_weight=dpost, dgate=dgate)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------

_E2M1 = [0, .5, 1, 1.5, 2, 3, 4, 6]
_E4M3 = [m * 2.0 ** -9 for m in range(8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)][:-1]


def _nearest(a, grid):
    """|values| -> the nearest points of grid, ties to the even place in it."""
    up = torch.searchsorted(grid, a).clamp(max=len(grid) - 1)
    dn = (up - 1).clamp(min=0)
    over, under = grid[up] - a, a - grid[dn]
    return torch.where((over < under) | ((over == under) & (up % 2 == 0)), grid[up], grid[dn])


def _unit(big, top):
    """The least power of two that top times it is on or above big (1 where big is 0)."""
    e = torch.ceil(torch.log2(torch.where(big > 0, big, 1.0) / top))
    e = torch.where(top * torch.exp2(e - 1) >= big, e - 1, e)                    # log2 may be off by a rounding
    e = torch.where(top * torch.exp2(e) < big, e + 1, e)
    return torch.exp2(torch.where(big > 0, e, 0.0).clamp(-127, 127))


def _snap64(x, block, grid):
    """float64 [rows, K] -> the nearest points of each block's grid."""
    rows, k = x.shape
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    out = torch.empty_like(x)
    for r in range(0, rows, 512):
        b = x[r:r + 512].reshape(-1, block)
        unit = _unit(b.abs().amax(dim=1, keepdim=True), grid[-1])
        out[r:r + 512] = (torch.sign(b) * _nearest(b.abs() / unit, grid) * unit).view(-1, k)
    return out


def _mx64(x):
    return _snap64(x.double(), 32, _E2M1)


def _mx64t(x):
    """The transposed operand: [rows, c] -> [c, rows up to whole blocks]."""
    rows, c = x.shape
    full = torch.zeros(c, (rows + 127) // 128 * 128, dtype=torch.float64, device=x.device)
    full[:, :rows] = x.double().t()
    return _mx64(full)


def _unpack64(q, sf):
    """4-bit values read nibble by nibble."""
    rows, k = q.shape[0], 2 * q.shape[1]
    v = torch.empty(rows, k, dtype=torch.float64, device=q.device)
    mag = torch.tensor(_E2M1, dtype=torch.float64, device=q.device)
    for half, code in ((0, (q & 15).long()), (1, (q >> 4).long())):
        v[:, half::2] = torch.where(code >= 8, -mag[code & 7], mag[code & 7])
    for i in range(4):
        unit = torch.exp2(((sf.long() >> (8 * i)) & 255).double() - 127).t()       # [rows, K/128]
        v.view(rows, k // 128, 4, 32)[:, :, i] *= unit[..., None]
    return v


def _act64(u, act):
    """act(u) and its derivative."""
    one = torch.ones_like(u)
    if act == "none":
        return u, one
    if act == "relu":
        on = torch.where(u > 0, one, 0.0)
        return u * on, on
    if act == "gelu":
        phi = torch.special.ndtr(u)
        return u * phi, phi + u * torch.exp(-u * u / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        s = torch.sigmoid(u)
        return u * s, s + u * s * torch.sigmoid(-u)
    t = torch.tanh(_TANH * (u + 0.044715 * u ** 3))
    return 0.5 * u * (1 + t), 0.5 * (1 + t) + 0.5 * u * (1 - t * t) * _TANH * (1 + 3 * 0.044715 * u ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    op, m, k = case["op"], case["m"], case["k"]
    if op == "linear":
        u = torch.einsum("ij,kj->ik", _unpack64(s["xq"], s["xsf"]), _unpack64(s["wq"], s["wsf"])) + s["bias"].double()
        if case["gated"]:
            g, up = torch.chunk(u, 2, dim=1)
            y = _act64(g, case["act"])[0] * up
        else:
            y = _act64(u, case["act"])[0]
        if s["res"] is not None:
            y = y + s["res"].double()
        return dict(y=y, z=u) if case["z"] else dict(y=y)
    if op == "linear_back":
        dy, z = s["dy"].double(), s["z"].double()
        if case["gated"]:
            g, up = torch.chunk(z, 2, dim=1)
            a, d = _act64(g, case["act"])
            dz = torch.hstack([dy * up * d, dy * a])
        else:
            dz = dy * _act64(z, case["act"])[1]
        dzb = dz.to(torch.bfloat16)                                              # what the products read
        dx = _mx64(dzb) @ _unpack64(s["wqt"], s["wsft"]).t()
        return dict(dx=dx, dw=_mx64t(dzb) @ _unpack64(s["xqt"], s["xsft"]).t(), dbias=torch.einsum("ij->j", dz))
    if op == "experts":
        x, y, at = _unpack64(s["xq"], s["xsf"]), torch.empty(m, case["n"], dtype=torch.float64, device=DEV), 0
        for e, rows in enumerate(s["sizes"]):
            if rows:
                y[at:at + rows] = x[at:at + rows] @ _unpack64(s["wq"][e], s["wsf"][e]).t()
            at += rows
        return y
    if op == "experts_train":
        n, at = case["n"], 0
        y, dx, dw = (torch.zeros(*sh, dtype=torch.float64, device=DEV) for sh in ((m, n), (m, k), (case["groups"], n, k)))
        for e, rows in enumerate(s["sizes"]):
            if rows:
                x, dy, w = s["x"][at:at + rows], s["dy"][at:at + rows], s["w"][e]
                y[at:at + rows] = _mx64(x) @ _mx64(w).t()
                dx[at:at + rows] = _mx64(dy) @ _mx64t(w).t()
                dw[e] = _mx64t(dy) @ _mx64t(x).t()
            at += rows
        return dict(y=y, dx=dx, dw=dw)
    rows_gate = torch.arange(m, device=DEV) // s["gate_rows"]
    x, w, pw, gate = (s[t].double() for t in ("x", "weight", "post_weight", "gate"))
    if op == "sandwich":
        rstd_x = 1 / torch.sqrt((x * x).sum(dim=1) / k + EPS)
        h = s["residual"].double() + gate[rows_gate] * (x * pw) * (rstd_x * s["scale"])[:, None]
        h = h.to(torch.bfloat16).double()                                        # stored so; what follows reads it
        rstd = 1 / torch.sqrt((h * h).sum(dim=1) / k + EPS)
        y = (h * rstd[:, None] * w).view(m, k // 128, 128)
        big = y.abs().amax(dim=2)
        if case["scales"] == "f32":
            unit = torch.where(big > 0, (big / 448).clamp(min=2.0 ** -126), 1.0)
            sf = unit.t().contiguous()
        else:
            unit = _unit(big, 448.0)
            sf = torch.ones(m, (k // 128 + 3) // 4 * 4, dtype=torch.float64, device=DEV)
            sf[:, :k // 128] = unit
        grid = torch.tensor(_E4M3, dtype=torch.float64, device=DEV)
        code = (y / unit[..., None]).clamp(-448, 448)
        q = (torch.sign(code) * _nearest(code.abs(), grid)).view(m, k)
        return dict(q=q, sf=sf, h=h, rstd_x=rstd_x, rstd=rstd)
    # the gradients by the chain rule over the formula's parts
    dy, dh, h, rh, rx = (s[t].double() for t in ("dy", "dh", "h", "rstd", "rstd_x"))
    inner = torch.einsum("ij,j,ij->i", dy, w, h) / k
    dres = dh + rh[:, None] * dy * w - (rh ** 3 * inner)[:, None] * h
    dn = s["scale"] * gate[rows_gate] * dres                                     # the gradient of norm(x)
    inner = torch.einsum("ij,j,ij->i", dn, pw, x) / k
    dx = rx[:, None] * dn * pw - (rx ** 3 * inner)[:, None] * x
    of_row = s["scale"] * dres * (x * rx[:, None]) * pw
    dgate = torch.stack([of_row[b * s["gate_rows"]:(b + 1) * s["gate_rows"]].sum(dim=0) for b in range(len(gate))])
    return dict(dx=dx, dresidual=dres, dweight=torch.einsum("ij,ij,i->j", dy, h, rh),
                dpost_weight=torch.einsum("ij,ij,i->j", dn, x, rx), dgate=dgate)
