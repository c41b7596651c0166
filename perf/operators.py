"""The operators around a decode step of the MoE layer: the norm before it, MXFP4 linears, and the routed experts for a few tokens.

Three operators, by a case's "op":
  norm    r = x + residual, n = r / sqrt(mean(r^2) + eps) * gamma, as bf16 and as MXFP8 codes with E8M0 scales
  linear  y = x W^T, x in MXFP8, W in MXFP4 (both with one E8M0 scale per 32 elements of the contraction)
  decode  y = shared(x) + sum_j w_j expert_j(x), experts in MXFP4, for 1 to 8 tokens

With `own` false, `run` computes them from elementary torch operations in fp32; with `own` true it calls the package.
"""
import math

import torch

own = False

EPS = 1e-5
#: the layer's width, its experts' and the latent option's width
D, I, D_LATENT = 7168, 3072, 3584


def _api():
    from block_scaled_moe_sigmoid_b200 import api
    return api


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one token of a decode step before the layer: a pure latency
        {"name": "norm_t1", "op": "norm", "rows": 1, "cols": D, "residual": "bfloat16"},
        # a ragged batch of a model that keeps its residual stream in fp32, at the latent width
        {"name": "norm_t333_f32", "op": "norm", "rows": 333, "cols": D_LATENT, "residual": "float32"},
        # the first norm of a stack: no residual yet; a narrow model with an odd number of 32-blocks
        {"name": "norm_t1000_plain", "op": "norm", "rows": 1000, "cols": 736, "residual": "none"},
        # the prefill batch of the layer's benchmark
        {"name": "norm_t8192", "op": "norm", "rows": 8192, "cols": D, "residual": "bfloat16"},
        # one token through a projection between the latent width and the layer's
        {"name": "linear_t1", "op": "linear", "rows": 1, "n": D, "k": D_LATENT, "out": "bfloat16"},
        # a few tokens, an odd number of outputs, as fp32: a small classifier's logits
        {"name": "linear_t5_odd", "op": "linear", "rows": 5, "n": 1003, "k": 640, "out": "float32"},
        # eight sequences through a large output projection
        {"name": "linear_t8_wide", "op": "linear", "rows": 8, "n": 40000, "k": D, "out": "bfloat16"},
        # a short prompt through a square projection
        {"name": "linear_t300", "op": "linear", "rows": 300, "n": D, "k": D, "out": "bfloat16"},
        # the toy layer with three tokens and the clamped activation
        {"name": "decode_toy_t3", "op": "decode", "rows": 3, "d": 512, "i": 256, "e": 32, "k": 4, "i_shared": 0, "act": "clamped"},
        # narrow experts whose widths end inside a tile, with a shared expert
        {"name": "decode_odd_t5", "op": "decode", "rows": 5, "d": 1152, "i": 640, "e": 10, "k": 3, "i_shared": 384, "act": "silu"},
        # one token through the layer's experts and its shared expert, on a slice of 64 experts
        {"name": "decode_t1", "op": "decode", "rows": 1, "d": D, "i": I, "e": 64, "k": 16, "i_shared": I, "act": "silu"},
        # eight sequences at the latent width: every expert of the slice is touched
        {"name": "decode_t8_latent", "op": "decode", "rows": 8, "d": D_LATENT, "i": I, "e": 64, "k": 16, "i_shared": 0, "act": "silu"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "decode"])
    if op == "norm":
        cols = 32 * _log(rng, 1, 320)
        rows = min(_log(rng, 1, 8192), 8192 * D // cols)
        return {"op": op, "rows": rows, "cols": cols, "residual": rng.choice(["bfloat16", "float32", "none"])}
    if op == "linear":
        rows = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, _log(rng, 9, 300)])
        n, k = _log(rng, 1, 40000), 128 * _log(rng, 1, 56)
        if rows > 8:
            n = min(n, D)
        return {"op": op, "rows": rows, "n": n, "k": k, "out": rng.choice(["bfloat16", "float32"])}
    e = rng.randint(1, 64)
    k = rng.randint(1, min(e, 16))
    return {"op": op, "rows": rng.randint(1, 8), "d": 128 * _log(rng, 1, 28), "i": 128 * _log(rng, 1, 24), "e": e, "k": k,
            "i_shared": rng.choice([0, 128 * rng.randint(1, 24)]), "act": rng.choice(["silu", "clamped"])}


# ---------------------------------------------------------------- inputs

def _exponents(amax, emax):
    """The MX rule's block exponent floor(log2 amax) - emax, at least -127; -127 for a block of zeros."""
    e = torch.frexp(amax).exponent - 1 - emax
    return torch.where(amax == 0, torch.full_like(e, -127), e).clamp(min=-127)


def _pow2(e):
    """2^e as fp32, for whole e from -127 to 127, by its bits (a power function may be off by a unit in the last place)."""
    return torch.where(e > -127, (e + 127) << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _mx4(w):
    """fp32 [..., K] -> MXFP4: codes [..., K / 2], element 2j in the low nibble of byte j, and E8M0 scales [..., K / 32]."""
    b = w.unflatten(-1, (-1, 32))
    e = _exponents(b.abs().amax(-1), 2)
    v = b * _pow2(-e)[..., None]
    a = v.abs().clamp(max=6)
    step = 0.5 * (1 + (a >= 2).float() + 2 * (a >= 4).float())  # spacing 0.5, 1, 2 of the E2M1 grid
    a = torch.round(a / step) * step  # half to even: the grid's codes alternate as the multiples do
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)  # 0 .5 1 1.5 2 3 4 6 -> 0 .. 7
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _mx8(x):
    """[..., K] -> MXFP8: E4M3 values [..., K] and E8M0 scales [..., K / 32] (as bytes)."""
    b = x.float().unflatten(-1, (-1, 32))
    e = _exponents(b.abs().amax(-1), 8)
    q = (b * _pow2(-e)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.flatten(-2), (e + 127).to(torch.uint8)


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def prepare(case, seed):
    g = _gen(seed)

    def randn(*shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(std)

    s = dict(case)
    rows = case["rows"]
    if case["op"] == "norm":
        s["x"] = randn(rows, case["cols"]).bfloat16()
        s["gamma"] = 1 + randn(case["cols"], std=0.1)
        s["res"] = None if case["residual"] == "none" else randn(rows, case["cols"], std=4.0).to(getattr(torch, case["residual"]))
        return s
    if case["op"] == "linear":
        q, xs = _mx8(randn(rows, case["k"]).bfloat16())
        s["q"], s["xs"] = q.view(torch.uint8), xs
        w = randn(case["n"], case["k"], std=0.02)
        s["w"] = _mx4(w)
        if own:
            api = _api()
            s["lin"] = api.LinearMXFP4(case["n"], case["k"])
            s["lin"].pack(w)
            s["plan"] = api.LinearPlan(rows, case["n"], case["k"])
        return s
    d, i, e, k, ish = (case[n] for n in ("d", "i", "e", "k", "i_shared"))
    s["x"] = randn(rows, d).bfloat16()
    q, xs = _mx8(s["x"])
    s["q"], s["xs"] = q.view(torch.uint8), xs
    z, idx = torch.topk(randn(rows, e), k)
    s["idx"] = idx.int()
    s["wt"] = torch.sigmoid(z) / torch.sigmoid(z).sum(-1, keepdim=True)
    ex = None
    if own:
        api = _api()
        ex = s["experts"] = api.Experts(d, i, e)
        s["plan"] = api.Plan(rows, d, e, k, i, ish, act=api.MOE_ACT_CLAMPED_SWIGLU if case["act"] == "clamped" else api.MOE_ACT_SILU_GLU)
    s["wg"], s["wu"], s["wd"] = ((torch.empty(e, n, m // 2, dtype=torch.uint8, device="cuda"), torch.empty(e, n, m // 32, dtype=torch.uint8, device="cuda"))
                                 for n, m in ((i, d), (i, d), (d, i)))
    for j in range(e):
        ws = randn(i, d, std=0.02), randn(i, d, std=0.02), randn(d, i, std=0.02)
        for name, w in zip(("wg", "wu", "wd"), ws):
            s[name][0][j], s[name][1][j] = _mx4(w)
        if ex is not None:
            ex.pack(j, *ws)
    if ish:
        sw = [randn(n, m, std=0.02).bfloat16() for n, m in ((ish, d), (ish, d), (d, ish))]
        s["shared"] = sw
        if own:
            s["sh"] = api.Shared(d, ish)
            s["sh"].pack(*sw)
    return s


# ---------------------------------------------------------------- one pass

def _decode4(codes, scales):
    """MXFP4 codes and scales -> fp32."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    m = (c & 7).float()
    m = torch.where(m < 4, m * 0.5, torch.where(m < 6, m - 2, 2 * m - 8))  # 0 .5 1 1.5 2 3 4 6
    m = torch.where(c > 7, -m, m)
    return (m.unflatten(-1, (-1, 32)) * _pow2(scales.int() - 127)[..., None]).flatten(-2)


def _decode8(q, s):
    return (q.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32)) * _pow2(s.int() - 127)[..., None]).flatten(-2)


def _glu(g, u, act):
    if act == "clamped":
        g, u = g.clamp(max=7), u.clamp(-7, 7)
        return (u + 1) * g / (1 + torch.exp(-1.702 * g))
    return g / (1 + torch.exp(-g)) * u


def _run_norm(s):
    if own:
        r, xn, q, xs = _api().moe_add_rmsnorm_mxfp8(s["x"], s["gamma"], EPS, residual=s["res"])
    else:
        r = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(s["res"].dtype)
        n = r.float()
        n = n / torch.sqrt((n * n).mean(-1, keepdim=True) + EPS) * s["gamma"]
        xn = n.bfloat16()
        q, xs = _mx8(xn)  # of the rounded values: what the layer's own quantiser makes of xn
        q = q.view(torch.uint8)
        r = None if s["res"] is None else r
    out = [xn, q.view(torch.float8_e4m3fn), xs.view(torch.float8_e8m0fnu)]
    return out if r is None else [r] + out


def _run_linear(s):
    out = getattr(torch, s["out"])
    if own:
        return s["plan"].forward(s["q"], s["xs"], s["lin"], dtype=out)
    return (_decode8(s["q"], s["xs"]) @ _decode4(*s["w"]).T).to(out)


def _run_decode(s):
    if own:
        return s["plan"].forward_decode(s["x"], s["idx"], s["wt"], s["experts"], s.get("sh"), q=s["q"], scale=s["xs"])
    used = torch.unique(s["idx"]).long()
    x = _decode8(s["q"], s["xs"])
    g = x @ _decode4(s["wg"][0][used], s["wg"][1][used]).mT
    u = x @ _decode4(s["wu"][0][used], s["wu"][1][used]).mT
    h = _decode8(*_mx8(_glu(g, u, s["act"])))  # the experts' hidden values are MXFP8, as their inputs are
    o = h @ _decode4(s["wd"][0][used], s["wd"][1][used]).mT  # [used, rows, d]
    w = (s["wt"][:, :, None] * (s["idx"][:, :, None] == used)).sum(1)  # [rows, used]
    y = (w.T[:, :, None] * o).sum(0)
    if "shared" in s:
        sg, su, sd = (m.float() for m in s["shared"])
        xf = s["x"].float()
        y = y + _glu(xf @ sg.T, xf @ su.T, s["act"]).bfloat16().float() @ sd.T  # the shared expert's hidden values are bf16
    return y.bfloat16()


def run(state):
    return {"norm": _run_norm, "linear": _run_linear, "decode": _run_decode}[state["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    rows = case["rows"]
    if case["op"] == "norm":
        n = rows * case["cols"]
        res = {"bfloat16": 4, "float32": 8, "none": 0}[case["residual"]]
        return {"bytes": n * (2 + res + 2 + 1 + 1 / 32) + 4 * case["cols"], "flops": 0}
    if case["op"] == "linear":
        n, k = case["n"], case["k"]
        out = 2 if case["out"] == "bfloat16" else 4
        return {"bytes": (n * k / 2 + n * k / 32) + rows * k * 33 / 32 + rows * n * out, "flops": 2 * rows * n * k}
    d, i, e, k, ish = (case[n] for n in ("d", "i", "e", "k", "i_shared"))
    touched = e * (1 - (1 - k / e) ** rows)  # expected number of experts that some token uses
    return {"bytes": touched * 3 * i * d * 17 / 32 + 6 * ish * d + rows * d * (2 + (2 if ish else 0) + 33 / 32) + rows * k * 8,
            "flops": rows * (6 * k * i * d + 6 * ish * d)}


# ---------------------------------------------------------------- the definition in 64 bits

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def _two64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _scale64(s):
    return _two64(s.long() - 127)


def _w64(codes, scales):
    table = torch.tensor(_E2M1, dtype=torch.float64, device=codes.device)
    low = torch.index_select(table, 0, (codes.int() % 16).reshape(-1)).reshape(codes.shape)
    high = torch.index_select(table, 0, (codes.int() // 16).reshape(-1)).reshape(codes.shape)
    v = torch.stack((low, high), dim=-1).reshape(*codes.shape[:-1], -1, 32)
    return (v * _scale64(scales).unsqueeze(-1)).reshape(*codes.shape[:-1], -1)


def _x64(q, s):
    bits = q.long()
    exp, man = (bits >> 3) & 15, bits & 7
    v = torch.where(exp == 0, man.double() * 2.0 ** -9, (8 + man.double()) * _two64(exp - 10))
    v = torch.where(bits >= 128, -v, v).reshape(*q.shape[:-1], -1, 32)
    return (v * _scale64(s).unsqueeze(-1)).reshape(q.shape)


def _floor_log2(a):
    return (a.view(torch.int64) >> 52) - 1023  # the exponent field; of zero far below every border


def _mx8_64(x):
    """(E4M3 values, scales) of float64 [..., K] by the definition, both as float64."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    top = b.abs().amax(dim=-1, keepdim=True)
    e = (_floor_log2(top) - 8).clamp(min=-127)
    v = b / _two64(e)
    a = v.abs().clamp(max=448)
    step = _two64(_floor_log2(a.clamp(min=2.0 ** -6)) - 3)
    q = torch.copysign(torch.round(a / step) * step, v).clamp(-448, 448)
    return q.reshape(x.shape), _two64(e).squeeze(-1)


def _glu64(g, u, act):
    if act == "clamped":
        g, u = torch.minimum(g, torch.full_like(g, 7)), u.clamp(-7, 7)
        return (u + 1) * g * torch.sigmoid(1.702 * g)
    return g * torch.sigmoid(g) * u


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        r = s["x"].double()
        out = []
        if s["res"] is not None:
            out = [r + s["res"].double()]
            r = out[0].to(s["res"].dtype).double()  # the norm is that of the stored residual
        n = r * (r.square().mean(dim=-1, keepdim=True) + EPS).rsqrt() * s["gamma"].double()
        q, xs = _mx8_64(n.bfloat16().double())
        return out + [n, q, xs]
    if case["op"] == "linear":
        return _x64(s["q"], s["xs"]) @ _w64(*s["w"]).t()
    x, act = _x64(s["q"], s["xs"]), case["act"]
    y = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    for e in torch.unique(s["idx"]).tolist():
        t, j = torch.nonzero(s["idx"] == e, as_tuple=True)
        g, u = (x[t] @ _w64(s[n][0][e], s[n][1][e]).t() for n in ("wg", "wu"))
        q, xs = _mx8_64(_glu64(g, u, act))
        h = q * xs.repeat_interleave(32, dim=-1)
        y.index_add_(0, t, s["wt"][t, j].double()[:, None] * (h @ _w64(s["wd"][0][e], s["wd"][1][e]).t()))
    if "shared" in s:
        sg, su, sd = (m.double() for m in s["shared"])
        x = s["x"].double()
        y += _glu64(x @ sg.t(), x @ su.t(), act).bfloat16().double() @ sd.t()
    return y
