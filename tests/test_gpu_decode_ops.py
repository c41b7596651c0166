"""The operators around a decode step on the GPU, against the fp64 oracle: the norm before the layer,
MXFP4 linears, and the layer for a few tokens; then the three in a row, as a decode step uses them.

Tolerances.  A rounding is off by at most half a step: 2^-8 of the value for bf16, 2^-24 for fp32.
  norm    one bf16 rounding, plus the fp32 arithmetic before it: at most 32 terms per thread, 5 + 32 tree
          additions, a square root and two products, under 80 half steps of fp32 (80 x 2^-24 < 2^-17)
  linear  one rounding of the result, plus the fp32 sums: every product is exact; a term passes at most
          32 additions inside its block, K / 32 over the blocks and one per partial, each off by at most
          2^-23 (the tensor core truncates) of the sum of magnitudes S: (K / 32 + 64 + partials) 2^-23 S
  layer   the layer's own bounds: relative error (row-rms floor) at most 2e-2, on average 2e-3
"""
import numpy as np
import pytest
import torch

from block_scaled_moe_sigmoid_b200 import api, synth
from oracle import layer, mx

from .gpu_helpers import Case

pytestmark = pytest.mark.gpu


def randn(shape, seed, std=1.0, dtype=torch.float32):
    return synth.normal(shape, seed, 77, std=std).to(dtype).cuda()


def same_bytes(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---------------------------------------------------------------- norm
def norm_ref(x, gamma, eps, res):
    """(r as the stored tensor, n in fp64) from host copies."""
    r = x if res is None else (x.float() + res.float()).to(res.dtype)   # one fp32 addition, one rounding
    return r, layer.rms_norm(r.double().numpy(), gamma.double().numpy(), eps)


def check_norm(x, gamma, eps, res, out):
    r_out, xn, q, scale = out
    r, n = norm_ref(x.cpu(), gamma.cpu(), eps, None if res is None else res.cpu())
    if res is not None:
        assert r_out.dtype == res.dtype and same_bytes(r_out.cpu(), r)
    got = xn.double().cpu().numpy()
    assert np.all(np.abs(got - n) <= np.abs(n) * (2.0 ** -8 + 2.0 ** -17) + 2.0 ** -133)
    q_o, s_o = mx.quantize_mx(got, "e4m3")
    assert np.array_equal(q.cpu().numpy(), q_o) and np.array_equal(scale.cpu().numpy(), s_o)


@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows, cols", [(1, 32), (3, 64), (129, 96), (5, 736), (700, 1024), (1, 7168), (33, 7168), (7, 8224),
                                        (3, 16416), (2, 32768),
                                        (301, 4128), (310, 16384), (300, 16416), (320, 30016), (1000, 7168), (1200, 2112), (700, 4096), (500, 6144)])
def test_norm(rows, cols, res):
    seed = rows * 100003 + cols
    x, gamma = randn((rows, cols), seed, dtype=torch.bfloat16), 1 + randn((cols,), seed + 1, 0.1)
    residual = None if res is None else randn((rows, cols), seed + 2, 3.0, res)
    out = api.moe_add_rmsnorm_mxfp8(x, gamma, 1e-5, residual=residual)
    check_norm(x, gamma, 1e-5, residual, out)
    q, s = api.moe_quant_mxfp8(out[1])
    assert torch.equal(q, out[2]) and torch.equal(s, out[3])   # the bytes that the layer's quantiser makes of xn


def test_norm_in_place_and_subsets_of_outputs():
    rows, cols = 37, 352
    x, gamma = randn((rows, cols), 1, dtype=torch.bfloat16), 1 + randn((cols,), 2, 0.1)
    for dtype in (torch.bfloat16, torch.float32):
        res = randn((rows, cols), 3, 2.0, dtype)
        want = api.moe_add_rmsnorm_mxfp8(x, gamma, 1e-5, residual=res)
        buf = res.clone()
        got = api.moe_add_rmsnorm_mxfp8(x, gamma, 1e-5, residual=buf, residual_out=buf)
        assert got[0] is buf and all(same_bytes(a, b) for a, b in zip(got, want))
        a = api.moe_add_rmsnorm_mxfp8(x, gamma, 1e-5, residual=res, with_mx=False)
        b = api.moe_add_rmsnorm_mxfp8(x, gamma, 1e-5, residual=res, with_xn=False)
        c = api.moe_add_rmsnorm_mxfp8(x, gamma, 1e-5, residual=res, with_xn=False, with_mx=False)
        assert a[2] is a[3] is b[1] is c[1] is c[2] is None
        assert same_bytes(a[0], want[0]) and same_bytes(a[1], want[1])
        assert same_bytes(b[0], want[0]) and same_bytes(b[2], want[2]) and same_bytes(b[3], want[3])
        assert same_bytes(c[0], want[0])
    xc = x.clone()
    got = api.moe_add_rmsnorm_mxfp8(xc, gamma, 1e-5, xn=xc)    # the norm over its own input
    assert same_bytes(xc, api.moe_add_rmsnorm_mxfp8(x, gamma, 1e-5)[1]) and got[1] is xc
    # the same where rows stream through a resident grid
    rows, cols = 700, 4352
    x, gamma, res = randn((rows, cols), 6, dtype=torch.bfloat16), 1 + randn((cols,), 7, 0.1), randn((rows, cols), 8, 2.0, torch.bfloat16)
    want = api.moe_add_rmsnorm_mxfp8(x, gamma, 1e-5, residual=res)
    buf, xc = res.clone(), x.clone()
    got = api.moe_add_rmsnorm_mxfp8(xc, gamma, 1e-5, residual=buf, residual_out=buf, xn=xc)
    assert all(same_bytes(a, b) for a, b in zip(got, want))
    only = api.moe_add_rmsnorm_mxfp8(x, gamma, 1e-5, residual=res, with_xn=False, with_mx=False)
    assert same_bytes(only[0], want[0])
    none = api.moe_add_rmsnorm_mxfp8(x[:0], gamma)
    assert none[1].shape == (0, cols) and none[3].shape == (0, cols // 32)


def test_norm_zero_rows_and_values_that_are_not_finite():
    rows, cols = 6, 128
    x, gamma = randn((rows, cols), 5, dtype=torch.bfloat16), torch.ones(cols, device="cuda")
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 70] = float("nan")
    x[4] *= 2.0 ** 40
    x[5] *= 2.0 ** -60      # far below eps: the norm scales by 1 / sqrt(eps)
    _, xn, q, s = api.moe_add_rmsnorm_mxfp8(x, gamma, 1e-5)
    clean = [0, 1, 4, 5]
    _, n = norm_ref(x.cpu()[clean], gamma.cpu(), 1e-5, None)
    got = xn.double().cpu().numpy()[clean]
    assert np.all(np.abs(got - n) <= np.abs(n) * (2.0 ** -8 + 2.0 ** -17) + 2.0 ** -133)
    assert not xn[1].any() and not q[1].any() and not s[1].any()
    row = xn[2].float()
    assert torch.isnan(row[5]) and not row[:5].any() and not row[6:].any()     # inf * 0; the others over infinity
    assert torch.isnan(xn[3].float()).all()
    q2, s2 = api.moe_quant_mxfp8(xn)
    assert torch.equal(q, q2) and torch.equal(s, s2)


def test_norm_guards_and_other_stream():
    """Nothing is written behind the last row, and the call runs on the stream it is given."""
    rows, cols = 9, 96
    x, gamma = randn((rows, cols), 11, dtype=torch.bfloat16), 1 + randn((cols,), 12, 0.1)
    res = randn((rows, cols), 13)
    want = api.moe_add_rmsnorm_mxfp8(x, gamma, 1e-5, residual=res)
    torch.cuda.synchronize()
    pad = 64
    big = [torch.full((rows * c + pad,), 7, dtype=dt, device="cuda")
           for c, dt in ((cols, torch.float32), (cols, torch.bfloat16), (cols, torch.uint8), (cols // 32, torch.uint8))]
    views = [b[:-pad].view(rows, -1) for b in big]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    api.moe_add_rmsnorm_mxfp8(x, gamma, 1e-5, res, *views, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for v, w, b in zip(views, want, big):
        assert same_bytes(v, w) and bool((b[-pad:] == 7).all())


# ---------------------------------------------------------------- linear
def linear_case(T, N, K, seed, std=0.02):
    x = randn((T, K), seed, dtype=torch.bfloat16)
    q, s = api.moe_quant_mxfp8(x)
    w = randn((N, K), seed + 1, std)
    lin = api.LinearMXFP4(N, K)
    lin.pack(w)
    return q, s, lin, w


def check_linear(q, s, w, y, rows=None):
    X = mx.dequantize_mx(q.cpu().numpy(), s.cpu().numpy(), "e4m3")
    W = mx.dequantize_mx(*mx.quantize_mx(w.double().cpu().numpy(), "e2m1"), "e2m1")
    ref, S = X @ W.T, np.abs(X) @ np.abs(W).T
    K = X.shape[1]
    half = 2.0 ** -8 if y.dtype == torch.bfloat16 else 2.0 ** -24
    tol = (K / 32 + 64 + 256) * 2.0 ** -23 * S
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= tol + half * (np.abs(ref) + tol) + 2.0 ** -133), float((err / (tol + half * np.abs(ref) + 1e-30)).max())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T, N, K", [(1, 1, 128), (1, 256, 128), (2, 257, 256), (3, 255, 640), (5, 1003, 640), (8, 512, 1152),
                                     (7, 40, 7168), (4, 3333, 384), (8, 300, 10240), (8, 130, 10368), (6, 260, 20480), (16, 1003, 896), (13, 513, 512), (17, 300, 640),
                                     (9, 1003, 640), (64, 257, 256), (65, 7, 1152), (300, 512, 2048), (177, 1000, 128)])
def test_linear(T, N, K, dtype):
    q, s, lin, w = linear_case(T, N, K, T * 1000 + N)
    plan = api.LinearPlan(T, N, K)
    y = plan.forward(q, s, lin, dtype=dtype)
    assert plan.check()[0] == 0 and y.dtype == dtype
    check_linear(q, s, w, y)
    assert torch.equal(plan.forward(q, s, lin, dtype=dtype), y)      # a fixed order of sums


@pytest.mark.parametrize("T", [1, 8, 16, 17, 40, 64, 65, 130, 300, 520])
def test_linear_stays_inside_its_workspace(T):
    """Wide enough to be split over all SMs: right, and nothing written behind the workspace's bytes."""
    N, K = 4096, 4096
    q, s, lin, w = linear_case(T, N, K, T)
    plan = api.LinearPlan(T, N, K)
    need = api.moe_linear_workspace_bytes(plan.handle)
    ws = torch.full((need + (64 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    api.moe_linear_set_workspace(plan.handle, ws[:need])
    y = plan.forward(q, s, lin, dtype=torch.float32)
    assert plan.check()[0] == 0
    assert bool((ws[need:] == 0x5A).all())
    check_linear(q, s, w, y)
    assert torch.equal(plan.forward(q, s, lin, dtype=torch.float32), y)


@pytest.mark.parametrize("T, N, K, rows, split", [
    (100, 20003, 128, 112, False), (333, 15003, 384, 176, False), (700, 20003, 384, 144, False), (340, 36003, 256, 176, False),
    (65, 5003, 7168, 80, True), (129, 20003, 7168, 144, True), (331, 20003, 14336, 176, True),
    (1777, 5003, 384, 128, False), (1500, 7169, 640, 160, False), (2110, 9003, 256, 176, False), (3001, 9003, 512, 160, False),
    (1025, 255, 3584, 32, True), (2101, 1003, 1152, 64, False)])
def test_linear_wide_tiles_and_long_prompts(T, N, K, rows, split):
    """Tiles of more than 64 token rows, one and two atoms of token scales, whole and split, one and more a CTA, and past
    1024 rows: against the oracle in both types, with guards behind the output and the workspace.  The weight rows repeat
    with a period of 257, one more than a tile's, so that the oracle's product stays small."""
    period = 257
    x, base = randn((T, K), T, dtype=torch.bfloat16), randn((period, K), N, 0.02)
    q, s = api.moe_quant_mxfp8(x)
    lin, plan = api.LinearMXFP4(N, K), api.LinearPlan(T, N, K)
    lin.pack(base[torch.arange(N, device="cuda") % period])
    assert api.moe_linear_tiling(plan.handle, T) == (rows, split)    # of 148 SMs: what this case is here for
    need, pad = api.moe_linear_workspace_bytes(plan.handle), 4096
    ws = torch.full((need + (16 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    api.moe_linear_set_workspace(plan.handle, ws[:need])
    X = mx.dequantize_mx(q.cpu().numpy(), s.cpu().numpy(), "e4m3")
    W = mx.dequantize_mx(*mx.quantize_mx(base.double().cpu().numpy(), "e2m1"), "e2m1")
    cols = np.arange(N) % period
    ref, tol = X @ W.T, (K / 32 + 64 + 256) * 2.0 ** -23 * (np.abs(X) @ np.abs(W).T)
    for dtype, half in ((torch.float32, 2.0 ** -24), (torch.bfloat16, 2.0 ** -8)):
        bound = tol + half * (np.abs(ref) + tol) + 2.0 ** -133
        buf = torch.full((T * N + pad,), 7, dtype=dtype, device="cuda")
        y = plan.forward(q, s, lin, y=buf[:T * N].view(T, N))
        assert plan.check()[0] == 0 and bool((buf[T * N:] == 7).all()) and bool((ws[need:] == 0x5A).all())
        got = y.double().cpu().numpy()
        assert np.all(np.abs(got - ref[:, cols]) <= bound[:, cols]), float((np.abs(got - ref[:, cols]) / bound[:, cols]).max())
        assert torch.equal(plan.forward(q, s, lin, dtype=dtype), y)  # a fixed order of sums


def test_linear_rows_do_not_depend_on_the_batch():
    """A row's result on the weight stream is the same alone and among seven others."""
    N, K = 777, 896
    q, s, lin, _ = linear_case(8, N, K, 42)
    plan = api.LinearPlan(8, N, K)
    y = plan.forward(q, s, lin, dtype=torch.float32)
    for t in range(8):
        assert torch.equal(plan.forward(q[t:t + 1].contiguous(), s[t:t + 1].contiguous(), lin, dtype=torch.float32)[0], y[t])


@pytest.mark.parametrize("T", [5, 40])
def test_linear_scales_at_the_ends_and_rows_that_are_not_finite(T):
    N, K = 300, 512
    q, s, lin, w = linear_case(T, N, K, 7)
    plan = api.LinearPlan(T, N, K)
    clean = plan.forward(q, s, lin, dtype=torch.float32)
    q2, s2 = q.clone(), s.clone()
    q2[1, 3] = 0x7F                       # a NaN code: its row alone is lost
    q2[2] = 0                             # a row of zeros whose scales are the largest there are
    s2[2] = 254
    s2[3] = 0                             # the smallest scale: 2^-127
    y = plan.forward(q2, s2, lin, dtype=torch.float32)
    assert torch.isnan(y[1]).all() and not y[2].any()
    keep = [t for t in range(T) if t not in (1, 2, 3)]
    assert torch.equal(y[keep], clean[keep])
    assert float(y[3].abs().max()) < 2.0 ** -110 and (T > 8 or bool(y[3].any()))
    w0 = w.clone()
    w0[5] = 0                             # a row of zero weights
    w0[6] *= 2.0 ** 60
    lin.pack(w0)
    y = plan.forward(q, s, lin, dtype=torch.float32)
    assert not y[:, 5].any()
    check_linear(q, s, w0, y)


@pytest.mark.parametrize("T, N", [(5, 300), (16, 300), (40, 300), (100, 20003)])
def test_linear_values_at_the_ends_of_the_scales(T, N):
    """Rows and weights with the smallest scales and with large ones, against the oracle (the last case in tiles of 112 rows).
    Below 2^-126 an fp32 value is a multiple of 2^-149: each of a sum's additions may round there by that much more."""
    K, period = 512, 129
    x, base = randn((T, K), 3, dtype=torch.bfloat16), randn((period, K), 4, 0.02)
    base[6] *= 2.0 ** 60
    base[7] *= 2.0 ** -100
    base[8] *= 2.0 ** -125
    q, s = api.moe_quant_mxfp8(x)
    s[0] = 0                              # 2^-127
    s[1, ::2] = 1
    s[3] = 120                            # 2^-7 in all blocks
    s[4, 3] = 180                         # one block that outweighs the others by 2^50
    lin, plan = api.LinearMXFP4(N, K), api.LinearPlan(T, N, K)
    lin.pack(base[torch.arange(N, device="cuda") % period])
    y = plan.forward(q, s, lin, dtype=torch.float32).double().cpu().numpy()
    assert plan.check()[0] == 0
    X = mx.dequantize_mx(q.cpu().numpy(), s.cpu().numpy(), "e4m3")
    W = mx.dequantize_mx(*mx.quantize_mx(base.double().cpu().numpy(), "e2m1"), "e2m1")
    cols, terms = np.arange(N) % period, K / 32 + 64 + 256
    ref, tol = X @ W.T, terms * 2.0 ** -23 * (np.abs(X) @ np.abs(W).T)
    bound = tol + 2.0 ** -24 * (np.abs(ref) + tol) + terms * 2.0 ** -149
    assert np.all(np.abs(y - ref[:, cols]) <= bound[:, cols]), float((np.abs(y - ref[:, cols]) / bound[:, cols]).max())
    assert np.count_nonzero(y[0]) > N // 2     # the smallest scale is not taken for zero


@pytest.mark.parametrize("T, dtype", [(3, torch.float32), (8, torch.bfloat16), (20, torch.bfloat16), (100, torch.float32)])
def test_linear_writes_its_rows_only(T, dtype):
    N, K, pad = 1003, 256, 512
    q, s, lin, w = linear_case(T, N, K, 3)
    buf = torch.full((T * N + pad,), 7, dtype=dtype, device="cuda")
    y = buf[:T * N].view(T, N)
    plan = api.LinearPlan(T + 5, N, K)
    assert plan.forward(q, s, lin, y=y).data_ptr() == y.data_ptr()
    check_linear(q, s, w, y)
    assert bool((buf[T * N:] == 7).all())
    assert plan.forward(q[:0], s[:0], lin).shape == (0, N)


def test_linear_two_plans_on_two_streams_and_graph_replay():
    T, N, K = 4, 2048, 1024
    cases = [linear_case(T, N, K, 10 * i) for i in range(2)]
    plans = [api.LinearPlan(T, N, K) for _ in range(2)]
    want = [p.forward(c[0], c[1], c[2]) for p, c in zip(plans, cases)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            got[i].append(plans[i].forward(*cases[i][:3], stream=streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])
    # captured once, replayed on new inputs in the same tensors
    q, s, lin, _ = cases[0]
    y = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        plans[0].forward(q, s, lin, y=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plans[0].forward(q, s, lin, y=y)
    for i in (1, 0, 1):
        q.copy_(cases[i][0]) if i else q.copy_(linear_case(T, N, K, 0)[0])
        s.copy_(cases[i][1]) if i else s.copy_(linear_case(T, N, K, 0)[1])
        y.zero_()
        g.replay()
        assert torch.equal(y, plans[1].forward(q, s, lin))
    assert all(p.check()[0] == 0 for p in plans)


def test_packing_a_strided_weight_on_a_side_stream():
    """Packed while the current stream is busy, and its pool's memory in use: the bytes are those of the contiguous weight."""
    N = K = 512
    w = randn((K, N), 5, 0.02)
    sw = randn((K, N), 6, 0.02, torch.bfloat16)
    want, got = [(api.LinearMXFP4(N, K), api.Experts(K, N, 1), api.Shared(K, N)) for _ in range(2)]

    def pack(buffers, m, b, stream=None):
        buffers[0].pack(m, stream=stream)
        buffers[1].pack(0, m, m, m, stream=stream)
        buffers[2].pack(b, b, b, stream=stream)

    pack(want, w.t().contiguous(), sw.t().contiguous())
    side, junk = torch.cuda.Stream(), torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    for _ in range(20):
        junk.fill_(255)
    pack(got, w.t(), sw.t(), side)
    for _ in range(4):                      # what the current stream allocates next is not what the packing reads
        torch.empty(N * K, dtype=torch.float32, device="cuda").fill_(7.0)
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for name in ("w", "s", "w_gu", "s_gu", "w_dn", "s_dn"):
            if hasattr(a, name):
                assert same_bytes(getattr(a, name), getattr(b, name)), (type(a).__name__, name)


# ---------------------------------------------------------------- the layer for a few tokens
def check_decode(case, idx, w, y, T=None):
    rows = case.x_np() if T is None else case.x_np()[:T]
    ref = layer.moe_layer(rows, idx.cpu().numpy(), w.cpu().numpy(), case.oracle_expert, case.oracle_shared(), act=case.act)
    r, _ = layer.relative_errors(y.double().cpu().numpy(), ref)
    assert r.max() <= 2e-2 and r.mean() <= 2e-3, (r.max(), r.mean())


def draws(T, E, k, seed):
    g = torch.Generator().manual_seed(seed)
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).to(torch.int32).cuda()
    w = torch.rand(T, k, generator=g) + 0.1
    return idx, (w / w.sum(1, keepdim=True)).cuda()


@pytest.mark.parametrize("T, d, E, k, I, Is, act", [
    (1, 128, 1, 1, 128, 0, "silu"), (1, 256, 16, 4, 128, 128, "silu"), (2, 384, 8, 3, 256, 0, "clamped_swiglu"),
    (3, 512, 32, 4, 256, 0, "silu"), (5, 1152, 10, 3, 640, 384, "silu"), (8, 256, 40, 32, 128, 0, "silu"),
    (8, 640, 4, 4, 384, 256, "clamped_swiglu"), (7, 256, 300, 8, 128, 0, "silu"), (8, 1024, 64, 16, 512, 0, "silu"),
    (16, 384, 64, 32, 256, 128, "silu"), (1, 1024, 4, 2, 128, 1024, "silu"), (2, 3584, 4, 1, 256, 640, "clamped_swiglu"),
    (4, 128, 2, 1, 128, 2048, "silu"), (11, 256, 4096, 2, 128, 0, "silu")])
def test_forward_decode(T, d, E, k, I, Is, act):
    case = Case(synth.custom(seed=T + E, T=T, d=d, E=E, k=k, I=I, I_shared=Is), act=act)
    idx, w = draws(T, E, k, 5)
    y = case.plan.forward_decode(case.x, idx, w, case.experts, case.shared)
    assert case.plan.check()[0] == 0
    check_decode(case, idx, w, y)
    q, s = api.moe_quant_mxfp8(case.x)
    again = case.plan.forward_decode(case.x, idx, w, case.experts, case.shared, q=q, scale=s)
    assert torch.equal(again, y)                     # the same activations in either form, in a fixed order of sums
    if not Is:
        assert torch.equal(case.plan.forward_decode(None, idx, w, case.experts, q=q, scale=s), y)
    # the layer's tile form on the same operands: it holds each expert's output in bf16 (2^-8) before the combine
    ref = case.plan.forward(case.x, idx, w, case.experts, case.shared)
    r, _ = layer.relative_errors(y.double().cpu().numpy(), ref.double().cpu().numpy())
    assert r.max() <= 2e-2


def test_forward_decode_every_token_on_the_same_experts_and_rows_alone():
    T, E, k = 8, 16, 4
    case = Case(synth.custom(seed=2, T=T, d=512, E=E, k=k, I=256))
    idx, w = draws(1, E, k, 1)
    idx, w = idx.repeat(T, 1).contiguous(), draws(T, E, k, 2)[1]
    y = case.plan.forward_decode(case.x, idx, w, case.experts)
    check_decode(case, idx, w, y)
    for t in (0, 7):
        one = case.plan.forward_decode(case.x[t:t + 1].contiguous(), idx[t:t + 1].contiguous(), w[t:t + 1].contiguous(), case.experts)
        # the same products; the split of the sums over CTAs depends on the batch, not on the timing
        r, _ = layer.relative_errors(one.double().cpu().numpy(), y[t:t + 1].double().cpu().numpy())
        assert r.max() <= 2.0 ** -7


def test_forward_decode_ids_outside_and_named_twice():
    T, E, k = 3, 8, 3
    case = Case(synth.custom(seed=9, T=T, d=256, E=E, k=k, I=128, I_shared=128))
    idx, w = draws(T, E, k, 3)
    bad = idx.clone()
    bad[1, 0], bad[2, 2] = -1, E
    y = case.plan.forward_decode(case.x, bad, w, case.experts, case.shared)
    code, bits = case.plan.check()
    assert code == 7 and bits == 2                   # MOE_ERR_DEVICE_FAULT, the bounds bit
    w0 = w.clone()
    w0[1, 0] = w0[2, 2] = 0                          # the same as the valid ids with no weight there
    check_decode(case, idx, w0, y)
    none = case.plan.forward_decode(case.x, torch.full_like(idx, -1), w, case.experts, case.shared)
    assert case.plan.check()[0] == 7
    ys = layer.shared_expert(case.x_np(), *case.oracle_shared())[0]
    assert layer.relative_errors(none.double().cpu().numpy(), ys)[0].max() <= 2.0 ** -7
    plain = Case(synth.custom(seed=9, T=T, d=256, E=E, k=k, I=128))
    none = plain.plan.forward_decode(plain.x, torch.full_like(idx, E), w, plain.experts)
    assert not none.any() and plain.plan.check()[0] == 7
    twice = idx.clone()
    twice[:, 1] = twice[:, 0]
    y2 = case.plan.forward_decode(case.x, twice, w, case.experts, case.shared)
    assert case.plan.check()[0] == 0
    w1 = w.clone()
    w1[:, 0] += w[:, 1]
    w1[:, 1] = 0
    assert layer.relative_errors(y2.double().cpu().numpy(),
                                 case.plan.forward_decode(case.x, idx, w1, case.experts, case.shared).double().cpu().numpy())[0].max() <= 2.0 ** -7
    assert case.plan.check()[0] == 0


def test_check_is_done_with_the_workspace_when_it_returns():
    """On a stream that does not order itself after the legacy one, calls right after a check that has flags to clear:
    the check leaves the tile counters and the status word alone from then on."""
    T, E, k = 4, 16, 4
    case = Case(synth.custom(seed=31, T=T, d=1024, E=E, k=k, I=512, I_shared=512))
    idx, w = draws(T, E, k, 6)
    bad = torch.full_like(idx, E)
    want = case.plan.forward_decode(case.x, idx, w, case.experts, case.shared)
    assert case.plan.check()[0] == 0
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for i in range(100):
        case.plan.forward_decode(case.x, bad, w, case.experts, case.shared, stream=side)
        assert case.plan.check(side) == (7, 2)               # MOE_ERR_DEVICE_FAULT, the bounds bit
        got.append(case.plan.forward_decode(case.x, idx, w, case.experts, case.shared, stream=side))
        if i % 10 == 0:
            assert case.plan.check(side) == (0, 0)
            api.moe_debug_timeout_probe(case.plan.handle, side) if i == 50 else None
            assert case.plan.check(side)[0] == (5 if i == 50 else 0)
            got.append(case.plan.forward_decode(case.x, idx, w, case.experts, case.shared, stream=side))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in got) and case.plan.check(side) == (0, 0)


def test_forward_decode_tokens_that_are_not_finite_keep_to_themselves():
    T, E, k = 4, 8, 2
    case = Case(synth.custom(seed=4, T=T, d=256, E=E, k=k, I=128))
    idx, w = draws(T, E, k, 8)
    idx[1] = idx[0]                                  # the clean token shares its experts with the broken one
    y = case.plan.forward_decode(case.x, idx, w, case.experts)
    x = case.x.clone()
    x[1, 17] = float("nan")
    z = case.plan.forward_decode(x, idx, w, case.experts)
    assert torch.isnan(z[1].float()).all()
    keep = [0, 2, 3]
    assert torch.equal(z[keep], y[keep])


def test_forward_decode_graph_replay_and_calls_in_between():
    """Captured and replayed on new inputs; other calls of the same plan between replays leave it alone."""
    T, E, k = 2, 16, 4
    case = Case(synth.custom(seed=6, T=64, d=512, E=E, k=k, I=256, I_shared=256))
    x = case.x[:T].clone()
    idx, w = draws(T, E, k, 1)
    y = torch.empty(T, 512, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        case.plan.forward_decode(x, idx, w, case.experts, case.shared, y=y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        case.plan.forward_decode(x, idx, w, case.experts, case.shared, y=y)
    for i in range(3):
        x.copy_(case.x[T * i:T * i + T])
        i2, w2 = draws(T, E, k, 20 + i)
        idx.copy_(i2)
        w.copy_(w2)
        y.zero_()
        g.replay()
        want = case.plan.forward_decode(x, idx, w, case.experts, case.shared)
        assert torch.equal(y, want)
        r_idx, r_w = case.plan.route(case.x, case.W_r, case.bias)
        case.plan.forward(case.x, r_idx, r_w, case.experts, case.shared)
    assert case.plan.check()[0] == 0


@pytest.mark.parametrize("T", [1, 9, 16])
def test_forward_decode_stays_inside_its_workspace(T):
    d, E, k, I, Is = 1024, 24, 6, 512, 512
    case = Case(synth.custom(seed=T, T=T, d=d, E=E, k=k, I=I, I_shared=Is))
    idx, w = draws(T, E, k, 4)
    plan = api.Plan(T, d, E, k, I, Is)
    need = api.moe_plan_workspace_bytes(plan.handle)
    ws = torch.full((need + (32 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    api.moe_plan_set_workspace(plan.handle, ws[:need])
    y = plan.forward_decode(case.x, idx, w, case.experts, case.shared)
    assert plan.check()[0] == 0
    assert bool((ws[need:] == 0x5A).all())
    check_decode(case, idx, w, y)


def test_forward_decode_writes_its_rows_only():
    T, d, E, k, pad = 3, 384, 8, 2, 1024
    case = Case(synth.custom(seed=3, T=8, d=d, E=E, k=k, I=128))
    idx, w = draws(T, E, k, 1)
    buf = torch.full((T * d + pad,), 7, dtype=torch.bfloat16, device="cuda")
    y = buf[:T * d].view(T, d)
    case.plan.forward_decode(case.x[:T].contiguous(), idx, w, case.experts, y=y)
    check_decode(case, idx, w, y, T)
    assert bool((buf[T * d:] == 7).all())


def test_forward_decode_follows_a_router_that_writes_in_place():
    """The second kernel begins before the first is done; ids and weights that the kernel before them has
    just written, over those of the last step, are the ones it uses."""
    T, d, E, k = 4, 256, 64, 8
    case = Case(synth.custom(seed=21, T=T, d=d, E=E, k=k, I=128))
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    w = torch.empty(T, k, dtype=torch.float32, device="cuda")
    xs = [randn((T, d), 300 + i, dtype=torch.bfloat16) for i in range(60)]
    got = []
    for x in xs:
        api.moe_route(case.plan.handle, x, case.W_r, case.bias, k, idx=idx, w=w)
        got.append(case.plan.forward_decode(x, idx, w, case.experts))
    torch.cuda.synchronize()
    for x, y in zip(xs, got):
        i2, w2 = case.plan.route(x, case.W_r, case.bias)
        torch.cuda.synchronize()
        assert torch.equal(case.plan.forward_decode(x, i2, w2, case.experts), y)
        torch.cuda.synchronize()
    assert case.plan.check()[0] == 0


def test_plans_made_and_used_on_another_stream():
    """The workspace may be memory that other work of that stream was still using."""
    T, N, K, d, E, k = 3, 2048, 2048, 512, 16, 4
    q, s, lin, w = linear_case(T, N, K, 77)
    case = Case(synth.custom(seed=8, T=T, d=d, E=E, k=k, I=256))
    idx, wt = draws(T, E, k, 2)
    want = case.plan.forward_decode(case.x, idx, wt, case.experts)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(3):
            n = 64 << 20
            junk = torch.empty(n, dtype=torch.uint8, device="cuda")
            for _ in range(20):
                junk.fill_(255)
            del junk                                   # its block goes to the next plan while the fills run
            plan = api.LinearPlan(T, N, K)
            y = plan.forward(q, s, lin)
            layer_plan = api.Plan(T, d, E, k, 256)
            z = layer_plan.forward_decode(case.x, idx, wt, case.experts)
            assert plan.check(side)[0] == 0 and layer_plan.check(side)[0] == 0
            check_linear(q, s, w, y)
            assert torch.equal(z, want)


# ---------------------------------------------------------------- the three in a row
@pytest.mark.parametrize("T, res", [(1, torch.bfloat16), (6, torch.float32)])
def test_a_decode_step(T, res):
    """norm -> router and experts -> residual and norm of the next block -> a linear, on one stream without a
    wait, against the oracle on the operands each step really had."""
    d, E, k, N = 512, 32, 4, 700
    case = Case(synth.custom(seed=12, T=T, d=d, E=E, k=k, I=256, I_shared=256))
    gamma = [1 + randn((d,), 30 + i, 0.1) for i in range(2)]
    resid = randn((T, d), 40, 2.0, res)
    w_out = randn((N, d), 41, 0.02)
    lin, lplan = api.LinearMXFP4(N, d), api.LinearPlan(T, N, d)
    lin.pack(w_out)
    r1, xn, q, s = api.moe_add_rmsnorm_mxfp8(case.x, gamma[0], residual=resid)
    idx, w = case.plan.route(xn, case.W_r, case.bias)
    y = case.plan.forward_decode(xn, idx, w, case.experts, case.shared, q=q, scale=s)
    r2, xn2, q2, s2 = api.moe_add_rmsnorm_mxfp8(y, gamma[1], residual=r1, with_xn=True)
    logits = lplan.forward(q2, s2, lin, dtype=torch.float32)
    assert case.plan.check()[0] == 0 and lplan.check()[0] == 0
    check_norm(case.x, gamma[0], 1e-5, resid, (r1, xn, q, s))
    z = xn.double().cpu().numpy() @ case.W_r.double().cpu().numpy() + case.bias.double().cpu().numpy()
    top = np.sort(z, axis=1)[:, ::-1]
    for t in range(T):
        if top[t, k - 1] - top[t, k] > 1e-4:
            assert set(idx[t].tolist()) == set(np.argsort(-z[t])[:k].tolist())
    ref = layer.moe_layer(xn.double().cpu().numpy(), idx.cpu().numpy(), w.cpu().numpy(), case.oracle_expert, case.oracle_shared())
    r, _ = layer.relative_errors(y.double().cpu().numpy(), ref)
    assert r.max() <= 2e-2 and r.mean() <= 2e-3
    # the whole step captured once and replayed on another residual
    out = {}

    def step():
        a = api.moe_add_rmsnorm_mxfp8(case.x, gamma[0], residual=resid)
        i, v = case.plan.route(a[1], case.W_r, case.bias)
        z = case.plan.forward_decode(a[1], i, v, case.experts, case.shared, q=a[2], scale=a[3])
        b = api.moe_add_rmsnorm_mxfp8(z, gamma[1], residual=a[0])
        out["logits"] = lplan.forward(b[2], b[3], lin, dtype=torch.float32)
        return out["logits"]

    assert torch.equal(step(), logits)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    captured = out["logits"]
    keep = resid.clone()
    resid.copy_(randn((T, d), 99, 1.0, res))
    g.replay()
    first = captured.clone()
    assert torch.equal(step(), first) and not torch.equal(first, logits)
    resid.copy_(keep)
    g.replay()
    assert torch.equal(captured, logits)
    check_norm(y, gamma[1], 1e-5, r1, (r2, xn2, q2, s2))
    check_linear(q2, s2, w_out, logits)
