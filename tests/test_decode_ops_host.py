"""Refusals of the operators around a decode step, without a GPU: every check stands before the
first launch, so made-up pointers are never followed."""
import ctypes
from types import SimpleNamespace

import pytest
import torch

from block_scaled_moe_sigmoid_b200 import api

P = ctypes.c_void_p
INVALID, SHAPE, ALIGN, NOT_INIT = 1, 2, 3, 6
A = P(1 << 20)          # an aligned address
B = P((1 << 20) + 8)    # one that is only 8-byte aligned


def norm(x=A, res=None, rtype=0, gamma=A, eps=1e-5, rows=4, cols=64, res_out=None, xn=A, q=A, scale=A):
    return api.lib().moe_add_rmsnorm_mxfp8(x, res, rtype, gamma, ctypes.c_float(eps), rows, cols, res_out, xn, q, scale, None)


@pytest.mark.parametrize("kw, code", [
    (dict(rows=-1), INVALID), (dict(cols=0), INVALID), (dict(cols=33), SHAPE), (dict(cols=32768 + 32), SHAPE),
    (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(rtype=2), INVALID), (dict(rtype=-1), INVALID),
    (dict(x=None), INVALID), (dict(gamma=None), INVALID),
    (dict(q=None), INVALID), (dict(scale=None), INVALID),                 # codes and scales come together
    (dict(xn=None, q=None, scale=None), INVALID),                         # no output at all
    (dict(res_out=A), INVALID),                                           # an output without its input
    (dict(x=B), ALIGN), (dict(res=B), ALIGN), (dict(gamma=B), ALIGN), (dict(res=A, res_out=B), ALIGN),
    (dict(xn=B), ALIGN), (dict(q=B), ALIGN),
    (dict(rows=0), 0), (dict(rows=0, x=None, gamma=None), 0),
])
def test_norm_refusals(kw, code):
    assert norm(**kw) == code


def test_linear_create_and_size_refusals():
    L, h = api.lib(), P()
    for args, code in (((-1, 8, 128), INVALID), ((8, 0, 128), INVALID), ((8, 8, 0), INVALID), ((8, 8, 96), SHAPE),
                       ((8, 1 << 30, 1 << 15), SHAPE), ((8, 8, (1 << 22) + 128), SHAPE), (((1 << 30) + 1, 8, 128), SHAPE)):
        assert L.moe_linear_create(*args, ctypes.byref(h)) == code, args
        assert not h
    assert L.moe_linear_create(8, 8, 128, None) == INVALID
    w, s = ctypes.c_size_t(), ctypes.c_size_t()
    assert L.moe_linear_bytes(8, 100, ctypes.byref(w), ctypes.byref(s)) == SHAPE
    assert L.moe_linear_bytes(0, 128, ctypes.byref(w), ctypes.byref(s)) == INVALID
    assert api.moe_linear_bytes(257, 384) == (2 * 3 * 16384, 2 * 3 * 1024)   # two m-tiles, three K tiles
    assert L.moe_linear_workspace_bytes(None, ctypes.byref(w)) == INVALID
    assert L.moe_linear_check(None, None, None) == INVALID
    assert L.moe_linear_destroy(None) == INVALID
    m = api.MatrixMXFP4(A.value, A.value)
    assert L.moe_pack_linear_mxfp4(8, 100, A, ctypes.byref(m), None) == SHAPE
    assert L.moe_pack_linear_mxfp4(8, 128, None, ctypes.byref(m), None) == INVALID
    assert L.moe_pack_linear_mxfp4(8, 128, B, ctypes.byref(m), None) == ALIGN
    assert L.moe_pack_linear_mxfp4(8, 128, A, ctypes.byref(api.MatrixMXFP4(A.value, None)), None) == INVALID
    assert L.moe_pack_linear_mxfp4(8, 128, A, ctypes.byref(api.MatrixMXFP4(A.value + 16, A.value)), None) == ALIGN


def test_linear_call_refusals():
    L = api.lib()
    h = api.moe_linear_create(16, 40, 256)
    m = api.MatrixMXFP4(A.value, A.value)

    def call(h=h, q=A, s=A, T=4, w=m, y=A, ytype=0):
        return L.moe_linear_mxfp4(h, q, s, T, ctypes.byref(w) if w is not None else None, y, ytype, None)

    assert call(h=None) == INVALID
    assert call(T=-1) == INVALID and call(T=17) == SHAPE and call(ytype=2) == INVALID
    assert call(q=None) == INVALID and call(s=None) == INVALID and call(w=None) == INVALID and call(y=None) == INVALID
    assert call(w=api.MatrixMXFP4(None, A.value)) == INVALID and call(w=api.MatrixMXFP4(A.value, None)) == INVALID
    assert call(q=B) == ALIGN and call(y=B) == ALIGN and call(s=P((1 << 20) + 2)) == ALIGN
    assert call(w=api.MatrixMXFP4(A.value + 16, A.value)) == ALIGN
    assert call() == NOT_INIT                                # no workspace attached
    assert call(T=0) == 0
    assert L.moe_linear_set_workspace(h, B, 1 << 40) == ALIGN
    assert L.moe_linear_set_workspace(h, A, 16) == INVALID   # too small
    assert L.moe_linear_set_workspace(h, None, 1 << 40) == INVALID
    assert L.moe_linear_check(h, None, None) == NOT_INIT
    api.moe_linear_destroy(h)


def test_linear_workspace_bounds():
    """The partials of the weight stream are always there; a split K needs room only past 8 rows."""
    L = api.lib()
    n = []
    for T, N, K in ((1, 256, 7168), (8, 256, 7168), (300, 256, 7168), (8192, 7168, 7168)):
        h = api.moe_linear_create(T, N, K)
        n.append(api.moe_linear_workspace_bytes(h))
        L.moe_linear_destroy(h)
    assert 4 << 20 <= n[0] <= n[1] <= n[2] <= n[3] < 80 << 20


def test_forward_decode_refusals():
    L = api.lib()
    h = api.moe_plan_create(64, 256, 8, 2, 128)
    hs = api.moe_plan_create(64, 256, 8, 2, 128, 128)
    lat = api.moe_plan_create(64, 256, 8, 2, 128)
    assert L.moe_plan_set_latent(lat, 128, ctypes.c_float(1e-5)) == 0
    ex, sh = api.ExpertsMXFP4(*[A.value] * 4), api.SharedBF16(A.value, A.value)

    def call(h=h, x=A, q=None, s=None, T=4, idx=A, w=A, ex=ex, sh=None, y=A):
        ref = lambda v: ctypes.byref(v) if v is not None else None  # noqa: E731
        return L.moe_forward_decode(h, x, q, s, T, idx, w, ref(ex), ref(sh), y, None)

    assert call(h=None) == INVALID and call(h=lat) == INVALID
    assert call(T=-1) == INVALID and call(T=17) == SHAPE
    assert call(x=None) == INVALID                                    # neither form of the tokens
    assert call(q=A) == INVALID and call(s=A) == INVALID              # codes and scales come together
    assert call(idx=None) == INVALID and call(w=None) == INVALID and call(y=None) == INVALID and call(ex=None) == INVALID
    assert call(ex=api.ExpertsMXFP4(A.value, A.value, A.value, None)) == INVALID
    assert call(sh=sh) == INVALID                                     # the plan has no shared expert
    assert call(h=hs) == INVALID                                      # the plan has one
    assert call(h=hs, sh=api.SharedBF16(A.value, None)) == INVALID
    assert call(h=hs, sh=sh, x=None, q=A, s=A) == INVALID             # the shared expert reads x
    assert call(x=B) == ALIGN and call(q=B, s=A) == ALIGN and call(y=B) == ALIGN
    assert call(ex=api.ExpertsMXFP4(A.value + 16, A.value, A.value, A.value)) == ALIGN
    assert call() == NOT_INIT and call(x=None, q=A, s=A) == NOT_INIT and call(h=hs, sh=sh) == NOT_INIT
    assert call(T=0) == 0
    for p in (h, hs, lat):
        api.moe_plan_destroy(p)


def test_binding_refuses_what_a_pointer_cannot_carry():
    x, g = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64)
    with pytest.raises(ValueError):
        api.moe_add_rmsnorm_mxfp8(x, g)                        # host tensors
    with pytest.raises(ValueError):
        api.moe_add_rmsnorm_mxfp8(x[0], g)                     # one dimension
    with pytest.raises(ValueError):
        api.moe_add_rmsnorm_mxfp8(x, g, residual=x.half())     # a residual type that is not offered
    with pytest.raises(ValueError):
        api.moe_add_rmsnorm_mxfp8(x, g, residual_out=x)
    with pytest.raises(ValueError):
        api.moe_add_rmsnorm_mxfp8(x, g, xn=x, with_xn=False)
    host = -1
    ok = torch.zeros(4, 8)
    assert api._checked("t", None, torch.float32, (4, 8), host) is None
    assert api._checked("t", ok, torch.float32, (4, 8), host) == ok.data_ptr()
    for t, dtype, shape in ((ok.double(), torch.float32, (4, 8)), (ok, torch.float32, (8, 4)), (ok[:, ::2], torch.float32, (4, 4)),
                            (ok.t(), torch.float32, (8, 4))):
        with pytest.raises(ValueError):
            api._checked("t", t, dtype, shape, host)
    with pytest.raises(ValueError):
        api._checked("t", ok, torch.float32, (4, 8), 0)


def test_packing_copies_strided_weights_on_its_own_stream(monkeypatch):
    """The copy that makes a strided weight contiguous is ordered with the packing that reads it, and its memory goes
    back to that stream."""
    packed = [api.LinearMXFP4(64, 128, device="cpu"), api.Experts(128, 128, 1, device="cpu"), api.Shared(128, 128, device="cpu")]
    log = []

    class On:
        def __init__(self, index, stream):
            self.stream = stream

        def __enter__(self):
            log.append(("on", self.stream))

        def __exit__(self, *exc):
            log.append("off")

    class Weight(torch.Tensor):
        def contiguous(self):
            log.append("copy")
            return torch.Tensor.contiguous(self).as_subclass(torch.Tensor)

    monkeypatch.setattr(api, "_On", On)
    monkeypatch.setattr(api, "_elsewhere", lambda index, stream: stream is not None)
    monkeypatch.setattr(api, "_stream", lambda stream=None: stream)
    monkeypatch.setattr(api, "_raw_stream", lambda index: None)
    monkeypatch.setattr(api, "_call", lambda name, *args: log.append(name))
    square, tall = torch.zeros(128, 128).as_subclass(Weight).t(), torch.zeros(128, 64).as_subclass(Weight).t()
    for buffers, args in zip(packed, ((tall,), (0, square, square, square), (square, square, square))):
        log.clear()
        buffers.pack(*args, stream="side")
        copies = sum(isinstance(a, torch.Tensor) for a in args)
        assert log[0] == ("on", "side") and log[-1] == "off" and log[1:-2] == ["copy"] * copies
        assert log[-2].startswith("moe_pack_")


def linear_tiling(T, N, K, T_max=None):
    h = api.moe_linear_create(T if T_max is None else T_max, N, K)
    try:
        return api.moe_linear_tiling(h, T)
    finally:
        api.moe_linear_destroy(h)


def test_linear_tiling_refusals():
    L, n, split = api.lib(), ctypes.c_int(), ctypes.c_int()
    h = api.moe_linear_create(64, 512, 256)
    for args, code in (((None, 4, n, split), INVALID), ((h, -1, n, split), INVALID), ((h, 65, n, split), SHAPE),
                       ((h, 4, None, split), INVALID), ((h, 4, n, None), INVALID), ((h, 0, n, split), 0), ((h, 64, n, split), 0)):
        assert L.moe_linear_tiling(args[0], args[1], *(ctypes.byref(a) if a is not None else None for a in args[2:])) == code, args
    api.moe_linear_destroy(h)


@pytest.mark.parametrize("N", [256, 576, 1003, 1536, 4096, 7168])
def test_linear_tiling_has_no_jump(N):
    """One row more does not change how a prompt is cut, and narrow outputs use most of the 148 SMs at any length."""
    K = 7168
    assert linear_tiling(16, N, K) == (0, False)
    assert linear_tiling(1025, N, K) == linear_tiling(1024, N, K)
    for T in (1025, 2048, 4096, 8192):
        rows, split = linear_tiling(T, N, K)
        assert 16 <= rows <= 176 and rows % 16 == 0
        tiles = -(-T // rows) * -(-N // 256)
        assert split or tiles >= 96, (T, rows, tiles)


def test_linear_tiling_keeps_the_steps_countable():
    """Tiles of few rows would be more than 2^31 steps; the choice is among those that are not."""
    T, N, K = 1 << 23, 1 << 20, 128
    rows, split = linear_tiling(T, N, K)
    assert -(-T // rows) * (N // 256) * (K // 128) < 1 << 31


def test_a_stream_of_another_device_is_refused():
    """Not replaced by the current stream of the tensors' device."""
    with pytest.raises(ValueError, match="cuda:1"):
        api._On(0, SimpleNamespace(device=torch.device("cuda", 1)))
    with pytest.raises(ValueError):
        api._On(-1, None)
    weights = SimpleNamespace(w=SimpleNamespace(get_device=lambda: 0), N=8, K=128)
    other = SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="cuda:1"):
        api.moe_linear_mxfp4(None, torch.zeros(1, 128, dtype=torch.uint8), torch.zeros(1, 4, dtype=torch.uint8), weights, stream=other)
