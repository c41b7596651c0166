"""Thin ctypes binding to ``libmoe_sm100.so`` (include/moe.h).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current CUDA stream.  There is
no fallback: if the library is missing or cannot load, every call raises.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_sm100.so")

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED_SHAPE",
                3: "MOE_ERR_ALIGNMENT", 4: "MOE_ERR_CUDA", 5: "MOE_ERR_TIMEOUT",
                6: "MOE_ERR_NOT_INITIALIZED", 7: "MOE_ERR_DEVICE_FAULT"}

# exported symbols and their argument types (ctypes)
_P, _I, _S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
# moe_bias_rule_t: (quantiles, n_levels, E, bias, bias_next, stream, user)
BIAS_RULE = ctypes.CFUNCTYPE(None, _P, _I, _I, _P, _P, _P, _P)
SIGNATURES = {
    "moe_plan_create": [_I, _I, _I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(_P)],
    "moe_plan_workspace_bytes": [_P, ctypes.POINTER(_S)],
    "moe_plan_set_workspace": [_P, _P, _S],
    "moe_plan_check": [_P, _P, ctypes.POINTER(ctypes.c_uint)],
    "moe_plan_destroy": [_P],
    "moe_status_string": [_I],
    "moe_quant_mxfp8": [_P, _I, _I, _P, _P, _P],
    "moe_route": [_P, _P, _I, _P, _P, _P, _P, _P, _P],
    "moe_permute": [_P, _P, _I, _P, _P, _P, _P, _P],
    "moe_forward": [_P, _P, _I, _P, _P, _P, _P, _P, _P],
    "moe_expert_bytes": [_I, _I, _I, ctypes.POINTER(_S), ctypes.POINTER(_S), ctypes.POINTER(_S),
                         ctypes.POINTER(_S)],
    "moe_pack_expert_mxfp4": [_I, _I, _I, _P, _P, _P, _P, _P],
    "moe_pack_shared_bf16": [_I, _I, _P, _P, _P, _P, _P],
    "moe_debug_buffer": [_P, _I, ctypes.POINTER(_P), ctypes.POINTER(_S)],
    "moe_debug_timeout_probe": [_P, _P],
    "moe_plan_set_latent": [_P, _I, ctypes.c_float],
    "moe_forward_latent": [_P, _P, _I, _P, _P, _P, _P, _P, _P, _P],
    "moe_plan_set_profiling": [_P, _I],
    "moe_plan_set_option": [_P, _I, _I],
    "moe_plan_get_option": [_P, _I, ctypes.POINTER(_I)],
    "moe_permute_noalloc": [_P, _I, _I, _I, _P, _P, _P, _P, _P],
    "moe_plan_stage_ms": [_P, ctypes.POINTER(ctypes.c_float), ctypes.POINTER(ctypes.c_int), _I],
    "moe_route_margin_quantiles": [_P, _P, _P, _I, ctypes.POINTER(ctypes.c_double), _I, _P, _P],
    "moe_add_rmsnorm_mxfp8": [_P, _P, _I, _P, ctypes.c_float, _I, _I, _P, _P, _P, _P, _P],
    "moe_linear_create": [_I, _I, _I, ctypes.POINTER(_P)],
    "moe_linear_workspace_bytes": [_P, ctypes.POINTER(_S)],
    "moe_linear_set_workspace": [_P, _P, _S],
    "moe_linear_check": [_P, _P, ctypes.POINTER(ctypes.c_uint)],
    "moe_linear_destroy": [_P],
    "moe_linear_tiling": [_P, _I, ctypes.POINTER(_I), ctypes.POINTER(_I)],
    "moe_linear_bytes": [_I, _I, ctypes.POINTER(_S), ctypes.POINTER(_S)],
    "moe_pack_linear_mxfp4": [_I, _I, _P, _P, _P],
    "moe_linear_mxfp4": [_P, _P, _P, _I, _P, _P, _I, _P],
    "moe_forward_decode": [_P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P],
    "moe_quantile_balance": [_P, _P, _P, _I, ctypes.POINTER(ctypes.c_double), _I, BIAS_RULE, _P, _P, _P],
}


STAGES = ["router_split", "router_gemm", "topk", "permute", "quant_scatter", "gate_up_glu",
          "down", "shared_gate_up", "shared_down", "combine", "latent_in", "latent_out"]
# kernel launches per recorded stage instance ("topk" is the selection kernel, which also
# sums the router GEMM's K-split partials)
STAGE_KERNELS = {"permute": 3, "quant_scatter": 2, "latent_in": 2, "latent_out": 2}


class MoeError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(code, code)}")
        self.code = code


class ExpertsMXFP4(ctypes.Structure):
    _fields_ = [("w_gu", _P), ("s_gu", _P), ("w_dn", _P), ("s_dn", _P)]


class SharedBF16(ctypes.Structure):
    _fields_ = [("w_gu", _P), ("w_dn", _P)]


class LatentBF16(ctypes.Structure):
    _fields_ = [("w_down", _P), ("gamma", _P), ("w_up", _P)]


class MatrixMXFP4(ctypes.Structure):
    _fields_ = [("w", _P), ("s", _P)]


_lib = None


def lib():
    """Load the library (raises if it is missing: there is no CPU fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                               "`python -m block_scaled_moe_sigmoid_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, argtypes in SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = argtypes
            fn.restype = ctypes.c_char_p if name == "moe_status_string" else ctypes.c_int
        _lib = L
    return _lib


def _call(name, *args):
    code = getattr(_lib or lib(), name)(*args)
    if code != MOE_OK:
        raise MoeError(name, code)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _checked(name, t, dtype, shape, index):
    """t's data pointer, after checks that a pointer alone cannot carry: type, shape, contiguity, device index."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != index:
        raise ValueError(f"{name}: expected a contiguous {dtype} tensor of shape {tuple(shape)} on CUDA device {index}, got "
                         f"{t.dtype} {tuple(t.shape)} strides {t.stride()} on {t.device}")
    return t.data_ptr()


class _On:
    """A device made current, and a stream: outputs allocated inside belong to it."""

    def __init__(self, index, stream):
        if index < 0:
            raise ValueError("expected CUDA tensors")
        if stream is not None and stream.device.index != index:
            raise ValueError(f"a stream of {stream.device} for tensors on CUDA device {index}")
        self.guards = [torch.cuda.device(index)] + ([torch.cuda.stream(stream)] if stream is not None else [])

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _elsewhere(index, stream):
    """Whether a call on device `index` and `stream` needs _On around it."""
    return stream is not None or index < 0 or index != torch.cuda.current_device()


def _raw_stream(index):
    """The handle of the current stream of a device."""
    return torch._C._cuda_getCurrentRawStream(index)


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


# ------------------------------------------------------------------ same names as the C ABI
def moe_plan_create(T_max, d, E, k, I, I_shared=0, act=0, bias_mode=0, flags=0):
    h = ctypes.c_void_p()
    _call("moe_plan_create", T_max, d, E, k, I, I_shared, act, bias_mode, flags, ctypes.byref(h))
    return h


def moe_plan_workspace_bytes(plan):
    n = ctypes.c_size_t()
    _call("moe_plan_workspace_bytes", plan, ctypes.byref(n))
    return n.value


def moe_plan_set_workspace(plan, ws):
    _call("moe_plan_set_workspace", plan, _ptr(ws), ws.numel() * ws.element_size())


def moe_plan_check(plan, stream=None):
    bits = ctypes.c_uint()
    code = lib().moe_plan_check(plan, _stream(stream), ctypes.byref(bits))
    return code, bits.value


def moe_debug_timeout_probe(plan, stream=None):
    """One bounded wait that runs out on the GPU (see include/moe.h)."""
    _call("moe_debug_timeout_probe", plan, _stream(stream))


def moe_plan_destroy(plan):
    _call("moe_plan_destroy", plan)


def moe_quant_mxfp8(x, q=None, scale=None, stream=None):
    """x: cuda bf16 [rows, cols] -> (q uint8 [rows, cols], scale uint8 [rows, cols/32])."""
    rows, cols = x.shape
    q = torch.empty((rows, cols), dtype=torch.uint8, device=x.device) if q is None else q
    scale = torch.empty((rows, cols // 32), dtype=torch.uint8, device=x.device) if scale is None else scale
    _call("moe_quant_mxfp8", _ptr(x), rows, cols, _ptr(q), _ptr(scale), _stream(stream))
    return q, scale


def moe_route(plan, x, W_r, bias, k, idx=None, w=None, logits=None, stream=None):
    T = x.shape[0]
    idx = torch.empty((T, k), dtype=torch.int32, device=x.device) if idx is None else idx
    w = torch.empty((T, k), dtype=torch.float32, device=x.device) if w is None else w
    _call("moe_route", plan, _ptr(x), T, _ptr(W_r), _ptr(bias), _ptr(idx), _ptr(w), _ptr(logits),
          _stream(stream))
    return idx, w


def moe_permute(plan, idx, E, stream=None):
    T, k = idx.shape
    dev = idx.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm_tok = torch.empty(T * k, dtype=torch.int32, device=dev)
    inv = torch.empty((T, k), dtype=torch.int32, device=dev)
    _call("moe_permute", plan, _ptr(idx), T, _ptr(counts), _ptr(offsets), _ptr(perm_tok), _ptr(inv),
          _stream(stream))
    return counts, offsets, perm_tok, inv


def moe_permute_noalloc(idx, E, stream=None):
    """moe_permute for callers that cannot allocate device memory: the library uses its own
    fixed device scratch array (see include/moe.h for the size limit).  The output
    tensors here are allocated by torch for convenience."""
    T, k = idx.shape
    dev = idx.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm_tok = torch.empty(T * k, dtype=torch.int32, device=dev)
    inv = torch.empty((T, k), dtype=torch.int32, device=dev)
    _call("moe_permute_noalloc", _ptr(idx), T, E, k, _ptr(counts), _ptr(offsets), _ptr(perm_tok),
          _ptr(inv), _stream(stream))
    return counts, offsets, perm_tok, inv


def moe_forward(plan, x, idx, w, experts, shared, y=None, stream=None):
    T, d = x.shape
    y = torch.empty((T, d), dtype=torch.bfloat16, device=x.device) if y is None else y
    ex = experts.struct()
    sh = shared.struct() if shared is not None else None
    _call("moe_forward", plan, _ptr(x), T, _ptr(idx), _ptr(w), ctypes.byref(ex),
          ctypes.byref(sh) if sh is not None else None, _ptr(y), _stream(stream))
    return y


def moe_forward_latent(plan, x, idx, w, latent, experts, shared, y=None, stream=None):
    T, d = x.shape
    y = torch.empty((T, d), dtype=torch.bfloat16, device=x.device) if y is None else y
    lat = latent.struct()
    ex = experts.struct()
    sh = shared.struct() if shared is not None else None
    _call("moe_forward_latent", plan, _ptr(x), T, _ptr(idx), _ptr(w), ctypes.byref(lat), ctypes.byref(ex),
          ctypes.byref(sh) if sh is not None else None, _ptr(y), _stream(stream))
    return y


def moe_route_margin_quantiles(plan, logits, E, levels, select_bias=None, quantiles=None, stream=None):
    """Per-expert quantiles of the routing margins of logits [T, E] (fp32, device) at the
    given levels; returns fp32 [len(levels), E] on the device."""
    T = logits.shape[0]
    lv = (ctypes.c_double * len(levels))(*levels)
    if quantiles is None:
        quantiles = torch.empty((len(levels), E), dtype=torch.float32, device=logits.device)
    _call("moe_route_margin_quantiles", plan, _ptr(logits), _ptr(select_bias), T, lv, len(levels),
          _ptr(quantiles), _stream(stream))
    return quantiles


def moe_quantile_balance(plan, logits, bias, levels, rule, bias_next=None, user=None, stream=None):
    """Margin quantiles of this step, then the caller's rule (a BIAS_RULE callable) writes the
    next step's bias into bias_next (fp32 [E], device)."""
    T = logits.shape[0]
    lv = (ctypes.c_double * len(levels))(*levels)
    if bias_next is None:
        bias_next = torch.empty_like(bias)
    _call("moe_quantile_balance", plan, _ptr(logits), _ptr(bias), T, lv, len(levels), rule, user,
          _ptr(bias_next), _stream(stream))
    return bias_next


def moe_expert_bytes(d, I, E):
    a, b, c, e = (ctypes.c_size_t() for _ in range(4))
    _call("moe_expert_bytes", d, I, E, ctypes.byref(a), ctypes.byref(b), ctypes.byref(c), ctypes.byref(e))
    return a.value, b.value, c.value, e.value


def moe_pack_expert_mxfp4(d, I, e, w_gate, w_up, w_down, experts, stream=None):
    ex = experts.struct()
    _call("moe_pack_expert_mxfp4", d, I, e, _ptr(w_gate), _ptr(w_up), _ptr(w_down), ctypes.byref(ex),
          _stream(stream))


def moe_pack_shared_bf16(d, I_shared, w_gate, w_up, w_down, shared, stream=None):
    sh = shared.struct()
    _call("moe_pack_shared_bf16", d, I_shared, _ptr(w_gate), _ptr(w_up), _ptr(w_down), ctypes.byref(sh),
          _stream(stream))


MOE_TYPE_BF16, MOE_TYPE_F32 = 0, 1
_TYPES = {torch.bfloat16: MOE_TYPE_BF16, torch.float32: MOE_TYPE_F32}


def _type(name, dtype):
    if dtype not in _TYPES:
        raise ValueError(f"{name}: expected torch.bfloat16 or torch.float32, got {dtype}")
    return _TYPES[dtype]


def moe_add_rmsnorm_mxfp8(x, gamma, eps=1e-5, residual=None, residual_out=None, xn=None, q=None, scale=None,
                          with_xn=True, with_mx=True, stream=None):
    """r = x + residual (x alone without one), the RMSNorm of r as bf16 and as MXFP8.

    x: bf16 [rows, cols]; gamma: fp32 [cols]; residual: bf16 or fp32 [rows, cols] or None.
    Returns (r in the residual's type or None, xn bf16, q uint8 [rows, cols], scale uint8
    [rows, cols / 32]).  Outputs are allocated where not given; residual_out may be the residual
    itself.  with_xn / with_mx = False leave xn / (q, scale) out (None)."""
    i = x.get_device()
    if _elsewhere(i, stream):
        with _On(i, stream):
            return moe_add_rmsnorm_mxfp8(x, gamma, eps, residual, residual_out, xn, q, scale, with_xn, with_mx)
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"x: expected [rows, cols], got {tuple(shape)}")
    if (xn is not None and not with_xn) or ((q is not None or scale is not None) and not with_mx):
        raise ValueError("an output was given that with_xn / with_mx leave out")
    rows, cols = shape
    blocks = (rows, cols // 32)
    px = _checked("x", x, torch.bfloat16, shape, i)
    rtype, pr, pro, pn, pq, ps = MOE_TYPE_BF16, None, None, None, None, None
    if residual is not None:
        rtype, pr = _type("residual", residual.dtype), _checked("residual", residual, residual.dtype, shape, i)
        if residual_out is None:
            residual_out = torch.empty_like(residual)
            pro = residual_out.data_ptr()
        else:
            pro = _checked("residual_out", residual_out, residual.dtype, shape, i)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if with_xn:
        if xn is None:
            xn = torch.empty_like(x)
            pn = xn.data_ptr()
        else:
            pn = _checked("xn", xn, torch.bfloat16, shape, i)
    if with_mx:
        if q is None:
            q = torch.empty_like(x, dtype=torch.uint8)
            pq = q.data_ptr()
        else:
            pq = _checked("q", q, torch.uint8, shape, i)
        if scale is None:
            scale = torch.empty_strided(blocks, (blocks[1], 1), dtype=torch.uint8, device=x.device)
            ps = scale.data_ptr()
        else:
            ps = _checked("scale", scale, torch.uint8, blocks, i)
    _call("moe_add_rmsnorm_mxfp8", px, pr, rtype, _checked("gamma", gamma, torch.float32, (cols,), i), eps, rows, cols, pro,
          pn, pq, ps, _raw_stream(i))
    return residual_out, xn, q, scale


def moe_linear_create(T_max, N, K):
    h = ctypes.c_void_p()
    _call("moe_linear_create", T_max, N, K, ctypes.byref(h))
    return h


def moe_linear_workspace_bytes(linear):
    n = ctypes.c_size_t()
    _call("moe_linear_workspace_bytes", linear, ctypes.byref(n))
    return n.value


def moe_linear_set_workspace(linear, ws):
    _call("moe_linear_set_workspace", linear, _ptr(ws), ws.numel() * ws.element_size())


def moe_linear_check(linear, stream=None):
    bits = ctypes.c_uint()
    code = lib().moe_linear_check(linear, _stream(stream), ctypes.byref(bits))
    return code, bits.value


def moe_linear_destroy(linear):
    _call("moe_linear_destroy", linear)


def moe_linear_tiling(linear, T):
    """(token rows of a tile, or 0 where a call with T rows is a stream of the weights; whether tiles are split along K)."""
    rows, split = ctypes.c_int(), ctypes.c_int()
    _call("moe_linear_tiling", linear, T, ctypes.byref(rows), ctypes.byref(split))
    return rows.value, bool(split.value)


def moe_linear_bytes(N, K):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    _call("moe_linear_bytes", N, K, ctypes.byref(a), ctypes.byref(b))
    return a.value, b.value


def moe_pack_linear_mxfp4(N, K, w, weights, stream=None):
    i = weights.w.get_device()
    if _elsewhere(i, stream):
        with _On(i, stream):
            return moe_pack_linear_mxfp4(N, K, w, weights)
    _call("moe_pack_linear_mxfp4", N, K, _checked("w", w, torch.float32, (N, K), i), ctypes.byref(weights.struct()),
          _raw_stream(i))


def moe_linear_mxfp4(linear, q, scale, weights, y=None, dtype=torch.bfloat16, stream=None):
    """y [T, N] (bf16 or fp32) = W x for MXFP8 rows q uint8 [T, K], scale uint8 [T, K / 32] and a
    LinearMXFP4 on `linear`, a handle of moe_linear_create for its shape."""
    i = weights.w.get_device()
    if _elsewhere(i, stream):
        with _On(i, stream):
            return moe_linear_mxfp4(linear, q, scale, weights, y, dtype)
    N, K, T = weights.N, weights.K, q.shape[0]
    if y is None:
        y = torch.empty_strided((T, N), (N, 1), dtype=dtype, device=q.device)
    _call("moe_linear_mxfp4", linear, _checked("q", q, torch.uint8, (T, K), i),
          _checked("scale", scale, torch.uint8, (T, K // 32), i), T, ctypes.byref(weights.struct()),
          _checked("y", y, y.dtype, (T, N), i), _type("y", y.dtype), _raw_stream(i))
    return y


def moe_forward_decode(plan, x, idx, w, experts, shared=None, q=None, scale=None, y=None, stream=None):
    """The layer for up to 16 tokens x bf16 [T, d]; (q, scale) is their MXFP8 form where it is at
    hand, and x may then be None without a shared expert."""
    i = experts.w_gu.get_device()
    if _elsewhere(i, stream):
        with _On(i, stream):
            return moe_forward_decode(plan, x, idx, w, experts, shared, q, scale, y)
    routes = idx.shape
    if len(routes) != 2:
        raise ValueError(f"idx: expected [T, k], got {tuple(routes)}")
    T, d = routes[0], experts.d
    if y is None:
        y = torch.empty_strided((T, d), (d, 1), dtype=torch.bfloat16, device=idx.device)
    _call("moe_forward_decode", plan, _checked("x", x, torch.bfloat16, (T, d), i), _checked("q", q, torch.uint8, (T, d), i),
          _checked("scale", scale, torch.uint8, (T, d // 32), i), T, _checked("idx", idx, torch.int32, routes, i),
          _checked("w", w, torch.float32, routes, i), ctypes.byref(experts.struct()),
          ctypes.byref(shared.struct()) if shared is not None else None, _checked("y", y, torch.bfloat16, (T, d), i),
          _raw_stream(i))
    return y


def moe_debug_buffer(plan, which):
    """(device pointer, bytes) of a workspace buffer (see include/moe.h)."""
    p, n = ctypes.c_void_p(), ctypes.c_size_t()
    _call("moe_debug_buffer", plan, which, ctypes.byref(p), ctypes.byref(n))
    return p.value, n.value


MOE_OPT_PREFETCH_DIST, MOE_OPT_PREFETCH_B, MOE_OPT_TILE_N, MOE_OPT_ROUTER_SPLIT = 0, 1, 2, 3
MOE_OPT_SHARED_SPLIT, MOE_OPT_SHARED_SPLIT_DOWN = 4, 5


def moe_plan_set_option(plan, option, value):
    _call("moe_plan_set_option", plan, option, int(value))


def moe_plan_get_option(plan, option):
    v = ctypes.c_int()
    _call("moe_plan_get_option", plan, option, ctypes.byref(v))
    return v.value


def moe_plan_set_profiling(plan, enable=True):
    _call("moe_plan_set_profiling", plan, 1 if enable else 0)


def moe_plan_stage_ms(plan):
    """{stage: (summed ms, recorded launches)} since profiling was enabled / last queried."""
    n = len(STAGES)
    ms = (ctypes.c_float * n)()
    cnt = (ctypes.c_int * n)()
    _call("moe_plan_stage_ms", plan, ms, cnt, n)
    return {STAGES[i]: (ms[i], cnt[i]) for i in range(n)}


# ------------------------------------------------------------------ buffers
class Experts:
    """Device buffers of packed MXFP4 experts (allocated by torch)."""

    def __init__(self, d, I, E, device="cuda"):
        self.d, self.I, self.E = d, I, E
        sizes = moe_expert_bytes(d, I, E)
        # 256-byte aligned allocations (torch's caching allocator returns 512-aligned blocks)
        self.w_gu, self.s_gu, self.w_dn, self.s_dn = (
            torch.empty(n, dtype=torch.uint8, device=device) for n in sizes)

    def struct(self):
        return ExpertsMXFP4(self.w_gu.data_ptr(), self.s_gu.data_ptr(), self.w_dn.data_ptr(),
                            self.s_dn.data_ptr())

    def pack(self, e, w_gate, w_up, w_down, stream=None):
        with _On(self.w_gu.get_device(), stream):   # copies of strided weights belong to the stream that packs them
            moe_pack_expert_mxfp4(self.d, self.I, e, w_gate.contiguous(), w_up.contiguous(),
                                  w_down.contiguous(), self)


class Shared:
    def __init__(self, d, I_shared, device="cuda"):
        self.d, self.I_shared = d, I_shared
        self.w_gu = torch.empty((2 * I_shared, d), dtype=torch.bfloat16, device=device)
        self.w_dn = torch.empty((d, I_shared), dtype=torch.bfloat16, device=device)

    def struct(self):
        return SharedBF16(self.w_gu.data_ptr(), self.w_dn.data_ptr())

    def pack(self, w_gate, w_up, w_down, stream=None):
        with _On(self.w_gu.get_device(), stream):   # as Experts.pack
            moe_pack_shared_bf16(self.d, self.I_shared, w_gate.contiguous(), w_up.contiguous(),
                                 w_down.contiguous(), self)


class LinearMXFP4:
    """Device buffers of a packed MXFP4 matrix [N, K] (allocated by torch)."""

    def __init__(self, N, K, device="cuda"):
        self.N, self.K = N, K
        self.w, self.s = (torch.empty(n, dtype=torch.uint8, device=device) for n in moe_linear_bytes(N, K))

    def struct(self):
        return MatrixMXFP4(self.w.data_ptr(), self.s.data_ptr())

    def pack(self, w, stream=None):
        with _On(self.w.get_device(), stream):   # as Experts.pack
            moe_pack_linear_mxfp4(self.N, self.K, w.contiguous(), self)


class LinearPlan:
    """A handle for MXFP4 linears of one shape plus its torch-allocated workspace."""

    def __init__(self, T_max, N, K, device="cuda"):
        self.T_max, self.N, self.K = T_max, N, K
        self.handle = None
        with torch.cuda.device(device):
            self.handle = moe_linear_create(T_max, N, K)
            self.workspace = torch.empty(moe_linear_workspace_bytes(self.handle), dtype=torch.uint8, device=device)
            torch.cuda.current_stream(self.workspace.device).synchronize()   # the memory's earlier user
            moe_linear_set_workspace(self.handle, self.workspace)

    def forward(self, q, scale, weights, y=None, dtype=torch.bfloat16, stream=None):
        if (weights.N, weights.K) != (self.N, self.K) or weights.w.device != self.workspace.device:
            raise ValueError(f"weights [{weights.N}, {weights.K}] on {weights.w.device}: the plan is for [{self.N}, {self.K}] "
                             f"on {self.workspace.device}")
        return moe_linear_mxfp4(self.handle, q, scale, weights, y, dtype, stream)

    def check(self, stream=None):
        return moe_linear_check(self.handle, stream)

    def __del__(self):
        try:
            if getattr(self, "handle", None) is not None:
                moe_linear_destroy(self.handle)
                self.handle = None
        except Exception:
            pass


MOE_ACT_SILU_GLU, MOE_ACT_CLAMPED_SWIGLU = 0, 1
MOE_BIAS_LOGIT, MOE_BIAS_SELECT_ONLY = 0, 1
MOE_FLAG_STATIC_ROUTER = 1


class Latent:
    """Latent-option weights on the device: W_ld bf16 [d_latent][d], gamma fp32 [d_latent],
    W_lu bf16 [d][d_latent]."""

    def __init__(self, w_down, gamma, w_up):
        self.w_down = w_down.to(torch.bfloat16).contiguous()
        self.gamma = gamma.to(torch.float32).contiguous()
        self.w_up = w_up.to(torch.bfloat16).contiguous()

    def struct(self):
        return LatentBF16(self.w_down.data_ptr(), self.gamma.data_ptr(), self.w_up.data_ptr())


class Plan:
    """A plan plus its torch-allocated workspace."""

    def __init__(self, T_max, d, E, k, I, I_shared=0, device="cuda", act=MOE_ACT_SILU_GLU,
                 bias_mode=MOE_BIAS_LOGIT, flags=0, d_latent=0, eps=1e-5):
        self.T_max, self.d, self.E, self.k, self.I, self.I_shared = T_max, d, E, k, I, I_shared
        self.act, self.bias_mode, self.flags, self.d_latent = act, bias_mode, flags, d_latent
        self.handle = moe_plan_create(T_max, d, E, k, I, I_shared, act, bias_mode, flags)
        if d_latent:
            _call("moe_plan_set_latent", self.handle, d_latent, ctypes.c_float(eps))
        n = moe_plan_workspace_bytes(self.handle)
        self.workspace = torch.empty(max(n, 256), dtype=torch.uint8, device=device)
        torch.cuda.current_stream(self.workspace.device).synchronize()   # the memory's earlier user
        moe_plan_set_workspace(self.handle, self.workspace)

    def route(self, x, W_r, bias=None, logits=None, stream=None):
        return moe_route(self.handle, x, W_r, bias, self.k, logits=logits, stream=stream)

    def permute(self, idx, stream=None):
        return moe_permute(self.handle, idx, self.E, stream)

    def forward(self, x, idx, w, experts, shared=None, y=None, stream=None, latent=None):
        if self.d_latent:
            return moe_forward_latent(self.handle, x, idx, w, latent, experts, shared, y, stream)
        return moe_forward(self.handle, x, idx, w, experts, shared, y, stream)

    def forward_decode(self, x, idx, w, experts, shared=None, q=None, scale=None, y=None, stream=None):
        """forward for up to 16 tokens, from their MXFP8 form (q, scale) where it is given."""
        if (experts.d, experts.I, experts.E, idx.shape[-1]) != (self.d, self.I, self.E, self.k):
            raise ValueError(f"experts d={experts.d} I={experts.I} E={experts.E}, idx {tuple(idx.shape)}: the plan has "
                             f"d={self.d} I={self.I} E={self.E} k={self.k}")
        if shared is not None and (shared.d, shared.I_shared) != (self.d, self.I_shared):
            raise ValueError(f"shared expert d={shared.d} I_shared={shared.I_shared}: the plan has d={self.d} "
                             f"I_shared={self.I_shared}")
        return moe_forward_decode(self.handle, x, idx, w, experts, shared, q, scale, y, stream)

    def check(self, stream=None):
        return moe_plan_check(self.handle, stream)

    def debug_tensor(self, which, dtype, shape):
        """A torch view of a workspace buffer (copy it before the next call)."""
        ptr, n = moe_debug_buffer(self.handle, which)
        off = ptr - self.workspace.data_ptr()
        count = 1
        for s in shape:
            count *= s
        nbytes = count * torch.empty((), dtype=dtype).element_size()
        assert 0 <= off and nbytes <= n
        return self.workspace[off:off + nbytes].view(dtype).view(*shape)

    def __del__(self):
        try:
            if getattr(self, "handle", None) is not None:
                moe_plan_destroy(self.handle)
                self.handle = None
        except Exception:
            pass
