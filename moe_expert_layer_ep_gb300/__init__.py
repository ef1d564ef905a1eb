"""Python binding of libmoe, the GB300 (sm_103a) MoE expert-layer library.

Argument marshalling only: every step of the layer runs in libmoe's CUDA
kernels; this module turns torch tensors into device pointers and the current
torch stream into a cudaStream_t, and raises on error codes.  PyTorch supplies
device memory and streams.  Importing fails loudly when libmoe.so has not
been built (run ``python moe_expert_layer_ep_gb300/build.py`` or
``__graft_entry__.build()``); there is no
fallback implementation.

The C functions and their contracts are declared in include/moe.h; the
functions here carry the same names.
"""

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

MOE_DTYPE_FP8 = 0
MOE_DTYPE_BF16 = 1
MOE_DTYPE_MXFP8 = 2
MOE_DTYPE_MXFP4 = 3
MOE_ELEM_BF16 = 0
MOE_ELEM_F32 = 1
MOE_ACTS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3, "relu": 4, "relu2": 5}   # moe_act_t
MOE_LAYOUT_AUTO = 0
MOE_LAYOUT_COMPACT = 1
MOE_LAYOUT_MASKED = 2

STATUS_NAMES = {
    0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED", 3: "MOE_ERR_BUFFER_TOO_SMALL",
    4: "MOE_ERR_MISALIGNED", 5: "MOE_ERR_CUDA", 6: "MOE_ERR_EXPERT_ID", 7: "MOE_ERR_MASKED_OVERFLOW",
    8: "MOE_ERR_TIMEOUT", 9: "MOE_ERR_DTYPE_MISMATCH",
}
STATUS = {v: k for k, v in STATUS_NAMES.items()}


class MoeError(RuntimeError):
    def __init__(self, code, what):
        self.code = code
        super().__init__(f"{what}: {STATUS_NAMES.get(code, code)} ({_lib.moe_strerror(code).decode()})")


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("K", ctypes.c_int64), ("I", ctypes.c_int64),
                ("E_global", ctypes.c_int32), ("E_local", ctypes.c_int32), ("expert_start", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("block_e", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("layout", ctypes.c_int32), ("reserved", ctypes.c_int32), ("max_m", ctypes.c_int64)]


_WS_FIELDS = ["total_bytes", "status", "meta", "counts", "padded", "start", "masked_m", "m_indices", "src2dst",
              "block_info", "chunk_hist", "chunk_rank", "a", "a_sf", "h", "h_sf", "y"]


class MoePlanOutputs(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in ("status", "meta", "counts", "padded", "start", "masked_m",
                                               "m_indices", "src2dst", "block_info")]


class MoeWsLayout(ctypes.Structure):
    _fields_ = [(f, ctypes.c_uint64) for f in _WS_FIELDS] + [
        ("rows", ctypes.c_int64), ("all_tokens", ctypes.c_int64), ("blocks", ctypes.c_int64),
        ("layout", ctypes.c_int32), ("chunks", ctypes.c_int32),
        ("block_vrow", ctypes.c_uint64), ("partial", ctypes.c_uint64),
        ("partial_rows", ctypes.c_int64), ("k_splits1", ctypes.c_int32), ("k_splits2", ctypes.c_int32)]


class MoeAdamwTensor(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in ("param", "grad", "exp_avg", "exp_avg_sq", "avg_scale", "sq_scale",
                                               "master")] + [
        ("n", ctypes.c_int64), ("param_elem", ctypes.c_int32), ("grad_elem", ctypes.c_int32),
        ("state_bits", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class MoeAdamwHyper(ctypes.Structure):
    _fields_ = [(f, ctypes.c_double) for f in ("lr", "beta1", "beta2", "eps", "weight_decay")] + [
        ("step", ctypes.c_int64)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libmoe.so is not built ({LIB_PATH}); run python moe_expert_layer_ep_gb300/build.py")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, VP = ctypes.POINTER, ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    F64 = ctypes.c_double
    sig = {
        "moe_compact_all_tokens": (I64, [I64, I32, I32]),
        "moe_choose_layout": (I32, [I32, I32]),
        "moe_ctx_create": (I32, [P(MoeShape), VP, VP, VP, VP, P(VP)]),
        "moe_ctx_destroy": (None, [VP]),
        "moe_workspace_layout": (I32, [VP, P(MoeWsLayout)]),
        "moe_workspace_size": (I32, [VP, P(ctypes.c_size_t)]),
        "moe_plan_layout": (I32, [VP, VP, VP, VP]),
        "moe_quant_scatter": (I32, [VP, VP, VP, VP]),
        "moe_grouped_gemm_w13_act": (I32, [VP, VP, VP]),
        "moe_grouped_gemm_w2": (I32, [VP, VP, VP]),
        "moe_combine": (I32, [VP, VP, VP, VP, VP]),
        "moe_forward": (I32, [VP, VP, VP, VP, VP, VP, VP]),
        "moe_forward_launches": (I32, [VP]),
        "moe_read_device_status": (I32, [VP, VP, P(I32)]),
        "moe_clear_device_status": (I32, [VP, VP]),
        "moe_selftest_wait_timeout": (I32, [VP, I64, VP]),
        "moe_sf_offset": (I64, [I64, I64, I64, I32]),
        "moe_strerror": (ctypes.c_char_p, [I32]),
        "moe_plan_layout_noalloc": (I32, [P(MoeShape), VP, P(MoePlanOutputs), VP]),
        "moe_requant_weights_ue8m0": (I32, [VP, VP, VP, VP, I64, I64, I64, VP]),
        "moe_route": (I32, [VP, VP, I64, I64, I32, I32, VP, VP, VP, VP, I64, VP]),
        "moe_route_workspace_size": (I64, [I64, I64, I32]),
        "moe_router_prepare": (I32, [VP, VP, I64, I64, VP]),
        "moe_pack_mx_scales": (I32, [VP, I64, VP, I64, I64, I64, VP]),
        "moe_sort_plan_workspace_size": (I64, [I64, I32, I32]),
        "moe_sort_plan": (I32, [VP, I64, I32, I32, I32, I32, VP, VP, VP, VP, I64, VP]),
        "moe_sort_tokens": (I32, [VP, I64, VP, I64, I32, I64, I32, VP, I64, I64, VP]),
        "moe_unsort_tokens": (I32, [VP, I64, I64, VP, VP, I64, I32, I64, I32, VP, I64, VP]),
        "moe_unsort_tokens_backward": (I32, [VP, I64, VP, I64, I64, VP, VP, I64, I32, I64, I32, VP, I64, VP, VP]),
        "moe_expert_gemm": (I32, [VP, I64, I64, VP, VP, VP, I32, I64, I64, VP, I64, VP, VP]),
        "moe_expert_gemm_swiglu": (I32, [VP, I64, I64, VP, VP, VP, I32, I64, I64, VP, I64, VP, I64, VP, VP]),
        "moe_expert_gemm_dgrad": (I32, [VP, I64, I64, VP, VP, VP, I32, I64, I64, VP, I64, VP, VP]),
        "moe_expert_gemm_dgrad_swiglu": (I32, [VP, I64, I64, VP, VP, I64, VP, VP, I32, I64, I64, VP, I64, VP, VP]),
        "moe_expert_gemm_wgrad": (I32, [VP, I64, VP, I64, I64, VP, VP, I32, I64, I64, VP, I32, I32, VP, VP]),
        "moe_expert_gemm_act": (I32, [VP, I64, I64, VP, VP, I32, I32, VP, I64, VP, VP, I32, I64, I64, VP, I64, VP, I64, VP,
                                      VP]),
        "moe_expert_gemm_glu": (I32, [VP, I64, I64, VP, VP, I32, I32, VP, VP, I32, I64, I64, VP, I64, VP, I64, VP, VP]),
        "moe_expert_gemm_dgrad_act": (I32, [VP, I64, I64, VP, VP, I64, I32, VP, I64, VP, VP, I32, I64, I64, VP, I64, VP,
                                            VP]),
        "moe_expert_gemm_dgrad_glu": (I32, [VP, I64, I64, VP, VP, I64, I32, VP, VP, I32, I64, I64, VP, I64, VP, VP]),
        "moe_expert_bias_grad": (I32, [VP, I64, I64, VP, VP, I32, I64, VP, I32, VP, VP]),
        "moe_route_backward_workspace_size": (I64, [I64, I64, I32]),
        "moe_route_backward": (I32, [VP, VP, VP, VP, VP, VP, I64, I64, I32, I32, F64, F64, VP, VP, VP, I32, VP, VP, VP, I64,
                                     VP]),
        "moe_route_backward_kept": (I32, [VP, VP, VP, VP, VP, VP, VP, I64, I64, I32, I32, F64, F64, VP, VP, VP, I32, VP, VP, VP,
                                          I64, VP]),
        "moe_adamw_create": (I32, [P(MoeAdamwTensor), I32, P(VP)]),
        "moe_adamw_destroy": (None, [VP]),
        "moe_adamw_launches": (I32, [VP]),
        "moe_adamw_step": (I32, [VP, P(MoeAdamwHyper), VP, VP]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = _load()
EXPORTED = ("moe_compact_all_tokens", "moe_choose_layout", "moe_ctx_create", "moe_ctx_destroy",
            "moe_workspace_layout", "moe_workspace_size", "moe_plan_layout", "moe_quant_scatter",
            "moe_grouped_gemm_w13_act", "moe_grouped_gemm_w2", "moe_combine", "moe_forward",
            "moe_forward_launches", "moe_read_device_status", "moe_clear_device_status",
            "moe_selftest_wait_timeout", "moe_sf_offset", "moe_strerror", "moe_plan_layout_noalloc",
            "moe_requant_weights_ue8m0", "moe_route", "moe_pack_mx_scales", "moe_route_workspace_size",
            "moe_router_prepare", "moe_sort_plan_workspace_size", "moe_sort_plan", "moe_sort_tokens",
            "moe_unsort_tokens", "moe_unsort_tokens_backward", "moe_expert_gemm", "moe_expert_gemm_swiglu",
            "moe_expert_gemm_dgrad", "moe_expert_gemm_dgrad_swiglu", "moe_expert_gemm_wgrad", "moe_adamw_create", "moe_adamw_destroy",
            "moe_adamw_launches", "moe_adamw_step", "moe_expert_gemm_act", "moe_expert_gemm_glu",
            "moe_expert_gemm_dgrad_act", "moe_expert_gemm_dgrad_glu", "moe_expert_bias_grad",
            "moe_route_backward_workspace_size", "moe_route_backward", "moe_route_backward_kept")


def _check(code, what):
    if code != 0:
        raise MoeError(code, what)


def _ptr(t):
    if t is None or isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:   # the current stream's handle, without a torch.cuda.Stream object
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _empty(shape, dtype, like, stream):
    """An output or scratch tensor of a call that runs on stream (None: the current one).  Memory of the pool of the
    stream that writes it: a free block of the current stream's pool may still be in use by work queued there, which
    another stream does not wait for.  The current stream, where the tensor is then read, has passed its release
    before that pool gives the memory away again."""
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(_stream(stream), device=like.device)
        current = torch.cuda.current_stream(like.device)
        if stream != current:
            with torch.cuda.stream(stream):
                t = torch.empty(shape, dtype=dtype, device=like.device)
            t.record_stream(current)
            return t
    return torch.empty(shape, dtype=dtype, device=like.device)


def _require_cuda(name, t, dtype=None, numel=None):
    if (t.is_cuda and (dtype is None or t.dtype is dtype) and (numel is None or t.numel() == numel)
            and t.is_contiguous()):
        return
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} has {t.numel()} elements, expected {numel}")


def moe_compact_all_tokens(num_assignments, num_experts, block_e=128):
    return int(_lib.moe_compact_all_tokens(num_assignments, num_experts, block_e))


def moe_choose_layout(E_global, E_local):
    return int(_lib.moe_choose_layout(E_global, E_local))


class MoeContext:
    """Owns one moe_ctx (shape + weights); see moe_ctx_create in include/moe.h."""

    def __init__(self, handle, shape, weights):
        self.handle = handle
        self.shape = shape
        self._weights = weights   # keep the weight tensors alive with the context
        lay = MoeWsLayout()
        _check(_lib.moe_workspace_layout(handle, ctypes.byref(lay)), "moe_workspace_layout")
        self.ws_layout = lay

    @property
    def fp8(self):
        """FP8 operands (1x128 / 128x128 or MXFP8 1x32 scales)."""
        return self.shape.dtype in (MOE_DTYPE_FP8, MOE_DTYPE_MXFP8, MOE_DTYPE_MXFP4)

    @property
    def mx(self):
        """1x32 scales on activations and h (MXFP8 and MXFP4)."""
        return self.shape.dtype in (MOE_DTYPE_MXFP8, MOE_DTYPE_MXFP4)

    @property
    def masked(self):
        return self.ws_layout.layout == MOE_LAYOUT_MASKED

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h and _lib is not None:
            _lib.moe_ctx_destroy(h)


def make_shape(T, K, I, E_global, E_local, topk, dtype, layout=MOE_LAYOUT_AUTO, expert_start=0, max_m=0,
               block_e=128):
    if isinstance(dtype, str):
        dtype = {"fp8": MOE_DTYPE_FP8, "bf16": MOE_DTYPE_BF16, "mxfp8": MOE_DTYPE_MXFP8, "mxfp4": MOE_DTYPE_MXFP4}[dtype]
    if isinstance(layout, str):
        layout = {"auto": MOE_LAYOUT_AUTO, "compact": MOE_LAYOUT_COMPACT, "masked": MOE_LAYOUT_MASKED}[layout]
    return MoeShape(T=T, K=K, I=I, E_global=E_global, E_local=E_local, expert_start=expert_start, topk=topk,
                    block_e=block_e, dtype=dtype, layout=layout, reserved=0, max_m=max_m)


def moe_ctx_create(shape, w13, w13_sf, w2, w2_sf):
    """shape: MoeShape; weights as in include/moe.h (CUDA tensors)."""
    fp4 = shape.dtype == MOE_DTYPE_MXFP4
    mx = shape.dtype == MOE_DTYPE_MXFP8 or fp4
    fp8 = shape.dtype == MOE_DTYPE_FP8 or mx
    E, K, I = shape.E_local, shape.K, shape.I
    wdt = torch.uint8 if fp8 else torch.bfloat16
    wd = 2 if fp4 else 1      # two FP4 codes per byte
    _require_cuda("w13", w13, wdt, E * 2 * I * K // wd)
    _require_cuda("w2", w2, wdt, E * K * I // wd)
    if w13_sf is not None:
        _require_cuda("w13_sf", w13_sf, torch.uint8, E * 2 * I * K // 32 if mx else E * (2 * I // 128) * (K // 128))
    if w2_sf is not None:
        _require_cuda("w2_sf", w2_sf, torch.uint8, E * K * I // 32 if mx else E * (K // 128) * (I // 128))
    h = ctypes.c_void_p()
    _check(_lib.moe_ctx_create(ctypes.byref(shape), _ptr(w13), _ptr(w13_sf), _ptr(w2), _ptr(w2_sf),
                               ctypes.byref(h)), "moe_ctx_create")
    return MoeContext(h, shape, (w13, w13_sf, w2, w2_sf))


def moe_workspace_size(ctx):
    return int(ctx.ws_layout.total_bytes)


def alloc_workspace(ctx, device=None):
    """Device workspace of moe_workspace_size bytes (torch allocation)."""
    return torch.empty(max(1, moe_workspace_size(ctx)), dtype=torch.uint8, device=device or "cuda")


def moe_plan_layout(ctx, topk_ids, ws, stream=None):
    _require_cuda("topk_ids", topk_ids, torch.int32, ctx.shape.T * ctx.shape.topk)
    _check(_lib.moe_plan_layout(ctx.handle, _ptr(topk_ids), _ptr(ws), _stream(stream)), "moe_plan_layout")


def moe_quant_scatter(ctx, x, ws, stream=None):
    _require_cuda("x", x, torch.bfloat16, ctx.shape.T * ctx.shape.K)
    _check(_lib.moe_quant_scatter(ctx.handle, _ptr(x), _ptr(ws), _stream(stream)), "moe_quant_scatter")


def moe_grouped_gemm_w13_act(ctx, ws, stream=None):
    _check(_lib.moe_grouped_gemm_w13_act(ctx.handle, _ptr(ws), _stream(stream)), "moe_grouped_gemm_w13_act")


def moe_grouped_gemm_w2(ctx, ws, stream=None):
    _check(_lib.moe_grouped_gemm_w2(ctx.handle, _ptr(ws), _stream(stream)), "moe_grouped_gemm_w2")


def moe_combine(ctx, topk_weights, ws, out, stream=None):
    _require_cuda("topk_weights", topk_weights, torch.float32, ctx.shape.T * ctx.shape.topk)
    _require_cuda("out", out, torch.bfloat16, ctx.shape.T * ctx.shape.K)
    _check(_lib.moe_combine(ctx.handle, _ptr(topk_weights), _ptr(ws), _ptr(out), _stream(stream)), "moe_combine")


def moe_forward(ctx, x, topk_ids, topk_weights, ws, out, stream=None):
    s = ctx.shape
    _require_cuda("x", x, torch.bfloat16, s.T * s.K)
    _require_cuda("topk_ids", topk_ids, torch.int32, s.T * s.topk)
    _require_cuda("topk_weights", topk_weights, torch.float32, s.T * s.topk)
    _require_cuda("out", out, torch.bfloat16, s.T * s.K)
    _check(_lib.moe_forward(ctx.handle, _ptr(x), _ptr(topk_ids), _ptr(topk_weights), _ptr(ws), _ptr(out),
                            _stream(stream)), "moe_forward")


def moe_forward_launches(ctx):
    return int(_lib.moe_forward_launches(ctx.handle))


def moe_read_device_status(ws, stream=None):
    v = ctypes.c_int32()
    _check(_lib.moe_read_device_status(_ptr(ws), _stream(stream), ctypes.byref(v)), "moe_read_device_status")
    return int(v.value)


def moe_clear_device_status(ws, stream=None):
    _check(_lib.moe_clear_device_status(_ptr(ws), _stream(stream)), "moe_clear_device_status")


def moe_selftest_wait_timeout(ws, timeout_ns, stream=None):
    _check(_lib.moe_selftest_wait_timeout(_ptr(ws), int(timeout_ns), _stream(stream)), "moe_selftest_wait_timeout")


def moe_sf_offset(block, group, n_groups, row):
    return int(_lib.moe_sf_offset(block, group, n_groups, row))


def moe_plan_layout_noalloc(shape, topk_ids, outputs, stream=None):
    """outputs: dict of int32 CUDA tensors keyed like MoePlanOutputs's fields
    (missing keys are passed as NULL)."""
    if topk_ids is not None:
        _require_cuda("topk_ids", topk_ids, torch.int32, shape.T * shape.topk)
    o = MoePlanOutputs(**{k: _ptr(v) for k, v in outputs.items()})
    _check(_lib.moe_plan_layout_noalloc(ctypes.byref(shape), _ptr(topk_ids), ctypes.byref(o), _stream(stream)),
           "moe_plan_layout_noalloc")


def moe_requant_weights_ue8m0(w_in, scale_in, w_out=None, scale_out=None, stream=None):
    """w_in uint8 [E, N, C] e4m3; scale_in float32 [E, N/128, C/128].  Returns
    (w_out, scale_out) with UE8M0 block scales (see include/moe.h)."""
    E, N, C = w_in.shape
    _require_cuda("w_in", w_in, torch.uint8)
    _require_cuda("scale_in", scale_in, torch.float32, E * (N // 128) * (C // 128))
    if w_out is None:
        w_out = _empty(tuple(w_in.shape), w_in.dtype, w_in, stream)
    if scale_out is None:
        scale_out = _empty((E, N // 128, C // 128), torch.uint8, w_in, stream)
    _require_cuda("w_out", w_out, torch.uint8, w_in.numel())
    _require_cuda("scale_out", scale_out, torch.uint8, E * (N // 128) * (C // 128))
    _check(_lib.moe_requant_weights_ue8m0(_ptr(w_in), _ptr(scale_in), _ptr(w_out), _ptr(scale_out), E, N, C,
                                          _stream(stream)), "moe_requant_weights_ue8m0")
    return w_out, scale_out


def moe_router_prepare(w_router, out=None, stream=None):
    """fp32 router weights [E, K] -> bf16 planes [3, E, K] (hi + mid + lo == w);
    see include/moe.h."""
    E, K = w_router.shape
    _require_cuda("w_router", w_router, torch.float32)
    if out is None:
        out = _empty((3, E, K), torch.bfloat16, w_router, stream)
    _require_cuda("out", out, torch.bfloat16, 3 * E * K)
    _check(_lib.moe_router_prepare(_ptr(w_router), _ptr(out), E, K, _stream(stream)), "moe_router_prepare")
    return out


def moe_route_workspace_size(T, K, E):
    return int(_lib.moe_route_workspace_size(T, K, E))


def moe_route(x, w_planes, topk, logits=None, topk_ids=None, topk_weights=None, ws=None, stream=None):
    """x bf16 [T, K], w_planes bf16 [3, E, K] (moe_router_prepare) ->
    (topk_ids int32 [T, k], topk_weights fp32 [T, k], logits fp32 [T, E]);
    see include/moe.h.  ws: uint8 device scratch (allocated here if None)."""
    T, K = x.shape
    E = w_planes.shape[1]
    _require_cuda("x", x, torch.bfloat16)
    _require_cuda("w_planes", w_planes, torch.bfloat16, 3 * E * K)
    if logits is None:
        logits = _empty((T, E), torch.float32, x, stream)
    if topk_ids is None:
        topk_ids = _empty((T, topk), torch.int32, x, stream)
    if topk_weights is None:
        topk_weights = _empty((T, topk), torch.float32, x, stream)
    if ws is None:
        ws = _empty((max(16, moe_route_workspace_size(T, K, E)),), torch.uint8, x, stream)
    _require_cuda("logits", logits, torch.float32, T * E)
    _require_cuda("topk_ids", topk_ids, torch.int32, T * topk)
    _require_cuda("topk_weights", topk_weights, torch.float32, T * topk)
    _require_cuda("ws", ws, torch.uint8)
    _check(_lib.moe_route(_ptr(x), _ptr(w_planes), T, K, E, topk, _ptr(logits), _ptr(topk_ids), _ptr(topk_weights),
                          _ptr(ws), ws.numel(), _stream(stream)), "moe_route")
    return topk_ids, topk_weights, logits


def moe_pack_mx_scales(sf, out=None, stream=None, C=None):
    """MXFP8 weight scales uint8 [E, N, ld] (natural layout; ld = C/32, or
    more when the scale rows are padded, in which case pass C) -> the packed
    order moe_ctx_create takes for MOE_DTYPE_MXFP8 (see include/moe.h)."""
    E, N, ld = sf.shape
    C = ld * 32 if C is None else C
    _require_cuda("sf", sf, torch.uint8)
    if out is None:
        out = _empty((E, N, C // 32), torch.uint8, sf, stream)
    _require_cuda("out", out, torch.uint8, E * N * (C // 32))
    _check(_lib.moe_pack_mx_scales(_ptr(sf), ld, _ptr(out), E, N, C, _stream(stream)), "moe_pack_mx_scales")
    return out


# ------------------------------------------------------------------ training
_ELEM = {torch.bfloat16: MOE_ELEM_BF16, torch.float32: MOE_ELEM_F32}


def _rows(name, t, dtype=None, cols=None):
    """A matrix of rows that are contiguous in themselves; returns its row stride."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix")
    n, c = t.shape
    if cols is not None and c != cols:
        raise ValueError(f"{name} has {c} columns, expected {cols}")
    if t.is_contiguous():
        return c
    ld, one = t.stride()
    if one != 1 and c > 1:
        raise ValueError(f"{name} must have contiguous rows")
    if n > 1 and ld < c:
        raise ValueError(f"{name}'s rows overlap")
    return ld if ld > c else c


def _elem(name, t):
    try:
        return _ELEM[t.dtype]
    except KeyError:
        raise ValueError(f"{name} must be bfloat16 or float32, got {t.dtype}") from None


def moe_sort_plan_workspace_size(T, topk, E_local):
    return int(_lib.moe_sort_plan_workspace_size(T, topk, E_local))


def moe_sort_plan(topk_ids, E_global, E_local=None, expert_start=0, src2dst=None, start=None, counts=None, ws=None,
                  stream=None):
    """topk_ids int32 [T, k] -> (src2dst int32 [T, k], start int32 [E_local], counts int32 [E_local]), the compact
    layout of the routing; see include/moe.h.  ws: uint8 device scratch (allocated here if None) that begins with the
    status word."""
    T, topk = topk_ids.shape
    E_local = E_global if E_local is None else E_local
    _require_cuda("topk_ids", topk_ids, torch.int32)
    if src2dst is None:
        src2dst = _empty((T, topk), torch.int32, topk_ids, stream)
    else:
        _require_cuda("src2dst", src2dst, torch.int32, T * topk)
    if start is None:
        start = _empty((E_local,), torch.int32, topk_ids, stream)
    else:
        _require_cuda("start", start, torch.int32, E_local)
    if counts is None:
        counts = _empty((E_local,), torch.int32, topk_ids, stream)
    else:
        _require_cuda("counts", counts, torch.int32, E_local)
    if ws is None:
        ws = _empty((max(16, moe_sort_plan_workspace_size(T, topk, E_local)),), torch.uint8, topk_ids, stream)
    else:
        _require_cuda("ws", ws, torch.uint8)
    _check(_lib.moe_sort_plan(_ptr(topk_ids), T, topk, E_global, E_local, expert_start, _ptr(src2dst), _ptr(start),
                              _ptr(counts), _ptr(ws), ws.numel(), _stream(stream)), "moe_sort_plan")
    return src2dst, start, counts


def moe_sort_tokens(x, src2dst, rows=None, out=None, stream=None):
    """x [T, K] bf16 or fp32 -> the rows in sorted order [rows, K]; rows that carry no token are left as they are.
    rows is needed when out is not given (moe_compact_all_tokens)."""
    T, topk = src2dst.shape
    x_ld = _rows("x", x)
    K = x.shape[1]
    _require_cuda("src2dst", src2dst, torch.int32)
    if x.shape[0] != T:
        raise ValueError(f"x has {x.shape[0]} rows, src2dst {T}")
    if out is None:
        if rows is None:
            raise ValueError("rows or out must be given")
        out, out_ld = _empty((rows, K), x.dtype, x, stream), K
    else:
        out_ld = _rows("out", out, x.dtype, K)
    _check(_lib.moe_sort_tokens(_ptr(x), x_ld, _ptr(src2dst), T, topk, K, _elem("x", x), _ptr(out), out_ld,
                                out.shape[0], _stream(stream)), "moe_sort_tokens")
    return out


def moe_unsort_tokens(y, src2dst, topk_weights=None, out=None, stream=None):
    """Sorted rows y [rows, K] -> out [T, K], the (weighted) sum of each token's rows; without weights also the
    gradient of moe_sort_tokens."""
    T, topk = src2dst.shape
    y_ld = _rows("y", y)
    K = y.shape[1]
    _require_cuda("src2dst", src2dst, torch.int32)
    if topk_weights is not None:
        _require_cuda("topk_weights", topk_weights, torch.float32, T * topk)
    if out is None:
        out, out_ld = _empty((T, K), y.dtype, y, stream), K
    else:
        out_ld = _rows("out", out, y.dtype, K)
        if out.shape[0] != T:
            raise ValueError(f"out has {out.shape[0]} rows, src2dst {T}")
    _check(_lib.moe_unsort_tokens(_ptr(y), y_ld, y.shape[0], _ptr(src2dst), _ptr(topk_weights), T, topk, K,
                                  _elem("y", y), _ptr(out), out_ld, _stream(stream)), "moe_unsort_tokens")
    return out


def moe_unsort_tokens_backward(dout, y, src2dst, topk_weights, dy=None, dw=None, stream=None, rows=None):
    """Gradient of moe_unsort_tokens with weights: (dy [rows, K], dw fp32 [T, k]).  dy's rows that carry no token are
    left as they are.  y=None: the rows' gradient alone, for weights that are not learned; dw is None then, and rows is
    needed when dy is not given."""
    T, topk = src2dst.shape
    dout_ld = _rows("dout", dout)
    K = dout.shape[1]
    _require_cuda("src2dst", src2dst, torch.int32)
    _require_cuda("topk_weights", topk_weights, torch.float32, T * topk)
    if dout.shape[0] != T:
        raise ValueError(f"dout has {dout.shape[0]} rows, src2dst {T}")
    y_ld = 0
    if y is None:
        if dw is not None:
            raise ValueError("the gradient of the weights needs y")
        if dy is None and rows is None:
            raise ValueError("rows or dy must be given")
        if rows is None:
            _rows("dy", dy, dout.dtype, K)
            rows = dy.shape[0]
    else:
        y_ld = _rows("y", y, dout.dtype, K)
        if rows not in (None, y.shape[0]):
            raise ValueError(f"y has {y.shape[0]} rows, expected {rows}")
        rows = y.shape[0]
        if dw is None:
            dw = _empty((T, topk), torch.float32, y, stream)
        _require_cuda("dw", dw, torch.float32, T * topk)
    if dy is None:
        dy = _empty((rows, K), dout.dtype, dout, stream)
    dy_ld = _rows("dy", dy, dout.dtype, K)
    if dy.shape[0] != rows:
        raise ValueError(f"dy has {dy.shape[0]} rows, expected {rows}")
    _check(_lib.moe_unsort_tokens_backward(_ptr(dout), dout_ld, _ptr(y), y_ld, rows, _ptr(src2dst),
                                           _ptr(topk_weights), T, topk, K, _elem("dout", dout), _ptr(dy), dy_ld,
                                           _ptr(dw), _stream(stream)), "moe_unsort_tokens_backward")
    return dy, dw


def _expert_args(start, counts, status, E):
    if start is not None or counts is not None:
        if start is None or counts is None:
            raise ValueError("start and counts must both be given, or neither")
        _require_cuda("start", start, torch.int32, E)
        _require_cuda("counts", counts, torch.int32, E)
    elif E != 1:
        raise ValueError("start and counts may be left out for one expert only")
    if not status.is_cuda or status.numel() * status.element_size() < 4:
        raise ValueError("status must be a CUDA tensor of at least 4 bytes")


def _expert_weights(w, start, counts, status):
    """Checks of the arguments that the products with weights share: (E, N, C).  Without start and counts, one
    expert that has all rows, the weights may be a matrix."""
    dense = w.dim() == 2 and start is None and counts is None
    if w.dim() != 3 and not dense:
        raise ValueError("the weights must be [E, N, C]")
    E, N, C = (1, *w.shape) if dense else w.shape
    _require_cuda("w", w, torch.bfloat16)
    _expert_args(start, counts, status, E)
    return E, N, C


def _sorted_out(name, t, rows, cols, like, stream):
    """An output of sorted rows, allocated when not given."""
    if t is None:
        return _empty((rows, cols), torch.bfloat16, like, stream), cols
    ld = _rows(name, t, torch.bfloat16, cols)
    if t.shape[0] != rows:
        raise ValueError(f"{name} has {t.shape[0]} rows, expected {rows}")
    return t, ld


def moe_expert_gemm(x, w, start, counts, status, y=None, stream=None):
    """Sorted rows x [rows, C], w [E, N, C] -> y [rows, N] = x W_e^T for each expert's rows; see include/moe.h.
    status: CUDA tensor whose first int32 is the status word (a moe_sort_plan workspace, or 4 zeroed int32).
    start = counts = None, here and in the other products: one expert, w [N, C] or [1, N, C], that has all rows."""
    E, N, C = _expert_weights(w, start, counts, status)
    x_ld = _rows("x", x, torch.bfloat16, C)
    y, y_ld = _sorted_out("y", y, x.shape[0], N, x, stream)
    _check(_lib.moe_expert_gemm(_ptr(x), x_ld, x.shape[0], _ptr(w), _ptr(start), _ptr(counts), E, N, C, _ptr(y), y_ld,
                                _ptr(status), _stream(stream)), "moe_expert_gemm")
    return y


def moe_expert_gemm_swiglu(x, w13, start, counts, status, h=None, gu=None, keep_gu=True, stream=None):
    """Sorted rows x [rows, C], w13 [E, 2I, C] -> (h [rows, I], gu [rows, 2I]): the first product and its gated
    activation.  keep_gu=False: gu (which only the gradient needs) is not stored, and None is returned for it."""
    E, N, C = _expert_weights(w13, start, counts, status)
    if N % 2:
        raise ValueError("w13 must have 2I rows per expert")
    I = N // 2
    x_ld = _rows("x", x, torch.bfloat16, C)
    h, h_ld = _sorted_out("h", h, x.shape[0], I, x, stream)
    gu_ld = 0
    if keep_gu or gu is not None:
        gu, gu_ld = _sorted_out("gu", gu, x.shape[0], N, x, stream)
    _check(_lib.moe_expert_gemm_swiglu(_ptr(x), x_ld, x.shape[0], _ptr(w13), _ptr(start), _ptr(counts), E, I, C,
                                       _ptr(gu), gu_ld, _ptr(h), h_ld, _ptr(status), _stream(stream)),
           "moe_expert_gemm_swiglu")
    return h, gu


def moe_expert_gemm_dgrad(dy, w, start, counts, status, dx=None, stream=None):
    """Gradient of moe_expert_gemm's rows: dy [rows, N], w [E, N, C] -> dx [rows, C]."""
    E, N, C = _expert_weights(w, start, counts, status)
    dy_ld = _rows("dy", dy, torch.bfloat16, N)
    dx, dx_ld = _sorted_out("dx", dx, dy.shape[0], C, dy, stream)
    _check(_lib.moe_expert_gemm_dgrad(_ptr(dy), dy_ld, dy.shape[0], _ptr(w), _ptr(start), _ptr(counts), E, N, C,
                                      _ptr(dx), dx_ld, _ptr(status), _stream(stream)), "moe_expert_gemm_dgrad")
    return dx


def moe_expert_gemm_dgrad_swiglu(dy, w2, gu, start, counts, status, dgu=None, stream=None):
    """Gradient through the second product and the activation: dy [rows, N], w2 [E, N, I], gu [rows, 2I] as
    moe_expert_gemm_swiglu stored it -> dgu [rows, 2I]."""
    E, N, I = _expert_weights(w2, start, counts, status)
    dy_ld = _rows("dy", dy, torch.bfloat16, N)
    gu_ld = _rows("gu", gu, torch.bfloat16, 2 * I)
    if gu.shape[0] != dy.shape[0]:
        raise ValueError(f"gu has {gu.shape[0]} rows, dy {dy.shape[0]}")
    dgu, dgu_ld = _sorted_out("dgu", dgu, dy.shape[0], 2 * I, dy, stream)
    _check(_lib.moe_expert_gemm_dgrad_swiglu(_ptr(dy), dy_ld, dy.shape[0], _ptr(w2), _ptr(gu), gu_ld, _ptr(start),
                                             _ptr(counts), E, N, I, _ptr(dgu), dgu_ld, _ptr(status), _stream(stream)),
           "moe_expert_gemm_dgrad_swiglu")
    return dgu


def moe_expert_gemm_wgrad(dy, x, start, counts, status, dw=None, accumulate=False, stream=None):
    """Gradient of the weights: dy [rows, N], x [rows, C] -> dw [E, N, C], zeros for experts without rows.  dw is
    bfloat16 (also when it is allocated here) or float32; accumulate adds the gradient to a float32 dw."""
    dy_ld, x_ld = _rows("dy", dy, torch.bfloat16), _rows("x", x, torch.bfloat16)
    E, N, C = 1 if counts is None else counts.numel(), dy.shape[1], x.shape[1]
    if x.shape[0] != dy.shape[0]:
        raise ValueError(f"x has {x.shape[0]} rows, dy {dy.shape[0]}")
    if dw is None:
        if accumulate:
            raise ValueError("accumulate needs a dw to add to")
        dw = _empty((E, N, C), torch.bfloat16, dy, stream)
    if tuple(dw.shape) != (E, N, C):
        raise ValueError(f"dw is {tuple(dw.shape)}, expected {(E, N, C)}")
    _require_cuda("dw", dw)
    _expert_args(start, counts, status, E)
    _check(_lib.moe_expert_gemm_wgrad(_ptr(dy), dy_ld, _ptr(x), x_ld, x.shape[0], _ptr(start), _ptr(counts), E, N, C,
                                      _ptr(dw), _elem("dw", dw), accumulate, _ptr(status), _stream(stream)),
           "moe_expert_gemm_wgrad")
    return dw


def _on_current_device(*tensors):
    """The kernels are launched on the current device: tensors (None is left out) must be there."""
    here = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{here}")


def _act(name):
    try:
        return MOE_ACTS[name]
    except (KeyError, TypeError):
        raise ValueError(f"act must be one of {', '.join(MOE_ACTS)}, got {name!r}") from None


def _bias(bias, numel):
    """An optional bias: its moe_elem_t."""
    if bias is None:
        return MOE_ELEM_BF16
    _require_cuda("bias", bias, None, numel)
    return _elem("bias", bias)


def _optional_rows(name, t, rows, cols):
    """The row stride of a matrix of sorted rows that may be missing."""
    if t is None:
        return 0
    ld = _rows(name, t, torch.bfloat16, cols)
    if t.shape[0] != rows:
        raise ValueError(f"{name} has {t.shape[0]} rows, expected {rows}")
    return ld


def moe_expert_gemm_act(x, w, start, counts, status, bias=None, act="none", residual=None, y=None, z=None, keep_z=False,
                        stream=None):
    """Sorted rows x [rows, C], w [E, N, C] -> (y, z) [rows, N]: z = x W_e^T + bias_e, y = act(z) + residual.  bias
    [E, N] bf16 or fp32; act: a name of MOE_ACTS; residual [rows, N] bf16, may be y.  z, which only the gradient needs,
    is stored where it is given or keep_z is set, else None."""
    E, N, C = _expert_weights(w, start, counts, status)
    x_ld = _rows("x", x, torch.bfloat16, C)
    rows = x.shape[0]
    bias_elem = _bias(bias, E * N)
    res_ld = _optional_rows("residual", residual, rows, N)
    _on_current_device(x, w, start, counts, status, bias, residual, y, z)
    y, y_ld = _sorted_out("y", y, rows, N, x, stream)
    z_ld = 0
    if keep_z or z is not None:
        z, z_ld = _sorted_out("z", z, rows, N, x, stream)
    _check(_lib.moe_expert_gemm_act(_ptr(x), x_ld, rows, _ptr(w), _ptr(bias), bias_elem, _act(act), _ptr(residual), res_ld,
                                    _ptr(start), _ptr(counts), E, N, C, _ptr(z), z_ld, _ptr(y), y_ld, _ptr(status),
                                    _stream(stream)), "moe_expert_gemm_act")
    return y, z


def moe_expert_gemm_glu(x, w13, start, counts, status, bias=None, act="silu", h=None, gu=None, keep_gu=True, stream=None):
    """moe_expert_gemm_swiglu with a bias [E, 2I] (bf16 or fp32) and any activation of the gate: (h, gu)."""
    E, N, C = _expert_weights(w13, start, counts, status)
    if N % 2:
        raise ValueError("w13 must have 2I rows per expert")
    I = N // 2
    x_ld = _rows("x", x, torch.bfloat16, C)
    bias_elem = _bias(bias, E * N)
    _on_current_device(x, w13, start, counts, status, bias, h, gu)
    h, h_ld = _sorted_out("h", h, x.shape[0], I, x, stream)
    gu_ld = 0
    if keep_gu or gu is not None:
        gu, gu_ld = _sorted_out("gu", gu, x.shape[0], N, x, stream)
    _check(_lib.moe_expert_gemm_glu(_ptr(x), x_ld, x.shape[0], _ptr(w13), _ptr(bias), bias_elem, _act(act), _ptr(start),
                                    _ptr(counts), E, I, C, _ptr(gu), gu_ld, _ptr(h), h_ld, _ptr(status), _stream(stream)),
           "moe_expert_gemm_glu")
    return h, gu


def moe_expert_gemm_dgrad_act(dy, w, start, counts, status, z=None, act="none", residual=None, dx=None, stream=None):
    """Gradient of a product's rows, through the activation before it: dy [rows, N], w [E, N, C], z [rows, C] as
    moe_expert_gemm_act kept it -> dx [rows, C] = act'(z) (dy W_e) + residual.  residual [rows, C] bf16, may be dx."""
    E, N, C = _expert_weights(w, start, counts, status)
    dy_ld = _rows("dy", dy, torch.bfloat16, N)
    rows, code = dy.shape[0], _act(act)
    if code and z is None:
        raise ValueError(f"the gradient of {act} needs z")
    z_ld = _optional_rows("z", z, rows, C)
    res_ld = _optional_rows("residual", residual, rows, C)
    _on_current_device(dy, w, start, counts, status, z, residual, dx)
    dx, dx_ld = _sorted_out("dx", dx, rows, C, dy, stream)
    _check(_lib.moe_expert_gemm_dgrad_act(_ptr(dy), dy_ld, rows, _ptr(w), _ptr(z), z_ld, code, _ptr(residual), res_ld,
                                          _ptr(start), _ptr(counts), E, N, C, _ptr(dx), dx_ld, _ptr(status),
                                          _stream(stream)), "moe_expert_gemm_dgrad_act")
    return dx


def moe_expert_gemm_dgrad_glu(dy, w2, gu, start, counts, status, act="silu", dgu=None, stream=None):
    """moe_expert_gemm_dgrad_swiglu for any activation of the gate."""
    E, N, I = _expert_weights(w2, start, counts, status)
    dy_ld = _rows("dy", dy, torch.bfloat16, N)
    gu_ld = _optional_rows("gu", gu, dy.shape[0], 2 * I)
    _on_current_device(dy, w2, gu, start, counts, status, dgu)
    dgu, dgu_ld = _sorted_out("dgu", dgu, dy.shape[0], 2 * I, dy, stream)
    _check(_lib.moe_expert_gemm_dgrad_glu(_ptr(dy), dy_ld, dy.shape[0], _ptr(w2), _ptr(gu), gu_ld, _act(act), _ptr(start),
                                          _ptr(counts), E, N, I, _ptr(dgu), dgu_ld, _ptr(status), _stream(stream)),
           "moe_expert_gemm_dgrad_glu")
    return dgu


def moe_expert_bias_grad(dy, start, counts, status, db=None, accumulate=False, stream=None):
    """Gradient of a product's bias: dy [rows, N] -> db fp32 [E, N], the sum of each expert's rows (accumulate: added to
    db)."""
    dy_ld = _rows("dy", dy, torch.bfloat16)
    E, N = 1 if counts is None else counts.numel(), dy.shape[1]
    _expert_args(start, counts, status, E)
    _on_current_device(dy, start, counts, status, db)
    if db is None:
        if accumulate:
            raise ValueError("accumulate needs a db to add to")
        db = _empty((E, N), torch.float32, dy, stream)
    _require_cuda("db", db, torch.float32, E * N)
    _check(_lib.moe_expert_bias_grad(_ptr(dy), dy_ld, dy.shape[0], _ptr(start), _ptr(counts), E, N, _ptr(db), accumulate,
                                     _ptr(status), _stream(stream)), "moe_expert_bias_grad")
    return db


def moe_route_backward_workspace_size(T, K, E):
    return int(_lib.moe_route_backward_workspace_size(T, K, E))


def moe_route_backward(x, w_planes, logits, topk_ids, topk_weights, dweights, balance=0.0, zloss=0.0, residual=None,
                       dx=None, dw=None, accumulate=False, dlogits=None, losses=None, ws=None, stream=None, kept=None):
    """Gradient of moe_route and of its losses: x bf16 [T, K], w_planes bf16 [3, E, K], logits fp32 [T, E], topk_ids
    int32, topk_weights and dweights fp32 [T, k] -> (dx bf16 [T, K], dw fp32 [E, K], losses fp32 [2]: the load balance
    and the mean squared logsumexp, of which balance and zloss are the factors in the total loss); see include/moe.h.
    residual: bf16 [T, K] added to dx (may be dx); accumulate: dw is added to; dlogits: fp32 [T, E], written if given.
    ws: uint8 device scratch (allocated here if None) that begins with the status word.  kept: bool or uint8 [T, k], 0 for
    an assignment that was dropped although the weights are still those of all k; its id stays.  (An id of -1 instead
    means that the weights are the softmax over the others.)"""
    if x.dim() != 2 or w_planes.dim() != 3 or topk_ids.dim() != 2:
        raise ValueError("x and topk_ids must be matrices, w_planes [3, E, K]")
    (T, K), E, topk = x.shape, w_planes.shape[1], topk_ids.shape[1]
    _require_cuda("x", x, torch.bfloat16)
    _require_cuda("w_planes", w_planes, torch.bfloat16, 3 * E * K)
    _require_cuda("logits", logits, torch.float32, T * E)
    _require_cuda("topk_ids", topk_ids, torch.int32, T * topk)
    _require_cuda("topk_weights", topk_weights, torch.float32, T * topk)
    _require_cuda("dweights", dweights, torch.float32, T * topk)
    if residual is not None:
        _require_cuda("residual", residual, torch.bfloat16, T * K)
    if kept is not None:
        _require_cuda("kept", kept, None, T * topk)
        if kept.dtype not in (torch.bool, torch.uint8):
            raise ValueError(f"kept must be bool or uint8, got {kept.dtype}")
    if accumulate and dw is None:
        raise ValueError("accumulate needs a dw to add to")
    _on_current_device(x, w_planes, logits, topk_ids, topk_weights, dweights, residual, dx, dw, dlogits, losses, ws,
                       kept)
    if dx is None:
        dx = _empty((T, K), torch.bfloat16, x, stream)
    if dw is None:
        dw = _empty((E, K), torch.float32, x, stream)
    if losses is None:
        losses = _empty((2,), torch.float32, x, stream)
    if ws is None:
        ws = _empty((moe_route_backward_workspace_size(T, K, E),), torch.uint8, x, stream)
    _require_cuda("dx", dx, torch.bfloat16, T * K)
    _require_cuda("dw", dw, torch.float32, E * K)
    if dlogits is not None:
        _require_cuda("dlogits", dlogits, torch.float32, T * E)
    _require_cuda("losses", losses, torch.float32, 2)
    _require_cuda("ws", ws, torch.uint8)
    _check(_lib.moe_route_backward_kept(_ptr(x), _ptr(w_planes), _ptr(logits), _ptr(topk_ids), _ptr(topk_weights),
                                        _ptr(dweights), _ptr(kept), T, K, E, topk, balance, zloss, _ptr(residual), _ptr(dx),
                                        _ptr(dw), accumulate, _ptr(dlogits), _ptr(losses), _ptr(ws), ws.numel(),
                                        _stream(stream)), "moe_route_backward")
    return dx, dw, losses


class MoeAdamw:
    """Owns one moe_adamw (the tensors of an optimizer step); see include/moe.h."""

    def __init__(self, handle, tensors):
        self.handle = handle
        self._tensors = tensors   # keep them alive with the handle

    def __del__(self):
        h, self.handle = getattr(self, "handle", None), None
        if h and _lib is not None:
            _lib.moe_adamw_destroy(h)


def moe_adamw_create(params, grads, exp_avgs, exp_avg_sqs, masters=None, avg_scales=None, sq_scales=None):
    """Lists of CUDA tensors, one entry per parameter.  States float32, or int8 (exp_avgs) and uint8 (exp_avg_sqs)
    with float32 scales of ceil(n / 256) elements.  masters: float32 copies of bf16 params (entries may be None)."""
    n = len(params)
    none = [None] * n
    lists = [params, grads, exp_avgs, exp_avg_sqs, avg_scales or none, sq_scales or none, masters or none]
    if any(len(x) != n for x in lists):
        raise ValueError("moe_adamw_create: lists of different lengths")
    table = (MoeAdamwTensor * max(1, n))()
    for i, (p, g, m, v, ms, vs, w) in enumerate(zip(*lists)):
        k, blocks = p.numel(), -(-p.numel() // 256)
        bits = 32 if m.dtype == torch.float32 else 8
        _require_cuda(f"params[{i}]", p)
        _require_cuda(f"grads[{i}]", g, None, k)
        _require_cuda(f"exp_avgs[{i}]", m, torch.float32 if bits == 32 else torch.int8, k)
        _require_cuda(f"exp_avg_sqs[{i}]", v, torch.float32 if bits == 32 else torch.uint8, k)
        for name, t, numel in (("avg_scales", ms, blocks), ("sq_scales", vs, blocks), ("masters", w, k)):
            if t is not None:
                _require_cuda(f"{name}[{i}]", t, torch.float32, numel)
        table[i] = MoeAdamwTensor(_ptr(p), _ptr(g), _ptr(m), _ptr(v), _ptr(ms), _ptr(vs), _ptr(w), k,
                                  _elem(f"params[{i}]", p), _elem(f"grads[{i}]", g), bits, 0)
    h = ctypes.c_void_p()
    _check(_lib.moe_adamw_create(table, n, ctypes.byref(h)), "moe_adamw_create")
    return MoeAdamw(h, lists)


def moe_adamw_launches(opt):
    return int(_lib.moe_adamw_launches(opt.handle))


def moe_adamw_step(opt, step, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, grad_scale=None, stream=None):
    """One step (step counts from 1).  grad_scale: float32 CUDA scalar that multiplies every gradient."""
    if grad_scale is not None:
        _require_cuda("grad_scale", grad_scale, torch.float32, 1)
    h = MoeAdamwHyper(lr, beta1, beta2, eps, weight_decay, step)
    _check(_lib.moe_adamw_step(opt.handle, ctypes.byref(h), _ptr(grad_scale), _stream(stream)), "moe_adamw_step")


def ws_view(ctx, ws, name):
    """A typed torch view of one workspace intermediate (test and debug use)."""
    L, s = ctx.ws_layout, ctx.shape
    off = getattr(L, name)
    i32 = {"status": 4, "meta": 8, "counts": s.E_local, "padded": s.E_local, "start": s.E_local,
           "masked_m": s.E_local, "m_indices": L.all_tokens, "src2dst": s.T * s.topk,
           "block_info": 4 * L.blocks}
    if name in i32:
        n = i32[name]
        return ws[off:off + 4 * n].view(torch.int32)
    esz = 1 if ctx.fp8 else 2
    if name in ("a", "h", "y"):
        cols = s.I if name == "h" else s.K
        nbytes = L.rows * cols * (2 if name == "y" else esz)
        v = ws[off:off + nbytes]
        if name == "y" or not ctx.fp8:
            v = v.view(torch.bfloat16)
        return v.view(L.rows, cols)
    if name in ("a_sf", "h_sf"):
        groups = (s.K if name == "a_sf" else s.I) // 128
        return ws[off:off + L.blocks * groups * 512]
    raise KeyError(name)
