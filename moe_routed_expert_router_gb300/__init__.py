"""Python binding of libmoe_nvfp4.so, the C-ABI library of the routed MoE FFN
over NVFP4 weights on GB300 (sm_103a).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  torch provides device memory and streams.  There is no fallback: if
the library cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

from . import build as _build

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = _build.LIB

ROUTER_SOFTMAX, ROUTER_SIGMOID = 0, 1
ROUTER_F32, ROUTER_BF16 = 0, 1
WEIGHTS_NVFP4, WEIGHTS_MXFP4 = 0, 1
W4A16, W4A4 = 0, 1

STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED_SHAPE", 3: "MOE_ERR_MISALIGNED",
          4: "MOE_ERR_NONFINITE", 5: "MOE_ERR_TIMEOUT", 6: "MOE_ERR_CUDA", 7: "MOE_ERR_OOM", 8: "MOE_ERR_DEVICE"}
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED_SHAPE, ERR_MISALIGNED, ERR_NONFINITE, ERR_TIMEOUT, ERR_CUDA, ERR_OOM, \
    ERR_DEVICE = range(9)

EXPORTS = ["moe_plan_create", "moe_plan_destroy", "moe_route", "moe_forward", "moe_forward_host",
           "moe_quantize_act", "moe_quantize_nvfp4", "moe_plan_sync_status", "moe_plan_debug_buffer",
           "moe_plan_set_profiling", "moe_plan_read_profile", "moe_plan_set_path", "moe_plan_check_timeout",
           "moe_route_static", "moe_convert_f32", "moe_quantize_mxfp4", "moe_plan_keep_h", "moe_status_string",
           "moe_version", "moe_rms_norm", "moe_rms_norm_backward", "moe_rms_norm_backward_workspace",
           "moe_rms_norm_backward_workspace_for",
           "moe_sorted_rows", "moe_sort_pairs", "moe_dispatch", "moe_combine", "moe_combine_backward",
           "moe_head_norm", "moe_head_norm_backward", "moe_head_norm_backward_workspace",
           "moe_linear_fp4", "moe_linear_fp4_workspace", "moe_linear_fp4_workspace_for", "moe_decode_layer", "moe_decode_layer_workspace"]
FMT_E4M3, FMT_E2M1 = 0, 1
DTYPE_F32, DTYPE_BF16, DTYPE_F16 = 0, 1, 2
QUANT_NONE, QUANT_E4M3_128, QUANT_E4M3_ROW, QUANT_MXFP8 = 0, 1, 2, 3
PATH_AUTO, PATH_CUDA_CORE, PATH_TENSOR_CORE, PATH_WARP_MMA = 0, 1, 2, 3
STAGES = ["route", "group", "quant_x", "permute", "gate_up", "quant_h", "down", "finalize"]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "hidden", "inter", "num_experts", "top_k", "max_tokens", "router", "renormalize", "mode",
        "has_shared", "shared_inter", "router_dtype", "weight_format")]


class Nvfp4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("tensor_scale", ctypes.c_void_p)]


class ExpertSetC(ctypes.Structure):
    _fields_ = [("gate", Nvfp4), ("up", Nvfp4), ("down", Nvfp4)]


_lib = None


def lib():
    """Load the library (building it first if the sources are newer)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH) or not _build.up_to_date():
            _build.build()
        L = ctypes.CDLL(LIB_PATH)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        L.moe_plan_create.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(P)]
        L.moe_plan_destroy.argtypes = [P]
        L.moe_route.argtypes = [P, P, I32, P, P, P, P, P, P, P]
        L.moe_forward.argtypes = [P, P, I32, P, P, ctypes.POINTER(ExpertSetC), ctypes.POINTER(ExpertSetC), P, P]
        L.moe_forward_host.argtypes = L.moe_forward.argtypes
        L.moe_quantize_act.argtypes = [P, P, I32, P, P, P, P]
        L.moe_quantize_nvfp4.argtypes = [P, I32, I32, I32, P, P, P, P]
        L.moe_plan_sync_status.argtypes = [P, P]
        L.moe_plan_debug_buffer.argtypes = [P, ctypes.c_char_p, ctypes.POINTER(P), ctypes.POINTER(ctypes.c_size_t)]
        L.moe_plan_set_profiling.argtypes = [P, I32]
        L.moe_plan_keep_h.argtypes = [P, I32]
        L.moe_plan_set_path.argtypes = [P, I32]
        L.moe_plan_check_timeout.argtypes = [P, ctypes.c_int64, P]
        L.moe_route_static.argtypes = [P, I32, I32, P, P, I32, I32, I32, I32, P, P, P, P, P]
        L.moe_plan_read_profile.argtypes = [P, P, P, P]
        L.moe_convert_f32.argtypes = [P, ctypes.c_int64, I32, P, P]
        L.moe_quantize_mxfp4.argtypes = [P, ctypes.c_int64, I32, P, P, P]
        L.moe_rms_norm.argtypes = [P, I64, P, I64, P, I32, I32, I32, ctypes.c_float, I32, P, P, P, P, P, P]
        L.moe_rms_norm_backward.argtypes = [P, P, P, P, P, I32, I32, I32, P, P, P, SZ, P]
        L.moe_rms_norm_backward_workspace.argtypes = [I32, I32]
        L.moe_rms_norm_backward_workspace_for.argtypes = [I32, I32, I32]
        L.moe_sorted_rows.argtypes = [I64, I32, I32]
        L.moe_sort_pairs.argtypes = [P, I32, I32, I32, I32, I64, P, P, P, P]
        L.moe_dispatch.argtypes = [P, I64, I64, P, I32, I32, I32, P, P, I64, P, P, P]
        L.moe_combine.argtypes = [P, I32, I32, I32, I32, P, I64, P, P, P, P]
        L.moe_combine_backward.argtypes = [P, P, I32, I32, I32, I32, P, P, I64, P, P, P, P]
        head = [P, P, P, P, I32, I32, I32, I32, I32, I32, I32, ctypes.c_float]   # weights, positions, turns; sizes
        L.moe_head_norm.argtypes = [P, I64, P, I64, *head, P, I64, P, I64, P]
        L.moe_head_norm_backward.argtypes = [P, I64, P, I64, P, I64, P, I64, *head, P, P, P, P, P, SZ, P]
        L.moe_head_norm_backward_workspace.argtypes = [I32, I32, I32, I32, I32]
        L.moe_linear_fp4.argtypes = [P, I64, ctypes.POINTER(Nvfp4), I32, I32, I32, I32, I32, I32, P, P, SZ, P]
        L.moe_linear_fp4_workspace.argtypes = [I32, I32, I32, I32]
        L.moe_linear_fp4_workspace_for.argtypes = [I32, I32, I32, I32, I32]
        L.moe_decode_layer.argtypes = [P, I32, I32, I32, P, I32, P, I32, I32, I32, I32, P, P, P, I32, P, P, P, I32, P, P, P, P, P, SZ, P]
        L.moe_decode_layer_workspace.argtypes = [I32, I32, I32, I32, I32]
        L.moe_status_string.argtypes = [I32]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_version.restype = ctypes.c_char_p
        for n in EXPORTS:
            if n not in ("moe_status_string", "moe_version"):
                getattr(L, n).restype = I32
        L.moe_rms_norm_backward_workspace.restype = L.moe_rms_norm_backward_workspace_for.restype = SZ
        L.moe_head_norm_backward_workspace.restype = L.moe_linear_fp4_workspace.restype = L.moe_linear_fp4_workspace_for.restype = L.moe_decode_layer_workspace.restype = SZ
        L.moe_sorted_rows.restype = I64
        _lib = L
    return _lib


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream=None):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# The current stream's handle: 0.1 us a call where torch has it, 2.9 us through a Stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_devices = 0    # of this process; 0 until the first call asks


def _check(status: int, where: str):
    if status != OK:
        raise MoeError(status, where)


class NvfpTensor:
    """One NVFP4 weight stacked over experts: codes [n][N][K/2] u8, scales [n][N][K/16] u8, ts [n] f32."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, ts: torch.Tensor):
        self.codes, self.scales, self.ts = codes, scales, ts

    def c(self) -> Nvfp4:
        return Nvfp4(_ptr(self.codes), _ptr(self.scales), _ptr(self.ts))


class ExpertSet:
    def __init__(self, gate: NvfpTensor, up: NvfpTensor, down: NvfpTensor):
        self.gate, self.up, self.down = gate, up, down

    def c(self) -> ExpertSetC:
        return ExpertSetC(self.gate.c(), self.up.c(), self.down.c())


def quantize_nvfp4(w: torch.Tensor, out: NvfpTensor | None = None, stream=None) -> NvfpTensor:
    """NVFP4-quantise fp32 weights [batch][rows][cols] on the device (one tensor scale per item)."""
    assert w.is_cuda and w.dtype == torch.float32 and w.is_contiguous()
    if w.dim() == 2:
        w = w.unsqueeze(0)
    b, r, c = w.shape
    if out is None:
        out = NvfpTensor(torch.empty(b, r, c // 2, dtype=torch.uint8, device=w.device),
                         torch.empty(b, r, c // 16, dtype=torch.uint8, device=w.device),
                         torch.empty(b, dtype=torch.float32, device=w.device))
    _check(lib().moe_quantize_nvfp4(_ptr(w), b, r, c, _ptr(out.codes), _ptr(out.scales), _ptr(out.ts),
                                    _stream(stream)), "moe_quantize_nvfp4")
    return out


def quantize_mxfp4(w: torch.Tensor, out: NvfpTensor | None = None, stream=None) -> NvfpTensor:
    """MXFP4-quantise fp32 weights [batch][rows][cols] (or [rows][cols]) on the
    device: E2M1 codes and E8M0 block-of-32 scales (no tensor scale: ts is None)."""
    assert w.is_cuda and w.dtype == torch.float32 and w.is_contiguous()
    if w.dim() == 2:
        w = w.unsqueeze(0)
    b, r, c = w.shape
    if out is None:
        out = NvfpTensor(torch.empty(b, r, c // 2, dtype=torch.uint8, device=w.device),
                         torch.empty(b, r, c // 32, dtype=torch.uint8, device=w.device), None)
    _check(lib().moe_quantize_mxfp4(_ptr(w), b * r, c, _ptr(out.codes), _ptr(out.scales), _stream(stream)),
           "moe_quantize_mxfp4")
    return out


def convert_f32(src: torch.Tensor, fmt: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The device's fp32 -> E4M3 byte (FMT_E4M3) or E2M1 code (FMT_E2M1) conversion, element-wise."""
    assert src.is_cuda and src.dtype == torch.float32 and src.is_contiguous()
    if out is None:
        out = torch.empty(src.shape, dtype=torch.uint8, device=src.device)
    _check(lib().moe_convert_f32(_ptr(src), src.numel(), fmt, _ptr(out), _stream(stream)), "moe_convert_f32")
    return out


# ------------------------------------------------ the token path around the experts' products
#
# A decode step makes these calls for a few microseconds of work each, so the checks are written
# to cost little when they pass: one expression an argument, the text of a refusal only when one is due.
# A call runs on its tensors' device, whichever is current, on `stream` or else on that device's current stream.
# Where `stream` is given the caller orders it behind the work that fills the tensors and, as with any work on another
# stream, the work that uses the results behind it; new results belong to that stream, and the memory of what is given
# is held until it has passed the call.
# Autograd does not see the calls.  The forward ones refuse tensors that require a gradient while it is on; a training
# program calls the gradients' entry points itself, or from the backward() of an autograd.Function.

_DTYPES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}
_GROUP = {QUANT_E4M3_128: 128, QUANT_MXFP8: 32}
_F32, _I32 = torch.float32, torch.int32


def _refuse(where: str, what: str, status: int = ERR_INVALID_ARG):
    raise MoeError(status, f"{where} ({what})")


def _too_large(where, *sizes):
    """The entry points take sizes of 32 bits; ctypes would pass on the lower 32 of a larger one."""
    _refuse(where, f"sizes {list(sizes)}; 2^31 - 1 is the largest", ERR_UNSUPPORTED_SHAPE)


def _followed(where):
    """The call's results would be cut from the graph that autograd keeps of its tensors."""
    if torch.is_grad_enabled():
        _refuse(where, "a tensor requires grad and the result has no history: call it under torch.no_grad() or in an "
                       "autograd.Function, and the gradient's own entry point for the way back")


def _dtype(t, where):
    d = _DTYPES.get(t.dtype)
    if d is None:
        _refuse(where, f"{t.dtype} rows; float32, bfloat16 or float16 expected")
    return d


def _device(t, where):
    dev = t.device
    if dev.type != "cuda":
        _refuse(where, f"tensor on {dev}; a CUDA device expected")
    return dev


def _want(t, where, name, shape, dtype, index):
    """The tensor is where and what the kernel takes it to be; returns its address."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _refuse(where, f"{name} {t.dtype}{list(t.shape)} on {t.device}; contiguous {dtype}{list(shape)} on cuda:{index} expected")
    return t.data_ptr()


def _want_rows(t, where, name, shape, dtype, index):
    """The same of rows of contiguous values a stride apart; returns their address and stride in values."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not (t.is_contiguous() or t.stride(1) == 1):
        _refuse(where, f"{name} {t.dtype}{list(t.shape)} on {t.device}; rows of contiguous {dtype}{list(shape)} on cuda:{index} expected")
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else shape[1]


def _new(shape, dtype, dev, stream):
    """Memory that belongs to the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _given(where, index, stream, *tensors):
    """The handle of a stream that the caller names; what the call reads and writes is held for it, because torch
    would give memory that is freed meanwhile to the stream it came from."""
    if stream.device_index != index:
        _refuse(where, f"stream of cuda:{stream.device_index}, tensors on cuda:{index}")
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream


def _elsewhere(index):
    """Whether another device than the tensors' is current."""
    global _devices
    if _devices == 0:
        _devices = torch.cuda.device_count()
    return _devices != 1 and _current_device() != index


def _there(index, function):
    """The library launches on the current device: its function, with the tensors' device current for the call."""
    def call(*args):
        with torch.cuda.device(index):
            return function(*args)
    return call


# Memory of the caching allocator for a stream of the current device; torch's own function makes the device current first,
# 2 us a call where it is that already.
_raw_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)


def _workspace(n, index, handle):
    """n bytes that belong to the call's stream (None for 0); caching_allocator_delete gives them back behind the launches."""
    if not n:
        return None
    if _raw_alloc is None or _elsewhere(index):
        return torch.cuda.caching_allocator_alloc(n, index, handle)
    return _raw_alloc(n, handle)


def rms_norm(x, weight, residual=None, eps=1e-6, quant=QUANT_NONE, out=None, stream=None):
    """Residual addition and root-mean-square norm of x [T][H] (rows may be strided).

    Returns a dict of what `out` holds, or of new tensors: "rstd" [T] fp32; "sum" (x + residual) with a residual;
    "y" for QUANT_NONE, else "q" float8_e4m3fn [T][H] and its "scales" (fp32 [T][ceil(H/128)] or [T][1],
    float8_e8m0fnu [T][ceil(H/32)] for QUANT_MXFP8).  An `out` may hold "y" beside "q", leave out "sum" or "rstd"
    (not written then), and give x or residual themselves as "sum"."""
    where = "moe_rms_norm"
    shape = x.shape
    if len(shape) != 2:
        _refuse(where, "x is not [T][H]")
    T, H = shape
    if (T | H) >> 31:
        _too_large(where, T, H)
    dev, dt, code = _device(x, where), x.dtype, _dtype(x, where)
    index = dev.index
    xp, xs = _want_rows(x, where, "x", shape, dt, index)
    wp = _want(weight, where, "weight", (H,), dt, index)
    rp, rs = (None, 0) if residual is None else _want_rows(residual, where, "residual", shape, dt, index)
    if x.requires_grad or weight.requires_grad or (residual is not None and residual.requires_grad):
        _followed(where)
    sc_shape, sc_dtype = None, _F32
    if quant != QUANT_NONE:
        if quant not in (QUANT_E4M3_128, QUANT_E4M3_ROW, QUANT_MXFP8):
            _refuse(where, f"quant {quant}")
        sc_shape = (T, -(-H // _GROUP.get(quant, H or 1)))
        if quant == QUANT_MXFP8:
            sc_dtype = torch.float8_e8m0fnu
    if out is None:
        out = {"rstd": _new((T,), _F32, dev, stream)}
        if residual is not None:
            out["sum"] = _new(shape, dt, dev, stream)
        if sc_shape is None:
            out["y"] = _new(shape, dt, dev, stream)
        else:
            out["q"] = _new(shape, torch.float8_e4m3fn, dev, stream)
            out["scales"] = _new(sc_shape, sc_dtype, dev, stream)
    get = out.get
    t_sum, t_y, t_rstd, t_q, t_scales = get("sum"), get("y"), get("rstd"), get("q"), get("scales")
    if (t_sum is not None) + (t_y is not None) + (t_rstd is not None) + (t_q is not None) + (t_scales is not None) != len(out):
        _refuse(where, f"outputs {sorted(out)}; sum, y, rstd, q and scales are known")
    sp = None if t_sum is None else _want(t_sum, where, "sum", shape, dt, index)
    yp = None if t_y is None else _want(t_y, where, "y", shape, dt, index)
    dp = None if t_rstd is None else _want(t_rstd, where, "rstd", (T,), _F32, index)
    qp = cp = None
    if t_q is not None or t_scales is not None:
        if sc_shape is None or t_q is None or t_scales is None:
            _refuse(where, "q and scales go together, and with a quant")
        qp = _want(t_q, where, "q", shape, torch.float8_e4m3fn, index)
        cp = _want(t_scales, where, "scales", sc_shape, sc_dtype, index)
    handle = _raw_stream(index) if stream is None else _given(
        where, index, stream, x, weight, residual, t_sum, t_y, t_rstd, t_q, t_scales)
    call = lib().moe_rms_norm
    if _devices != 1 and _elsewhere(index):
        call = _there(index, call)
    st = call(xp, xs, rp, rs, wp, T, H, code, eps, quant, sp, yp, qp, cp, dp, handle)
    if st:
        raise MoeError(st, where)
    return out


def rms_norm_backward(grad_y, sum, weight, rstd, grad_sum=None, out=None, stream=None):
    """Gradients of rms_norm: {"grad_sum": [T][H], x's and residual's; "grad_w": [H] fp32}.

    `sum` is rms_norm's "sum" (x itself without a residual), `rstd` its "rstd"; `grad_sum` the gradient that reaches
    the sum on its other way (the residual stream)."""
    where = "moe_rms_norm_backward"
    shape = sum.shape
    if len(shape) != 2:
        _refuse(where, "sum is not [T][H]")
    T, H = shape
    if (T | H) >> 31:
        _too_large(where, T, H)
    dev, dt, code = _device(sum, where), sum.dtype, _dtype(sum, where)
    index = dev.index
    sp = _want(sum, where, "sum", shape, dt, index)
    yp = _want(grad_y, where, "grad_y", shape, dt, index)
    wp = _want(weight, where, "weight", (H,), dt, index)
    dp = _want(rstd, where, "rstd", (T,), _F32, index)
    gp = None if grad_sum is None else _want(grad_sum, where, "grad_sum", shape, dt, index)
    if out is None:
        out = {"grad_sum": _new(shape, dt, dev, stream), "grad_w": _new((H,), _F32, dev, stream)}
    op = _want(out["grad_sum"], where, "out grad_sum", shape, dt, index)
    ow = _want(out["grad_w"], where, "out grad_w", (H,), _F32, index)
    L = lib()
    n = L.moe_rms_norm_backward_workspace_for(T, H, code)
    handle = _raw_stream(index) if stream is None else _given(
        where, index, stream, grad_y, sum, weight, rstd, grad_sum, out["grad_sum"], out["grad_w"])
    call = L.moe_rms_norm_backward
    if _devices != 1 and _elsewhere(index):
        call = _there(index, call)
    # plain memory of the call's stream, given back to it behind the launches (a tensor for it costs 2.4 us more)
    ws = torch.cuda.caching_allocator_alloc(n, index, handle) if n else None
    try:
        st = call(yp, sp, wp, dp, gp, T, H, code, op, ow, ws, n, handle)
    finally:
        if ws is not None:
            torch.cuda.caching_allocator_delete(ws)
    if st:
        raise MoeError(st, where)
    return out


def sorted_rows(pairs: int, num_experts: int, align: int = 1) -> int:
    """Rows of the sorted layout, whatever the routing (moe_sorted_rows)."""
    n = -1 if (pairs | num_experts | align) >> 31 else lib().moe_sorted_rows(pairs, num_experts, align)
    if n < 0:
        _refuse("moe_sorted_rows", f"{pairs} pairs, {num_experts} experts, align {align}", ERR_UNSUPPORTED_SHAPE)
    return n


def sort_pairs(topk_ids, num_experts, align=1, out=None, stream=None):
    """Stable sort of the (token, slot) pairs by expert, from ids [T][k] int32 (outside [0, num_experts): dropped).

    Returns {"expert_offsets": [E+1], "sorted_rows": [rows] (pair at a row, -1 none), "pair_rows": [T][k] (row of a
    pair, -1 dropped)}, int32; every expert's segment is padded to a multiple of `align` rows."""
    where = "moe_sort_pairs"
    shape = topk_ids.shape
    if len(shape) != 2:
        _refuse(where, "topk_ids is not [T][k]")
    T, k = shape
    dev = _device(topk_ids, where)
    index = dev.index
    ip = _want(topk_ids, where, "topk_ids", shape, _I32, index)
    R = sorted_rows(T * k, num_experts, align)
    if out is None:
        out = {"expert_offsets": _new((num_experts + 1,), _I32, dev, stream), "sorted_rows": _new((R,), _I32, dev, stream),
               "pair_rows": _new(shape, _I32, dev, stream)}
    op = _want(out["expert_offsets"], where, "out expert_offsets", (num_experts + 1,), _I32, index)
    rp = _want(out["sorted_rows"], where, "out sorted_rows", (R,), _I32, index)
    pp = _want(out["pair_rows"], where, "out pair_rows", shape, _I32, index)
    handle = _raw_stream(index) if stream is None else _given(
        where, index, stream, topk_ids, out["expert_offsets"], out["sorted_rows"], out["pair_rows"])
    call = lib().moe_sort_pairs
    if _devices != 1 and _elsewhere(index):
        call = _there(index, call)
    st = call(ip, T, k, num_experts, align, R, op, rp, pp, handle)
    if st:
        raise MoeError(st, where)
    return out


def _order(order, where, index):
    """sort_pairs' result: the addresses of sorted_rows and pair_rows, the number of rows, T and k."""
    rows, inv = order["sorted_rows"], order["pair_rows"]
    if rows.dim() != 1 or inv.dim() != 2:
        _refuse(where, "order is not sort_pairs' result")
    R, (T, k) = rows.shape[0], inv.shape
    if (R | T | k) >> 31:
        _too_large(where, R, T, k)
    return _want(rows, where, "sorted_rows", (R,), _I32, index), _want(inv, where, "pair_rows", (T, k), _I32, index), R, T, k


def dispatch(x, order, scales=None, out=None, stream=None):
    """Token rows x [T][H] (any type; rows may be strided) into sort_pairs' order, zeros where a row holds no pair.

    Returns {"rows": [rows][H]} and, with scales [T][n], {"scales": [rows][n]}."""
    where = "moe_dispatch"
    dev = _device(x, where)
    index = dev.index
    rp, pp, R, T, k = _order(order, where, index)
    if x.dim() != 2:
        _refuse(where, "x is not [T][H]")
    H, dt, es = x.shape[1], x.dtype, x.element_size()
    xp, xs = _want_rows(x, where, "x", (T, H), dt, index)
    if x.requires_grad or (scales is not None and scales.requires_grad):
        _followed(where)
    cp, cn, sb = None, 0, 0
    if scales is not None:
        if scales.dim() != 2:
            _refuse(where, "scales is not [T][n]")
        cn = scales.shape[1]
        cp, sb = _want(scales, where, "scales", (T, cn), scales.dtype, index), cn * scales.element_size()
        if sb >> 31:
            _too_large(where, sb)
    if out is None:
        out = {"rows": _new((R, H), dt, dev, stream)}
        if scales is not None:
            out["scales"] = _new((R, cn), scales.dtype, dev, stream)
    op, oc = _want(out["rows"], where, "out rows", (R, H), dt, index), None
    if scales is not None:
        oc = _want(out["scales"], where, "out scales", (R, cn), scales.dtype, index)
    handle = _raw_stream(index) if stream is None else _given(
        where, index, stream, x, scales, order["sorted_rows"], order["pair_rows"], out["rows"],
        None if scales is None else out["scales"])
    call = lib().moe_dispatch
    if _devices != 1 and _elsewhere(index):
        call = _there(index, call)
    st = call(xp, xs * es, H * es, cp, sb, T, k, rp, pp, R, op, oc, handle)
    if st:
        raise MoeError(st, where)
    return out


def combine(y, order, weights=None, base=None, out=None, stream=None):
    """out[t] = sum_j weights[t][j] * y[row of pair (t, j)] + base[t]: expert rows y [rows][H] back into token order.

    weights [T][k] fp32 (None: 1); base [T][H] is added where given.  Rows of y that hold no pair are not read."""
    where = "moe_combine"
    dev = _device(y, where)
    index = dev.index
    rp, pp, R, T, k = _order(order, where, index)
    if y.dim() != 2:
        _refuse(where, "y is not [rows][H]")
    H, dt, code = y.shape[1], y.dtype, _dtype(y, where)
    if H >> 31:
        _too_large(where, H)
    yp = _want(y, where, "y", (R, H), dt, index)
    wp = None if weights is None else _want(weights, where, "weights", (T, k), _F32, index)
    bp = None if base is None else _want(base, where, "base", (T, H), dt, index)
    if y.requires_grad or (weights is not None and weights.requires_grad) or (base is not None and base.requires_grad):
        _followed(where)
    if out is None:
        out = _new((T, H), dt, dev, stream)
    op = _want(out, where, "out", (T, H), dt, index)
    handle = _raw_stream(index) if stream is None else _given(
        where, index, stream, y, order["pair_rows"], weights, base, out)
    call = lib().moe_combine
    if _devices != 1 and _elsewhere(index):
        call = _there(index, call)
    st = call(yp, code, T, k, H, pp, R, wp, bp, op, handle)
    if st:
        raise MoeError(st, where)
    return out


def dispatch_backward(grad_rows, order, out=None, stream=None):
    """Gradient of dispatch: [T][H], the sum of a token's rows of grad_rows [rows][H]."""
    return combine(grad_rows, order, None, None, out, stream)


def combine_backward(grad_out, y, order, weights, out=None, stream=None):
    """Gradients of combine: {"grad_y": [rows][H] (zeros where a row holds no pair), "grad_w": [T][k] fp32}.

    base's gradient is grad_out itself.  out["grad_y"] may be y."""
    where = "moe_combine_backward"
    dev = _device(y, where)
    index = dev.index
    rp, pp, R, T, k = _order(order, where, index)
    if y.dim() != 2:
        _refuse(where, "y is not [rows][H]")
    H, dt, code = y.shape[1], y.dtype, _dtype(y, where)
    if H >> 31:
        _too_large(where, H)
    yp = _want(y, where, "y", (R, H), dt, index)
    gp = _want(grad_out, where, "grad_out", (T, H), dt, index)
    wp = _want(weights, where, "weights", (T, k), _F32, index)
    if out is None:
        out = {"grad_y": _new((R, H), dt, dev, stream), "grad_w": _new((T, k), _F32, dev, stream)}
    oy = _want(out["grad_y"], where, "out grad_y", (R, H), dt, index)
    ow = _want(out["grad_w"], where, "out grad_w", (T, k), _F32, index)
    handle = _raw_stream(index) if stream is None else _given(
        where, index, stream, grad_out, y, order["sorted_rows"], order["pair_rows"], weights, out["grad_y"], out["grad_w"])
    call = lib().moe_combine_backward
    if _devices != 1 and _elsewhere(index):
        call = _there(index, call)
    st = call(gp, yp, code, T, k, H, rp, pp, R, wp, oy, ow, handle)
    if st:
        raise MoeError(st, where)
    return out


# ------------------------------------------------ around attention and in a decode step

def rotary_turns(dim, base=10000.0, frequencies=None, device="cuda"):
    """What head_norm keeps of a rotation of `dim` values: int64 [dim / 2], a plane's frequency as a fraction of a turn a
    position in units of 2^-64.  Frequencies are base ** (-2 i / dim) radians a position, or the `frequencies` given
    (dim / 2 finite numbers, of a scaled rotation for instance)."""
    where = "rotary_turns"
    if dim < 0 or dim % 16:
        _refuse(where, f"dim {dim}; a multiple of 16 expected", ERR_UNSUPPORTED_SHAPE)
    if frequencies is None and not 0 < base < math.inf:
        _refuse(where, f"base {base}")
    try:
        freqs = [base ** (-2.0 * i / dim) for i in range(dim // 2)] if frequencies is None else [float(f) for f in frequencies]
    except OverflowError:
        _refuse(where, f"base {base}, whose frequencies pass the largest number")
    if len(freqs) != dim // 2 or not all(math.isfinite(f) for f in freqs):
        _refuse(where, f"{len(freqs)} frequencies for dim {dim}; dim / 2 finite numbers expected")
    turns = [math.floor(math.fmod(f / (2 * math.pi), 1.0) * 2.0 ** 64) % 2 ** 64 for f in freqs]      # whole turns drop out exactly
    return torch.tensor([t - 2 ** 64 if t >> 63 else t for t in turns], dtype=torch.int64, device=device)


def _want_heads(t, where, name, shape, dtype, index):
    """Heads of contiguous values behind one another, tokens a stride apart; returns their address and stride in values."""
    T, n, D = shape
    steps = t.stride()
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or (
            (steps[2] != 1 or (steps[1] != D and n != 1)) and not t.is_contiguous()):
        _refuse(where, f"{name} {t.dtype}{list(t.shape)} on {t.device}; heads of contiguous {dtype}{list(shape)} on cuda:{index} expected")
    return t.data_ptr(), steps[0] if T > 1 else n * D


def _heads(q, k, q_weight, k_weight, positions, turns, where):
    """The checks that both directions of head_norm share."""
    if len(q.shape) != 3 or len(k.shape) != 3 or len(turns.shape) != 1:
        _refuse(where, "q, k are not [T][heads][D] or turns is not [R / 2]")
    T, nq, D = q.shape
    nk, R = k.shape[1], 2 * turns.shape[0]
    if (T | nq | nk | D | R) >> 31:
        _too_large(where, T, nq, nk, D, R)
    dev, dt, code = _device(q, where), q.dtype, _dtype(q, where)
    index = dev.index
    qp, qs = _want_heads(q, where, "q", (T, nq, D), dt, index)
    kp, ks = _want_heads(k, where, "k", (T, nk, D), dt, index)
    small = (_want(q_weight, where, "q_weight", (D,), dt, index), _want(k_weight, where, "k_weight", (D,), dt, index),
             _want(positions, where, "positions", (T,), _I32, index) if R else None,
             _want(turns, where, "turns", (R // 2,), torch.int64, index) if R else None)
    return dev, index, dt, code, (qp, qs, kp, ks), small, (T, nq, nk, D, R)


def head_norm(q, k, q_weight, k_weight, positions, turns, interleaved=False, eps=1e-6, out=None, stream=None):
    """Root-mean-square norm of every head of q [T][heads][D] and k [T][heads][D] and the rotation of its first
    2 * len(turns) values by the token's position (int32 [T]); turns is rotary_turns' tensor (an empty one: no rotation).

    The planes of the rotation are values i and i + R / 2, or 2 i and 2 i + 1 where interleaved.  A token's heads lie
    behind one another and tokens may be strided, as in parts of one product's rows.  Returns {"q", "k"}: new tensors, or
    `out`'s, which may be strided as well and may be q and k themselves."""
    where = "moe_head_norm"
    dev, index, dt, code, given, small, sizes = _heads(q, k, q_weight, k_weight, positions, turns, where)
    if q.requires_grad or k.requires_grad or q_weight.requires_grad or k_weight.requires_grad:
        _followed(where)
    if out is None:
        out = {"q": _new(q.shape, dt, dev, stream), "k": _new(k.shape, dt, dev, stream)}
    op, os_ = _want_heads(out["q"], where, "out q", q.shape, dt, index)
    pp, ps = _want_heads(out["k"], where, "out k", k.shape, dt, index)
    handle = _raw_stream(index) if stream is None else _given(
        where, index, stream, q, k, q_weight, k_weight, positions, turns, out["q"], out["k"])
    call = lib().moe_head_norm
    if _devices != 1 and _elsewhere(index):
        call = _there(index, call)
    st = call(*given, *small, *sizes, int(bool(interleaved)), code, eps, op, os_, pp, ps, handle)
    if st:
        raise MoeError(st, where)
    return out


def head_norm_backward(grad_q, grad_k, q, k, q_weight, k_weight, positions, turns, interleaved=False, eps=1e-6, out=None,
                       stream=None):
    """Gradients of head_norm: {"grad_q", "grad_k" as q and k, contiguous; "grad_qw", "grad_kw": [D] fp32}.

    q and k are head_norm's inputs.  out's "grad_q" and "grad_k" may be the given gradients or inputs where those are
    contiguous."""
    where = "moe_head_norm_backward"
    dev, index, dt, code, given, small, sizes = _heads(q, k, q_weight, k_weight, positions, turns, where)
    gp, gs = _want_heads(grad_q, where, "grad_q", q.shape, dt, index)
    hp, hs = _want_heads(grad_k, where, "grad_k", k.shape, dt, index)
    D = sizes[3]
    if out is None:
        out = {"grad_q": _new(q.shape, dt, dev, stream), "grad_k": _new(k.shape, dt, dev, stream),
               "grad_qw": _new((D,), _F32, dev, stream), "grad_kw": _new((D,), _F32, dev, stream)}
    outs = (_want(out["grad_q"], where, "out grad_q", q.shape, dt, index), _want(out["grad_k"], where, "out grad_k", k.shape, dt, index),
            _want(out["grad_qw"], where, "out grad_qw", (D,), _F32, index), _want(out["grad_kw"], where, "out grad_kw", (D,), _F32, index))
    L = lib()
    n = L.moe_head_norm_backward_workspace(*sizes)
    handle = _raw_stream(index) if stream is None else _given(
        where, index, stream, grad_q, grad_k, q, k, q_weight, k_weight, positions, turns, out["grad_q"], out["grad_k"], out["grad_qw"],
        out["grad_kw"])
    call = L.moe_head_norm_backward
    if _devices != 1 and _elsewhere(index):
        call = _there(index, call)
    ws = _workspace(n, index, handle)
    try:
        st = call(gp, gs, hp, hs, *given, *small, *sizes, int(bool(interleaved)), code, eps, *outs, ws, n, handle)
    finally:
        if ws is not None:
            torch.cuda.caching_allocator_delete(ws)
    if st:
        raise MoeError(st, where)
    return out


_U8 = torch.uint8


def linear_fp4(x, weight: NvfpTensor, out=None, out_dtype=None, stream=None):
    """x [T][K] (bfloat16 or float16; rows may be strided) times the transpose of one 4-bit weight [N][K], as
    quantize_nvfp4 and quantize_mxfp4 give it: [T][N] in x's type, or in float32 with out_dtype=torch.float32.  out
    overlaps nothing else.

    Made for the few tokens of a decode step: every 32 of them read the weight, or every 16 where the product is large
    enough for the tensor cores that take 4-bit operands."""
    where = "moe_linear_fp4"
    codes, scales, ts = weight.codes, weight.scales, weight.ts
    shape, rows = x.shape, codes.shape[-2:]
    if len(shape) != 2 or len(rows) != 2 or len(scales.shape) < 2:
        _refuse(where, "x is not [T][K] or the weight's codes are not [N][K / 2]")
    T, K = shape
    N = rows[0]
    if (T | K | N) >> 31:
        _too_large(where, T, K, N)
    dev, dt = _device(x, where), x.dtype
    index = dev.index
    code = DTYPE_BF16 if dt is torch.bfloat16 else DTYPE_F16 if dt is torch.float16 else _refuse(where, f"{dt} rows; bfloat16 or float16 expected")
    xp, xs = _want_rows(x, where, "x", shape, dt, index)
    lead = codes.shape[:-2]
    if lead != () and lead != (1,):
        _refuse(where, f"codes {list(codes.shape)}; one weight expected")
    wp = _want(codes, where, "codes", (*lead, N, K // 2), _U8, index)
    fmt = WEIGHTS_MXFP4 if ts is None else WEIGHTS_NVFP4
    sp = _want(scales, where, "scales", (*lead, N, K // (32 if ts is None else 16)), _U8, index)
    tp = None
    if ts is not None:
        if ts.numel() != 1:
            _refuse(where, f"tensor scale {list(ts.shape)}; one value expected")
        tp = _want(ts, where, "tensor scale", ts.shape, _F32, index)
    if x.requires_grad:
        _followed(where)
    if out is None:
        out = _new((T, N), dt if out_dtype is None else out_dtype, dev, stream)
    elif out_dtype is not None and out.dtype is not out_dtype:
        _refuse(where, f"out {out.dtype}; {out_dtype} asked for")
    to = out.dtype
    if to is not dt and to is not _F32:
        _refuse(where, f"out {to}; {dt} or float32 expected")
    op = _want(out, where, "out", (T, N), to, index)
    handle = _raw_stream(index) if stream is None else _given(where, index, stream, x, codes, scales, ts, out)
    L = lib()
    n = L.moe_linear_fp4_workspace_for(fmt, code, T, N, K) if T * N * K >> 28 else 0       # a smaller product never wants one
    call = L.moe_linear_fp4
    if _devices != 1 and _elsewhere(index):
        call = _there(index, call)
    ws = _workspace(n, index, handle) if n else None
    try:
        st = call(xp, xs, ctypes.byref(Nvfp4(wp, sp, tp)), fmt, T, N, K, code, DTYPE_F32 if to is _F32 else code, op, ws, n, handle)
    finally:
        if ws is not None:
            torch.cuda.caching_allocator_delete(ws)
    if st:
        raise MoeError(st, where)
    return out


def _ffn(where, name, weights, lead, H, dtype, index):
    """An expert set's gate, up and down: their addresses and the intermediate size."""
    gate, up, down = weights
    if len(gate.shape) != len(lead) + 2:
        _refuse(where, f"{name}gate {list(gate.shape)}; {len(lead) + 2} dimensions expected")
    I = gate.shape[-2]
    return (_want(gate, where, name + "gate", (*lead, I, H), dtype, index), _want(up, where, name + "up", (*lead, I, H), dtype, index),
            _want(down, where, name + "down", (*lead, H, I), dtype, index)), I


def decode_layer(x, router_w, gate, up, down, top_k, router_bias=None, router=ROUTER_SOFTMAX, renormalize=True, shared=None, base=None,
                 out=None, stream=None):
    """The whole mixture-of-experts layer of a decode step's tokens, x [T][H] with T up to 16: router [E][H] (float32 or
    bfloat16), gate and up [E][I][H] and down [E][H][I] in x's type, and where given the shared expert's (gate, up, down)
    and base [T][H], which is added.

    Returns {"out": [T][H], "topk_ids": [T][k] int32, "topk_w": [T][k] fp32}; the ids are Plan.route's.  out's "out" may
    be x or base."""
    where = "moe_decode_layer"
    shape = x.shape
    if len(shape) != 2 or len(gate.shape) != 3 or len(router_w.shape) != 2:
        _refuse(where, "x is not [T][H], gate not [E][I][H] or router_w not [E][H]")
    T, H = shape
    E = gate.shape[0]
    dev, dt, code = _device(x, where), x.dtype, _dtype(x, where)
    index = dev.index
    xp = _want(x, where, "x", shape, dt, index)
    rt = router_w.dtype
    if rt is not _F32 and rt is not torch.bfloat16:
        _refuse(where, f"router_w {rt}; float32 or bfloat16 expected")
    rp = _want(router_w, where, "router_w", (E, H), rt, index)
    if router != ROUTER_SOFTMAX and router != ROUTER_SIGMOID:
        _refuse(where, f"router {router}")
    ep, I = _ffn(where, "", (gate, up, down), (E,), H, dt, index)
    if (T | H | E | I | top_k) >> 31:
        _too_large(where, T, H, E, I, top_k)
    bp = None if router_bias is None else _want(router_bias, where, "router_bias", (E,), _F32, index)
    sp, Is = (None, None, None), 0
    if shared is not None:
        sp, Is = _ffn(where, "shared ", shared, (), H, dt, index)
        if Is == 0 or Is >> 31:
            _refuse(where, f"a shared expert of {Is} features", ERR_UNSUPPORTED_SHAPE)
    ap = None if base is None else _want(base, where, "base", shape, dt, index)
    if (x.requires_grad or router_w.requires_grad or gate.requires_grad or up.requires_grad or down.requires_grad
            or (router_bias is not None and router_bias.requires_grad) or (base is not None and base.requires_grad)
            or (shared is not None and any(t.requires_grad for t in shared))):
        _followed(where)
    if out is None:
        out = {"out": _new(shape, dt, dev, stream), "topk_ids": _new((T, top_k), _I32, dev, stream), "topk_w": _new((T, top_k), _F32, dev, stream)}
    op = _want(out["out"], where, "out", shape, dt, index)
    ip, wp = _want(out["topk_ids"], where, "topk_ids", (T, top_k), _I32, index), _want(out["topk_w"], where, "topk_w", (T, top_k), _F32, index)
    L = lib()
    n = L.moe_decode_layer_workspace(T, E, I, top_k, Is)
    handle = _raw_stream(index) if stream is None else _given(
        where, index, stream, x, router_w, gate, up, down, router_bias, base, *(shared or ()), out["out"], out["topk_ids"], out["topk_w"])
    call = L.moe_decode_layer
    if _devices != 1 and _elsewhere(index):
        call = _there(index, call)
    ws = _workspace(n, index, handle)
    try:
        st = call(xp, code, T, H, rp, ROUTER_F32 if rt is _F32 else ROUTER_BF16, bp, E, top_k, router, int(bool(renormalize)), *ep, I, *sp, Is, ap,
                  op, ip, wp, ws, n, handle)
    finally:
        if ws is not None:
            torch.cuda.caching_allocator_delete(ws)
    if st:
        raise MoeError(st, where)
    return out


class Plan:
    """A moe_plan: configuration plus device workspace for up to max_tokens tokens."""

    def __init__(self, hidden, inter, num_experts, top_k, max_tokens, router=ROUTER_SOFTMAX, renormalize=True,
                 mode=W4A16, has_shared=False, shared_inter=0, router_dtype=ROUTER_F32, weight_format=WEIGHTS_NVFP4):
        self.cfg = Config(hidden, inter, num_experts, top_k, max_tokens, router, int(bool(renormalize)), mode,
                          int(bool(has_shared)), shared_inter if has_shared else 0, router_dtype, weight_format)
        h = ctypes.c_void_p()
        _check(lib().moe_plan_create(ctypes.byref(self.cfg), ctypes.byref(h)), "moe_plan_create")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None) and self.handle.value:
            lib().moe_plan_destroy(self.handle)
            self.handle = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *a):
        self.close()

    def route(self, x, router_w, router_bias=None, out=None, stream=None):
        T = x.shape[0]
        k, E = self.cfg.top_k, self.cfg.num_experts
        dev = x.device
        if out is None:
            out = dict(topk_ids=torch.empty(T, k, dtype=torch.int32, device=dev),
                       topk_w=torch.empty(T, k, dtype=torch.float32, device=dev),
                       expert_offsets=torch.empty(E + 1, dtype=torch.int32, device=dev),
                       sorted_rows=torch.empty(max(T * k, 1), dtype=torch.int32, device=dev))
        _check(lib().moe_route(self.handle, _ptr(x), T, _ptr(router_w), _ptr(router_bias), _ptr(out["topk_ids"]),
                               _ptr(out["topk_w"]), _ptr(out["expert_offsets"]), _ptr(out["sorted_rows"]),
                               _stream(stream)), "moe_route")
        return out

    def forward(self, x, router_w, router_bias, routed: ExpertSet, shared: ExpertSet | None = None, out=None,
                stream=None):
        T = x.shape[0]
        if out is None:
            out = torch.empty(T, self.cfg.hidden, dtype=torch.bfloat16, device=x.device)
        rs = routed.c()
        ss = shared.c() if shared is not None else None
        _check(lib().moe_forward(self.handle, _ptr(x), T, _ptr(router_w), _ptr(router_bias), ctypes.byref(rs),
                                 ctypes.byref(ss) if ss is not None else None, _ptr(out), _stream(stream)),
               "moe_forward")
        return out

    def forward_host(self, x_host, router_w, router_bias, routed: ExpertSet, shared: ExpertSet | None, out_host,
                     stream=None):
        T = x_host.shape[0]
        rs = routed.c()
        ss = shared.c() if shared is not None else None
        _check(lib().moe_forward_host(self.handle, _ptr(x_host), T, _ptr(router_w), _ptr(router_bias),
                                      ctypes.byref(rs), ctypes.byref(ss) if ss is not None else None,
                                      _ptr(out_host), _stream(stream)), "moe_forward_host")
        return out_host

    def quantize_act(self, x, stream=None):
        T, H = x.shape
        codes = torch.empty(T, H // 2, dtype=torch.uint8, device=x.device)
        scales = torch.empty(T, H // (32 if self.cfg.weight_format == WEIGHTS_MXFP4 else 16), dtype=torch.uint8,
                             device=x.device)
        ts = torch.empty(1, dtype=torch.float32, device=x.device)
        _check(lib().moe_quantize_act(self.handle, _ptr(x), T, _ptr(codes), _ptr(scales), _ptr(ts), _stream(stream)),
               "moe_quantize_act")
        return codes, scales, ts

    def sync_status(self, stream=None) -> int:
        return lib().moe_plan_sync_status(self.handle, _stream(stream))

    def check_timeout(self, wait_ns: int, stream=None):
        _check(lib().moe_plan_check_timeout(self.handle, wait_ns, _stream(stream)), "moe_plan_check_timeout")

    def set_path(self, path: int):
        _check(lib().moe_plan_set_path(self.handle, path), "moe_plan_set_path")

    def keep_h(self, on: bool):
        """Store the fp32 SwiGLU output also where gate/up quantises it itself (MXFP4 W4A4, tensor cores)."""
        _check(lib().moe_plan_keep_h(self.handle, int(bool(on))), "moe_plan_keep_h")

    def set_profiling(self, on: bool):
        _check(lib().moe_plan_set_profiling(self.handle, int(bool(on))), "moe_plan_set_profiling")

    def read_profile(self):
        """Per-stage summed event ms, kernel launches and executions since the last read."""
        import numpy as np
        ms = np.zeros(len(STAGES), np.float32)
        la = np.zeros(len(STAGES), np.int64)
        ca = np.zeros(len(STAGES), np.int64)
        _check(lib().moe_plan_read_profile(self.handle, ms.ctypes.data, la.ctypes.data, ca.ctypes.data),
               "moe_plan_read_profile")
        return {s: (float(ms[i]), int(la[i]), int(ca[i])) for i, s in enumerate(STAGES)}

    def debug_buffer(self, name: str):
        p = ctypes.c_void_p()
        n = ctypes.c_size_t()
        _check(lib().moe_plan_debug_buffer(self.handle, name.encode(), ctypes.byref(p), ctypes.byref(n)),
               "moe_plan_debug_buffer")
        return p.value, n.value


def device_view(ptr: int, nbytes: int, dtype=torch.uint8, device="cuda"):
    """A torch view of plan-owned device memory (for tests)."""
    class _A:
        __cuda_array_interface__ = {"shape": (nbytes,), "typestr": "|u1", "data": (ptr, False), "version": 3}
    t = torch.as_tensor(_A(), device=device)
    return t.view(dtype)
