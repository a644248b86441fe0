"""Python binding of libmoe_nvfp4.so, the C-ABI library of the routed MoE FFN
over NVFP4 weights on GB300 (sm_103a).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  torch provides device memory and streams.  There is no fallback: if
the library cannot be loaded, every call raises.
"""
from __future__ import annotations

import ctypes
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
           "moe_sorted_rows", "moe_sort_pairs", "moe_dispatch", "moe_combine", "moe_combine_backward"]
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
        L.moe_status_string.argtypes = [I32]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_version.restype = ctypes.c_char_p
        for n in EXPORTS:
            if n not in ("moe_status_string", "moe_version"):
                getattr(L, n).restype = I32
        L.moe_rms_norm_backward_workspace.restype = L.moe_rms_norm_backward_workspace_for.restype = SZ
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
