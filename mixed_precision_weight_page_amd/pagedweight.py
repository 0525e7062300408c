"""ctypes binding of libpagedweight.so (include/pagedweight.h).

Argument marshalling only: every function checks dtypes, devices and
contiguity, passes raw pointers and the current HIP stream to the C ABI and
turns a negative status into ``PagedWeightError``. The ordinary calls of
rms_norm, quantize_fp8, linear_fp8 and grouped_linear go through a small
extension module instead (binding/fastcall.cpp: the same checks, half the host
time), which leaves everything else to the functions here. All computation happens in
the library's HIP kernels; if the library is not built, importing the
binding works but every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional, Sequence, Tuple, Union

import numpy as np
import torch
from torch.autograd import forward_ad as _forward_ad

# PW_LIBRARY may name another build of the same library (the tests' host
# sanitizer build); by default the one built in-tree
_LIB_PATH = os.environ.get("PW_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)),
                                                         "libpagedweight.so")
_lib = None

PW_MASTER_F32 = 0
PW_MASTER_F16 = 1
PW_LAYOUT_EQ2 = 0
PW_LAYOUT_BITPLANE = 1
BITS = (3, 4, 8)


try:
    from . import _fastcall as _fast
except ImportError:   # not built
    _fast = None


class PagedWeightError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"pagedweight error {status}: {message}")
        self.status = status


class LayerDesc(ctypes.Structure):
    _fields_ = [("num_experts", ctypes.c_int32), ("d_model", ctypes.c_int32),
                ("d_ff", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("max_tokens", ctypes.c_int32),
                ("master_dtype", ctypes.c_int32), ("layout", ctypes.c_int32)]


class PageEntry(ctypes.Structure):
    _fields_ = [("offset", ctypes.c_uint64), ("nbytes", ctypes.c_uint64),
                ("scale", ctypes.c_float), ("bits", ctypes.c_uint8),
                ("pad_", ctypes.c_uint8 * 3)]


class ProfileData(ctypes.Structure):
    _fields_ = [("route_ms", ctypes.c_double), ("gate_up_ms", ctypes.c_double),
                ("down_ms", ctypes.c_double), ("combine_ms", ctypes.c_double),
                ("forwards", ctypes.c_int64)]


class BudgetPolicy(ctypes.Structure):
    """pw_budget_policy: memory shared by the pool and the KV cache, bytes
    kept free, headroom fraction, steps from a change to the next grow."""
    _fields_ = [("memory_bytes", ctypes.c_uint64), ("reserve_bytes", ctypes.c_uint64),
                ("headroom", ctypes.c_double), ("min_interval", ctypes.c_int32)]


BUDGET_KEEP, BUDGET_SHRINK, BUDGET_GROW, BUDGET_INIT = 0, 1, 2, 3

class GateDesc(ctypes.Structure):
    """pw_gate_desc: score, groups, groups kept, group score, renormalisation, scale."""
    _fields_ = [("score", ctypes.c_int32), ("n_group", ctypes.c_int32), ("topk_group", ctypes.c_int32),
                ("group_top2", ctypes.c_int32), ("renorm", ctypes.c_int32), ("scale", ctypes.c_float)]


class LinearDesc(ctypes.Structure):
    """pw_linear_desc: sizes, types, activation, row distances in elements."""
    _fields_ = [("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32),
                ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32), ("act", ctypes.c_int32),
                ("ldx", ctypes.c_int64), ("ldw", ctypes.c_int64), ("ldr", ctypes.c_int64), ("ldy", ctypes.c_int64)]


class RmsNormDesc(ctypes.Structure):
    """pw_rms_norm_desc: sizes, types, row distances, distances of scales, eps."""
    _fields_ = [("T", ctypes.c_int32), ("n", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("residual_dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("ldx", ctypes.c_int64), ("ldr", ctypes.c_int64), ("ldh", ctypes.c_int64), ("ldy", ctypes.c_int64),
                ("s_row", ctypes.c_int64), ("s_block", ctypes.c_int64), ("eps", ctypes.c_float)]


class QuantizeDesc(ctypes.Structure):
    """pw_quantize_desc: sizes, type, block shape, distances of x, q and scales."""
    _fields_ = [("batch", ctypes.c_int32), ("M", ctypes.c_int32), ("K", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("tile", ctypes.c_int32), ("ldx", ctypes.c_int64), ("x_batch", ctypes.c_int64),
                ("ldq", ctypes.c_int64), ("q_batch", ctypes.c_int64), ("s_row", ctypes.c_int64),
                ("s_block", ctypes.c_int64), ("s_batch", ctypes.c_int64)]


class LinearFp8Desc(ctypes.Structure):
    """pw_linear_fp8_desc: sizes, types, activation, distances of rows and scales."""
    _fields_ = [("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("act", ctypes.c_int32), ("ldx", ctypes.c_int64), ("ldw", ctypes.c_int64), ("ldr", ctypes.c_int64),
                ("ldy", ctypes.c_int64), ("xs_row", ctypes.c_int64), ("xs_block", ctypes.c_int64),
                ("ws_row", ctypes.c_int64), ("ws_block", ctypes.c_int64)]


class GroupedDesc(ctypes.Structure):
    """pw_grouped_desc: sizes, types, activation, distances of rows, experts and scales."""
    _fields_ = [("M", ctypes.c_int32), ("N", ctypes.c_int32), ("K", ctypes.c_int32), ("experts", ctypes.c_int32),
                ("x_rows", ctypes.c_int32), ("in_dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32),
                ("act", ctypes.c_int32), ("ldx", ctypes.c_int64), ("ldw", ctypes.c_int64), ("w_expert", ctypes.c_int64),
                ("ldr", ctypes.c_int64), ("ldy", ctypes.c_int64), ("xs_row", ctypes.c_int64),
                ("xs_block", ctypes.c_int64), ("ws_row", ctypes.c_int64), ("ws_block", ctypes.c_int64),
                ("ws_expert", ctypes.c_int64)]


class JoinDesc(ctypes.Structure):
    """pw_join_desc: sizes, types, row distances."""
    _fields_ = [("T", ctypes.c_int32), ("k", ctypes.c_int32), ("d", ctypes.c_int32), ("pairs", ctypes.c_int32),
                ("o_dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32), ("ldo", ctypes.c_int64),
                ("ldr", ctypes.c_int64), ("ldy", ctypes.c_int64)]


class Fp8(NamedTuple):
    """e4m3 codes and their fp32 scales. Rows (activations): q [M, K], scale
    [M, ceil(K / 128)]; tiles (weights): q [..., N, K], scale [...,
    ceil(N / 128), ceil(K / 128)]. A value is its code times its scale."""
    q: torch.Tensor
    scale: torch.Tensor


_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}   # pw_dtype
SCORES = {"softmax": 0, "sigmoid": 1}                                 # pw_score
GROUP_SCORES = {"max": 0, "top2": 1}
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "sigmoid": 3, "gelu": 4, "gelu_tanh": 5, "swiglu": 6}   # pw_act

_P = ctypes.c_void_p
_SIGNATURES = {
    "pw_create": (ctypes.c_int, [ctypes.POINTER(LayerDesc), ctypes.POINTER(_P)]),
    "pw_destroy": (None, [_P]),
    "pw_bind_masters": (ctypes.c_int, [_P, _P, _P, _P]),
    "pw_pool_bytes_for_bits": (ctypes.c_uint64, [_P, _P]),
    "pw_bind_pool": (ctypes.c_int, [_P, _P, ctypes.c_uint64]),
    "pw_workspace_bytes": (ctypes.c_uint64, [_P]),
    "pw_bind_workspace": (ctypes.c_int, [_P, _P, ctypes.c_uint64]),
    "pw_quantize_experts": (ctypes.c_int, [_P, _P, _P]),
    "pw_set_budget": (ctypes.c_int, [_P, ctypes.c_uint64, _P, _P, _P, _P]),
    "pw_moe_forward": (ctypes.c_int, [_P, _P, _P, ctypes.c_int32, _P, _P]),
    "pw_moe_forward_noalloc": (ctypes.c_int, [_P, _P, _P, ctypes.c_int32, _P, _P]),
    "pw_route": (ctypes.c_int, [_P, _P, ctypes.c_int32, _P, _P, _P, _P]),
    "pw_route_gated": (ctypes.c_int, [_P, ctypes.POINTER(GateDesc), _P, ctypes.c_int32, ctypes.c_int64, _P, _P,
                                      ctypes.c_int32, _P, _P, _P, _P]),
    "pw_moe_forward_routed": (ctypes.c_int, [_P, _P, _P, _P, ctypes.c_int32, _P, _P, ctypes.c_int32, _P]),
    "pw_linear": (ctypes.c_int, [ctypes.POINTER(LinearDesc), _P, _P, _P, _P, _P, _P]),
    "pw_rms_norm": (ctypes.c_int, [ctypes.POINTER(RmsNormDesc), _P, _P, _P, _P, _P, _P, _P]),
    "pw_quantize_fp8": (ctypes.c_int, [ctypes.POINTER(QuantizeDesc), _P, _P, _P, _P]),
    "pw_linear_fp8": (ctypes.c_int, [ctypes.POINTER(LinearFp8Desc), _P, _P, _P, _P, _P, _P, _P, _P]),
    "pw_grouped_linear": (ctypes.c_int, [ctypes.POINTER(GroupedDesc), _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "pw_group_routes": (ctypes.c_int, [_P, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _P, _P, _P, _P]),
    "pw_join_routes": (ctypes.c_int, [ctypes.POINTER(JoinDesc), _P, _P, _P, _P, _P, _P]),
    "pw_get_page_table": (ctypes.c_int, [_P, ctypes.POINTER(PageEntry)]),
    "pw_get_loss_table": (ctypes.c_int, [_P, _P, _P]),
    "pw_solve_allocation": (ctypes.c_int, [ctypes.c_int32, _P, _P, _P, ctypes.c_uint64, _P]),
    "pw_solve_allocation_layers": (ctypes.c_int, [ctypes.c_int32, _P, _P, _P, _P, _P, ctypes.c_uint64, _P, _P]),
    "pw_proportional_bits": (ctypes.c_int, [ctypes.c_int32, _P, _P, ctypes.c_uint64, _P, _P]),
    "pw_budget_decide": (ctypes.c_int, [ctypes.POINTER(BudgetPolicy), ctypes.c_uint64, ctypes.c_int32, _P,
                                        ctypes.c_uint64, ctypes.c_uint64, ctypes.c_int32, _P, _P, _P]),
    "pw_budget_step": (ctypes.c_int, [_P, ctypes.POINTER(BudgetPolicy), ctypes.c_uint64, _P, _P, _P, _P, _P, _P]),
    "pw_pool_used_bytes": (ctypes.c_uint64, [_P]),
    "pw_bind_host_tier": (ctypes.c_int, [_P, _P, ctypes.c_uint64]),
    "pw_get_residency": (ctypes.c_int, [_P, _P, _P, _P]),
    "pw_profile": (ctypes.c_int, [_P, ctypes.c_int32]),
    "pw_profile_read": (ctypes.c_int, [_P, ctypes.POINTER(ProfileData)]),
    "pw_last_error": (ctypes.c_char_p, [_P]),
    "pw_status_str": (ctypes.c_char_p, [ctypes.c_int32]),
}


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is not built; run __graft_entry__.build()")
        handle = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        if _fast is not None:
            _fast.bind(*(ctypes.cast(getattr(handle, n), _P).value
                         for n in ("pw_rms_norm", "pw_quantize_fp8", "pw_linear_fp8", "pw_grouped_linear")))
        _lib = handle
    return _lib


def library_path() -> str:
    return _LIB_PATH


def _check(status: int, ctx=None):
    if status != 0:
        L = lib()
        msg = L.pw_last_error(ctx).decode() if ctx else ""
        if not msg:
            msg = L.pw_status_str(status).decode()
        raise PagedWeightError(status, msg)


def _stream(stream=None) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _dev(t: torch.Tensor, dtype, name: str) -> int:
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


# handle of a device's current stream, without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)


# its number (of a device that a tensor lives on: the runtime is up)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on_gpu(t, dev: int, name: str):
    if isinstance(t, torch.Tensor) and t.requires_grad and torch.is_grad_enabled():
        raise ValueError(f"{name} requires a gradient, but this call is forward only: detach it, "
                         "or call under torch.no_grad()")
    if _forward_ad._current_level >= 0 and isinstance(t, torch.Tensor) and _forward_ad.unpack_dual(t).tangent is not None:
        raise ValueError(f"{name} carries a forward-mode tangent, which this call would drop: "
                         "pass torch.autograd.forward_ad.unpack_dual(...).primal")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the other tensors on cuda:{dev}")


def _here(t, name: str):
    """(device index, raw handle of its current stream) of a call on t. The
    library launches on the current device, so t has to live there."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    dev = t.get_device()
    if dev != _current_device():
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{torch.cuda.current_device()}")
    return dev, _raw_stream(dev)


def _whole(t, dtype, shape, dev: int, name: str) -> int:
    """Pointer of a contiguous tensor of the given type and shape."""
    _on_gpu(t, dev, name)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _rows(t, dtypes, shape, dev: int, name: str):
    """Pointer and row distance (in elements) of a 2-d tensor with
    contiguous rows."""
    _on_gpu(t, dev, name)
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    ld, one = t.stride()
    if one != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), ld


def _other_stream(stream):
    """None if `stream` is the current one (or None), else it as a torch
    stream. An integer is a handle on the current device, 0 its default stream."""
    if stream is None:
        return None
    here = torch.cuda.current_stream()
    if hasattr(stream, "cuda_stream"):
        return None if (stream.cuda_stream, stream.device) == (here.cuda_stream, here.device) else stream
    raw = int(stream)
    if raw == here.cuda_stream:
        return None
    # ExternalStream takes a null handle for none given, and makes a new stream
    return torch.cuda.default_stream() if raw == 0 else torch.cuda.ExternalStream(raw)


def _record(arg, stream):
    """Tensors of an argument, or of pairs and sequences of them, are not
    reused before `stream` is done with them."""
    if isinstance(arg, torch.Tensor):
        if arg.is_cuda:
            arg.record_stream(stream)
    elif isinstance(arg, (tuple, list)):
        for a in arg:
            _record(a, stream)


def _call_on(stream, args, call):
    """call() with `stream` as the current one: what it allocates belongs to
    that stream, and what it reads or writes (among args, which only call
    itself checks) is not reused before the stream is done with it, also where
    a later part of the call raises."""
    try:
        with torch.cuda.stream(stream):
            return call()
    finally:
        _record(args, stream)


def linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "none",
           residual: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
           out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """pw_linear: y = act(x w^T + bias) + residual. x [M, K] and w [N, K] (with
    act "swiglu" [2 N, K]: gate rows, then up rows) bf16 or fp16, bias fp32,
    residual and y [M, N] of out_dtype (default: y's, residual's or x's
    type); rows may be strided. act: none, relu, silu, sigmoid, gelu,
    gelu_tanh, swiglu. residual may be y. Forward only, as the layer's calls
    below: tensors that require a gradient are refused where one is recorded."""
    side = _other_stream(stream)
    if side is not None:
        return _call_on(side, (x, w, bias, residual, y), lambda: linear(x, w, bias, act, residual, y, out_dtype))
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}")
    if not isinstance(x, torch.Tensor) or not isinstance(w, torch.Tensor) or x.dim() != 2 or w.dim() != 2:
        raise ValueError("x and w must be 2-d tensors")
    M, K = x.shape
    rows = w.shape[0]
    if act == "swiglu" and rows % 2:
        raise ValueError("swiglu: w must have as many gate as up rows")
    N = rows // 2 if act == "swiglu" else rows
    dev, raw = _here(x, "x")
    xp, ldx = _rows(x, (torch.bfloat16, torch.float16), (M, K), dev, "x")
    wp, ldw = _rows(w, (x.dtype,), (rows, K), dev, "w")
    if out_dtype is None:
        out_dtype = y.dtype if y is not None else (residual.dtype if residual is not None else x.dtype)
    if out_dtype not in _DTYPES:
        raise ValueError(f"out_dtype must be float32, float16 or bfloat16, got {out_dtype}")
    bp = None if bias is None else _whole(bias, torch.float32, (rows,), dev, "bias")
    rp, ldr = (None, N) if residual is None else _rows(residual, (out_dtype,), (M, N), dev, "residual")
    if y is None:
        y = x.new_empty((M, N), dtype=out_dtype)
        yp, ldy = y.data_ptr(), N
    else:
        yp, ldy = _rows(y, (out_dtype,), (M, N), dev, "y")
    desc = LinearDesc(M, N, K, _DTYPES[x.dtype], _DTYPES[out_dtype], ACTIVATIONS[act], ldx, ldw, ldr, ldy)
    status = lib().pw_linear(ctypes.byref(desc), xp, wp, bp, rp, yp, raw)
    if status:
        raise PagedWeightError(status, lib().pw_last_error(None).decode())
    return y


def _done(status: int):
    """Raises for a failed call that has no context."""
    if status:
        raise PagedWeightError(status, lib().pw_last_error(None).decode())


_E4M3 = torch.float8_e4m3fn
_PW_E4M3 = 3


def _blocks(n: int) -> int:
    return (n + 127) // 128


def _new_codes(like: torch.Tensor, shape) -> torch.Tensor:
    """An e4m3 tensor whose rows start 16-byte aligned, as the products like them."""
    ld = (shape[-1] + 15) & ~15
    return like.new_empty_strided(shape, (ld, 1) if len(shape) == 2 else (shape[1] * ld, ld, 1), dtype=_E4M3)


def _row_scales(like: torch.Tensor, shape) -> torch.Tensor:
    """Scales [..., M, blocks] that lie block by block, so that those of neighbouring rows are neighbours."""
    M = shape[-2]
    return like.new_empty_strided(shape, (1, M) if len(shape) == 2 else (shape[2] * M, 1, M), dtype=torch.float32)


def _strided(t, dtypes, shape, dev: int, name: str):
    """Pointer of a tensor with contiguous rows and any other distances."""
    _on_gpu(t, dev, name)
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr()


def _scales(t, shape, dev: int, name: str):
    """Pointer of an fp32 tensor of any distances."""
    _on_gpu(t, dev, name)
    if t.dtype != torch.float32 or t.shape != shape:
        raise ValueError(f"{name} must be float32 {list(shape)}, got {t.dtype} {list(t.shape)}")
    return t.data_ptr()


def _is_pair(t) -> bool:
    return isinstance(t, tuple) and len(t) == 2


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
             residual: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None, out=None,
             out_dtype: Optional[torch.dtype] = None, stream=None):
    """pw_rms_norm: y = h weight / sqrt(mean(h^2) + eps) over each row of
    h = x + residual (x, if there is none). x [T, n] float32, bf16 or fp16;
    residual of x's type or float32, h (default: a new tensor; may be residual)
    of residual's; weight [n] of any of the three types or None. out_dtype: of
    y (default x's); torch.float8_e4m3fn gives an Fp8 with a scale for each 128
    columns. out: where y goes (an Fp8 in 8 bits). Rows may be strided.
    Returns y, with a residual (y, h). Forward only."""
    if stream is None and out is None and _fast is not None:
        got = _fast.rms_norm(x, weight, eps, residual, h, out_dtype)
        if got is not None:
            if out_dtype is not _E4M3:
                return got
            return Fp8(*got) if residual is None else (Fp8(got[0], got[1]), got[2])
    side = _other_stream(stream)
    if side is not None:
        return _call_on(side, (x, weight, residual, h, out),
                        lambda: rms_norm(x, weight, eps, residual, h, out, out_dtype))
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a 2-d tensor")
    T, n = x.shape
    dev, raw = _here(x, "x")
    xp, ldx = _rows(x, _DTYPES, (T, n), dev, "x")
    if out_dtype is None:
        out_dtype = x.dtype if out is None else _E4M3 if _is_pair(out) else out.dtype
    eight = out_dtype == _E4M3
    if not eight and out_dtype not in _DTYPES:
        raise ValueError(f"out_dtype must be float32, float16, bfloat16 or float8_e4m3fn, got {out_dtype}")
    if out is not None and _is_pair(out) != eight:
        raise ValueError("out must be an Fp8 where y is float8_e4m3fn, else a tensor")
    wp = None
    if weight is not None:
        if not isinstance(weight, torch.Tensor) or weight.dtype not in _DTYPES:
            raise ValueError("weight must be a float32, float16 or bfloat16 tensor")
        wp = _whole(weight, weight.dtype, (n,), dev, "weight")
    rp = hp = None
    ldr = ldh = n
    if residual is not None:
        rp, ldr = _rows(residual, (x.dtype, torch.float32), (T, n), dev, "residual")
        if h is None:
            h = residual.new_empty((T, n))
            hp = h.data_ptr()
        else:
            hp, ldh = _rows(h, (residual.dtype,), (T, n), dev, "h")
    elif h is not None:
        raise ValueError("h without residual: it would be x")
    sp, s_row, s_block = None, 0, 0
    if out is None:
        if eight:
            y = Fp8(_new_codes(x, (T, n)), _row_scales(x, (T, _blocks(n))))
            yp, ldy, sp, s_row, s_block = y.q.data_ptr(), (n + 15) & ~15, y.scale.data_ptr(), 1, T
        else:
            y = x.new_empty((T, n), dtype=out_dtype)
            yp, ldy = y.data_ptr(), n
    elif eight:
        y = Fp8(*out)
        yp, ldy = _rows(y.q, (_E4M3,), (T, n), dev, "out")
        sp = _scales(y.scale, (T, _blocks(n)), dev, "the scales of out")
        s_row, s_block = y.scale.stride()
    else:
        y = out
        yp, ldy = _rows(y, (out_dtype,), (T, n), dev, "out")
    desc = RmsNormDesc(T, n, _DTYPES[x.dtype], 0 if residual is None else _DTYPES[residual.dtype],
                       0 if weight is None else _DTYPES[weight.dtype], _PW_E4M3 if eight else _DTYPES[out_dtype],
                       ldx, ldr, ldh, ldy, s_row, s_block, eps)
    _done(lib().pw_rms_norm(ctypes.byref(desc), xp, wp, rp, hp, yp, sp, raw))
    return y if residual is None else (y, h)


def quantize_fp8(x: torch.Tensor, block: str = "row", out=None, stream=None) -> Fp8:
    """pw_quantize_fp8: e4m3 codes and scales of x [M, K] or [batch, M, K]
    (float32, bf16 or fp16, rows may be strided). block "row": a scale for
    each 128 columns of a row (activations), "tile": for each 128 x 128 tile
    (weights; gate and up rows of a SwiGLU as [2, N, K], so that each half's
    tiles start at its first row). out: an Fp8 to write into."""
    if stream is None and out is None and _fast is not None and (block == "row" or block == "tile"):
        got = _fast.quantize_fp8(x, block == "tile")
        if got is not None:
            return Fp8(*got)
    side = _other_stream(stream)
    if side is not None:
        return _call_on(side, (x, out), lambda: quantize_fp8(x, block, out))
    if block not in ("row", "tile"):
        raise ValueError("block must be 'row' or 'tile'")
    if not isinstance(x, torch.Tensor) or x.dim() not in (2, 3):
        raise ValueError("x must be a 2-d or 3-d tensor")
    shape = x.shape
    batched = len(shape) == 3
    M, K = shape[-2:]
    dev, raw = _here(x, "x")
    xp = _strided(x, _DTYPES, shape, dev, "x")
    tile = block == "tile"
    s_shape = (*shape[:-2], _blocks(M) if tile else M, _blocks(K))
    if out is None:
        q = _new_codes(x, shape)
        scale = x.new_empty(s_shape, dtype=torch.float32) if tile else _row_scales(x, s_shape)
        qp, sp = q.data_ptr(), scale.data_ptr()
    elif not _is_pair(out):
        raise ValueError("out must be an Fp8")
    else:
        q, scale = out
        qp = _strided(q, (_E4M3,), shape, dev, "the codes of out")
        sp = _scales(scale, s_shape, dev, "the scales of out")
    (*xb, ldx, _), (*qb, ldq, _), (*sb, s_row, s_block) = x.stride(), q.stride(), scale.stride()
    desc = QuantizeDesc(shape[0] if batched else 1, M, K, _DTYPES[x.dtype], 1 if tile else 0, ldx, xb[0] if batched else 0,
                        ldq, qb[0] if batched else 0, s_row, s_block, sb[0] if batched else 0)
    _done(lib().pw_quantize_fp8(ctypes.byref(desc), xp, qp, sp, raw))
    return Fp8(q, scale)


def _out_type(out_dtype, y, residual, default):
    if out_dtype is None:
        out_dtype = y.dtype if y is not None else (residual.dtype if residual is not None else default)
    if out_dtype not in _DTYPES:
        raise ValueError(f"out_dtype must be float32, float16 or bfloat16, got {out_dtype}")
    return out_dtype


def linear_fp8(x: Fp8, w: Fp8, bias: Optional[torch.Tensor] = None, act: str = "none",
               residual: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
               out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """pw_linear_fp8: linear for e4m3 operands. x: codes [M, K] and scales
    [M, ceil(K / 128)] (quantize_fp8, rms_norm), w: codes [N, K] and scales
    [ceil(N / 128), ceil(K / 128)] (quantize_fp8 with block "tile"); with act
    "swiglu" codes [2 N, K] and the gate's scale rows, then the up half's.
    out_dtype: default y's or residual's type, else bfloat16. A float32 y is
    summed from exact products; for a 16-bit one the matrix cores keep them to
    about 2^-13 of the largest of eight neighbours along K, in half the time.
    Else as linear."""
    if stream is None and _fast is not None:
        got = _fast.linear_fp8(x, w, bias, ACTIVATIONS.get(act), residual, y, out_dtype)
        if got is not None:
            return got if y is None else y
    side = _other_stream(stream)
    if side is not None:
        return _call_on(side, (x, w, bias, residual, y), lambda: linear_fp8(x, w, bias, act, residual, y, out_dtype))
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}")
    if not _is_pair(x) or not _is_pair(w):
        raise ValueError("x and w must be Fp8 (codes and scales)")
    (xq, xs), (wq, ws) = x, w
    if not isinstance(xq, torch.Tensor) or not isinstance(wq, torch.Tensor) or xq.dim() != 2 or wq.dim() != 2:
        raise ValueError("the codes of x and w must be 2-d tensors")
    M, K = xq.shape
    rows = wq.shape[0]
    halves = 2 if act == "swiglu" else 1
    if rows % halves:
        raise ValueError("swiglu: w must have as many gate as up rows")
    N = rows // halves
    dev, raw = _here(xq, "x")
    xp, ldx = _rows(xq, (_E4M3,), (M, K), dev, "x")
    wp, ldw = _rows(wq, (_E4M3,), (rows, K), dev, "w")
    xsp = _scales(xs, (M, _blocks(K)), dev, "the scales of x")
    wsp = _scales(ws, (halves * _blocks(N), _blocks(K)), dev, "the scales of w")
    out_dtype = _out_type(out_dtype, y, residual, torch.bfloat16)
    bp = None if bias is None else _whole(bias, torch.float32, (rows,), dev, "bias")
    rp, ldr = (None, N) if residual is None else _rows(residual, (out_dtype,), (M, N), dev, "residual")
    if y is None:
        y = xq.new_empty((M, N), dtype=out_dtype)
        yp, ldy = y.data_ptr(), N
    else:
        yp, ldy = _rows(y, (out_dtype,), (M, N), dev, "y")
    desc = LinearFp8Desc(M, N, K, _DTYPES[out_dtype], ACTIVATIONS[act], ldx, ldw, ldr, ldy, *xs.stride(), *ws.stride())
    _done(lib().pw_linear_fp8(ctypes.byref(desc), xp, xsp, wp, wsp, bp, rp, yp, raw))
    return y


def grouped_linear(x: Union[torch.Tensor, Fp8], offsets: torch.Tensor, w: Union[torch.Tensor, Fp8],
                   bias: Optional[torch.Tensor] = None, act: str = "none", residual: Optional[torch.Tensor] = None,
                   y: Optional[torch.Tensor] = None, rows: Optional[torch.Tensor] = None,
                   out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """pw_grouped_linear: rows offsets[e] .. offsets[e + 1] - 1 of y are those
    of x times w[e]^T. offsets int32 [E + 1] on the device, not descending from
    0 to at most M. x [M, K] and w [E, N, K] (act "swiglu": [E, 2 N, K]) bf16 or
    fp16, or both Fp8 with scales as in linear_fp8, w's for each expert. rows
    int32 [M]: row m is row rows[m] of x, which may then have any number of rows
    (a number outside it: zeros). bias fp32 [E, N (2 N)], residual and y [M, N];
    out_dtype: default y's, residual's or x's type (bfloat16 for Fp8). Rows of
    y from offsets[E] on are left as they are (without y: not set)."""
    if stream is None and _fast is not None:
        got = _fast.grouped_linear(x, offsets, w, bias, ACTIVATIONS.get(act), residual, y, rows, out_dtype)
        if got is not None:
            return got if y is None else y
    eight = _is_pair(x)
    side = _other_stream(stream)
    if side is not None:
        return _call_on(side, (x, offsets, w, bias, residual, y, rows),
                        lambda: grouped_linear(x, offsets, w, bias, act, residual, y, rows, out_dtype))
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}")
    if eight != _is_pair(w):
        raise ValueError("x and w must both be tensors or both Fp8 (codes and scales)")
    (xq, xs), (wq, ws) = (x, w) if eight else ((x, None), (w, None))
    if not isinstance(xq, torch.Tensor) or not isinstance(wq, torch.Tensor) or xq.dim() != 2 or wq.dim() != 3:
        raise ValueError("x must be [M, K] and w [E, N, K]")
    if not isinstance(offsets, torch.Tensor) or (rows is not None and (not isinstance(rows, torch.Tensor) or rows.dim() != 1)):
        raise ValueError("offsets and rows must be 1-d tensors")
    x_rows, K = xq.shape
    E, wide = wq.shape[:2]
    halves = 2 if act == "swiglu" else 1
    if wide % halves:
        raise ValueError("swiglu: w must have as many gate as up rows")
    N = wide // halves
    M = x_rows if rows is None else rows.shape[0]
    dev, raw = _here(xq, "x")
    xp, ldx = _rows(xq, (_E4M3,) if eight else (torch.bfloat16, torch.float16), (x_rows, K), dev, "x")
    wp = _strided(wq, (xq.dtype,), (E, wide, K), dev, "w")
    xsp = wsp = None
    strides = (0, 0, 0, 0, 0)
    if eight:
        xsp = _scales(xs, (x_rows, _blocks(K)), dev, "the scales of x")
        wsp = _scales(ws, (E, halves * _blocks(N), _blocks(K)), dev, "the scales of w")
        strides = (*xs.stride(), ws.stride(1), ws.stride(2), ws.stride(0))
    op = _whole(offsets, torch.int32, (E + 1,), dev, "offsets")
    ip = None if rows is None else _whole(rows, torch.int32, (M,), dev, "rows")
    out_dtype = _out_type(out_dtype, y, residual, torch.bfloat16 if eight else xq.dtype)
    bp = None if bias is None else _whole(bias, torch.float32, (E, wide), dev, "bias")
    rp, ldr = (None, N) if residual is None else _rows(residual, (out_dtype,), (M, N), dev, "residual")
    if y is None:
        y = xq.new_empty((M, N), dtype=out_dtype)
        yp, ldy = y.data_ptr(), N
    else:
        yp, ldy = _rows(y, (out_dtype,), (M, N), dev, "y")
    desc = GroupedDesc(M, N, K, E, x_rows, _PW_E4M3 if eight else _DTYPES[xq.dtype], _DTYPES[out_dtype],
                       ACTIVATIONS[act], ldx, wq.stride(1), wq.stride(0), ldr, ldy, *strides)
    _done(lib().pw_grouped_linear(ctypes.byref(desc), xp, xsp, wp, wsp, op, ip, bp, rp, yp, raw))
    return y


def group_routes(ids: torch.Tensor, num_experts: int, stream=None):
    """pw_group_routes: the (token, slot) pairs of ids int32 [T, k] in expert
    order, as grouped_linear takes them: (offsets int32 [E + 1], rows int32
    [T k]: the token of each position, place int32 [T, k]: the position of each
    pair, -1 for an id outside [0, E))."""
    side = _other_stream(stream)
    if side is not None:
        return _call_on(side, (ids,), lambda: group_routes(ids, num_experts))
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be [T, k]")
    T, k = ids.shape
    dev, raw = _here(ids, "ids")
    ip = _whole(ids, torch.int32, (T, k), dev, "ids")
    offsets = ids.new_empty((max(num_experts, 0) + 1,))
    rows, place = ids.new_empty((T * k,)), ids.new_empty((T, k))
    _done(lib().pw_group_routes(ip, T, k, num_experts, offsets.data_ptr(), rows.data_ptr(), place.data_ptr(), raw))
    return offsets, rows, place


def join_routes(o: torch.Tensor, place: torch.Tensor, g: torch.Tensor, residual: Optional[torch.Tensor] = None,
                y: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """pw_join_routes: y_t = residual_t + sum_j g_tj o[place_tj] for o [pairs, d]
    (float32, bf16 or fp16), place int32 and g fp32 [T, k] (group_routes). y
    and residual [T, d] of out_dtype (default: y's, residual's or o's type);
    residual may be y."""
    side = _other_stream(stream)
    if side is not None:
        return _call_on(side, (o, place, g, residual, y), lambda: join_routes(o, place, g, residual, y, out_dtype))
    if not isinstance(o, torch.Tensor) or not isinstance(place, torch.Tensor) or o.dim() != 2 or place.dim() != 2:
        raise ValueError("o must be [pairs, d] and place [T, k]")
    pairs, d = o.shape
    T, k = place.shape
    dev, raw = _here(o, "o")
    op, ldo = _rows(o, _DTYPES, (pairs, d), dev, "o")
    pp = _whole(place, torch.int32, (T, k), dev, "place")
    gp = _whole(g, torch.float32, (T, k), dev, "g")
    out_dtype = _out_type(out_dtype, y, residual, o.dtype)
    rp, ldr = (None, d) if residual is None else _rows(residual, (out_dtype,), (T, d), dev, "residual")
    if y is None:
        y = o.new_empty((T, d), dtype=out_dtype)
    yp, ldy = _rows(y, (out_dtype,), (T, d), dev, "y")
    desc = JoinDesc(T, k, d, pairs, _DTYPES[o.dtype], _DTYPES[out_dtype], ldo, ldr, ldy)
    _done(lib().pw_join_routes(ctypes.byref(desc), op, pp, gp, rp, yp, raw))
    return y


def moe_experts(x: torch.Tensor, ids: torch.Tensor, g: torch.Tensor, w_gate_up: Union[torch.Tensor, Fp8],
                w_down: Union[torch.Tensor, Fp8], residual: Optional[torch.Tensor] = None,
                y: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
    """The routed experts of a block whose weights are not in pages: y_t =
    residual_t + sum_j g_tj Wd_e (silu(Wg_e x_t) * (Wu_e x_t)) with e = ids_tj
    (an id outside [0, E): no expert). x [T, d] bf16 or fp16; w_gate_up [E, 2 F,
    d] and w_down [E, d, F] of x's type, or both Fp8 with scales for 128 x 128
    tiles (x and the SwiGLU rows are then quantized by rows). group_routes, two
    grouped_linear, join_routes. Rounded on the way: the SwiGLU rows to x's type
    (and to e4m3), each pair's product to x's type unless y is float32. x has
    less than 2^31 - 64 bytes (8-bit weights: elements), as grouped_linear
    gathers its rows.
    out_dtype: default y's, residual's or x's type."""
    side = _other_stream(stream)
    if side is not None:
        return _call_on(side, (x, ids, g, w_gate_up, w_down, residual, y),
                        lambda: moe_experts(x, ids, g, w_gate_up, w_down, residual, y, out_dtype))
    eight = _is_pair(w_gate_up)
    if eight != _is_pair(w_down):
        raise ValueError("w_gate_up and w_down must both be tensors or both Fp8")
    up, down = (w_gate_up[0], w_down[0]) if eight else (w_gate_up, w_down)
    if not all(isinstance(t, torch.Tensor) for t in (x, ids, up, down)):
        raise ValueError("x, ids, w_gate_up and w_down must be tensors (8-bit weights: codes and scales)")
    if up.dim() != 3 or down.dim() != 3 or x.dim() != 2 or ids.dim() != 2 or ids.shape[0] != x.shape[0]:
        raise ValueError("x must be [T, d], ids [T, k], w_gate_up [E, 2 F, d] and w_down [E, d, F]")
    E, d = up.shape[0], x.shape[1]
    if up.shape[2] != d or tuple(down.shape) != (E, d, up.shape[1] // 2):
        raise ValueError(f"w_gate_up {list(up.shape)} and w_down {list(down.shape)} do not fit x {list(x.shape)}")
    out_dtype = _out_type(out_dtype, y, residual, x.dtype)
    offsets, rows, place = group_routes(ids, E)
    h = grouped_linear(quantize_fp8(x) if eight else x, offsets, w_gate_up, act="swiglu", rows=rows, out_dtype=x.dtype)
    o = grouped_linear(quantize_fp8(h) if eight else h, offsets, w_down,
                       out_dtype=torch.float32 if out_dtype == torch.float32 else x.dtype)
    return join_routes(o, place, g, residual, y, out_dtype)


def _host_array(a, dtype, n: int, name: str) -> np.ndarray:
    arr = np.ascontiguousarray(np.asarray(a, dtype=dtype))
    if arr.shape != (n,) and arr.size != n:
        raise ValueError(f"{name} must hold {n} values")
    return arr.reshape(-1)


def solve_allocation(W: Sequence[int], p: Sequence[float], L, budget_bits: int) -> np.ndarray:
    """pw_solve_allocation: exact host solver of Eq. 1 (no GPU needed)."""
    E = len(p)
    Wa = _host_array(W, np.uint64, E, "W")
    pa = _host_array(p, np.float64, E, "p")
    La = np.ascontiguousarray(np.asarray(L, dtype=np.float64).reshape(E * 3))
    out = np.zeros(E, dtype=np.uint8)
    _check(lib().pw_solve_allocation(E, Wa.ctypes.data, pa.ctypes.data, La.ctypes.data,
                                     int(budget_bits), out.ctypes.data))
    return out


def solve_allocation_layers(Ws, ps, Ls, budget_bits: int, layer_weights=None):
    """pw_solve_allocation_layers: one exact solve of Eq. 1 for several layers
    sharing budget_bits. Ws, ps, Ls hold one entry per layer (W[E_l], p[E_l],
    L[E_l][3]). Returns (list of per-layer bit arrays, objective)."""
    n = len(ps)
    if not (len(Ws) == len(Ls) == n) or n == 0:
        raise ValueError("Ws, ps and Ls need one entry per layer")
    E = np.array([len(v) for v in ps], dtype=np.int32)
    Wa = np.ascontiguousarray(np.concatenate([_host_array(W, np.uint64, int(e), "W") for W, e in zip(Ws, E)]))
    pa = np.ascontiguousarray(np.concatenate([_host_array(p, np.float64, int(e), "p") for p, e in zip(ps, E)]))
    La = np.ascontiguousarray(np.concatenate([np.asarray(L, dtype=np.float64).reshape(int(e) * 3)
                                              for L, e in zip(Ls, E)]))
    wa = None if layer_weights is None else _host_array(layer_weights, np.float64, n, "layer_weights")
    out = np.zeros(int(E.sum()), dtype=np.uint8)
    obj = ctypes.c_double(0.0)
    _check(lib().pw_solve_allocation_layers(n, E.ctypes.data, Wa.ctypes.data, pa.ctypes.data, La.ctypes.data,
                                            None if wa is None else wa.ctypes.data, int(budget_bits),
                                            out.ctypes.data, ctypes.byref(obj)))
    return np.split(out, np.cumsum(E)[:-1]), obj.value


def proportional_bits(W: Sequence[int], p: Sequence[float], budget_bits: int):
    """pw_proportional_bits: the pages' simplified proportional sketch (a
    comparison mode; may exceed the budget). Returns (bits, used_bits)."""
    E = len(p)
    Wa = _host_array(W, np.uint64, E, "W")
    pa = _host_array(p, np.float64, E, "p")
    out = np.zeros(E, dtype=np.uint8)
    used = ctypes.c_uint64(0)
    _check(lib().pw_proportional_bits(E, Wa.ctypes.data, pa.ctypes.data, int(budget_bits), out.ctypes.data,
                                      ctypes.byref(used)))
    return out, used.value


def set_budget_layers(layers, budget_bits: int, importances, layer_weights=None, stream=None):
    """One budget shared by several PagedMoELayer objects: each layer's loss
    table (pw_get_loss_table), one exact solve over all their experts
    (pw_solve_allocation_layers), then each layer quantized to its share
    (pw_quantize_experts; its pool must hold the new pages). Returns (list of
    per-layer bit arrays, objective)."""
    Ls = [layer.get_loss_table(stream) for layer in layers]
    Ws = [[3 * layer.d * layer.F] * layer.E for layer in layers]
    bits, obj = solve_allocation_layers(Ws, importances, Ls, budget_bits, layer_weights)
    for layer, b in zip(layers, bits):
        layer.quantize_experts(b, stream)
    return bits, obj


NO_POOL = (1 << 64) - 1   # pool_bytes_now before the first allocation


def _policy(memory_bytes, reserve_bytes, headroom, min_interval) -> BudgetPolicy:
    return BudgetPolicy(int(memory_bytes), int(reserve_bytes), float(headroom), int(min_interval))


def budget_decide(memory_bytes: int, reserve_bytes: int, headroom: float, min_interval: int,
                  kv_used_bytes: int, W: Sequence[int], pool_bytes_now: Optional[int],
                  budget_now: Optional[int], steps_since_change: int):
    """pw_budget_decide (host only): (action, budget_bits, pressure)."""
    E = len(W)
    Wa = _host_array(W, np.uint64, E, "W")
    pol = _policy(memory_bytes, reserve_bytes, headroom, min_interval)
    act, press = ctypes.c_int32(0), ctypes.c_int32(0)
    out = ctypes.c_uint64(0)
    _check(lib().pw_budget_decide(ctypes.byref(pol), int(kv_used_bytes), E, Wa.ctypes.data,
                                  NO_POOL if pool_bytes_now is None else int(pool_bytes_now),
                                  0 if budget_now is None else int(budget_now), int(steps_since_change),
                                  ctypes.byref(act), ctypes.byref(out), ctypes.byref(press)))
    return act.value, out.value, bool(press.value)


class PagedMoELayer:
    """One MoE expert layer bound to its masters, pool and workspace."""

    def __init__(self, num_experts: int, d_model: int, d_ff: int, top_k: int,
                 max_tokens: int, renorm: int = 0, master_dtype: str = "f32", layout: str = "eq2"):
        """layout: "eq2" (pages of Eq. 2 codes at 3/4/8 bits) or "bitplane"
        (prefix-compatible bitplane pages; bits are depths 1..8)."""
        self._ctx = None
        if layout not in ("eq2", "bitplane"):
            raise ValueError("layout must be 'eq2' or 'bitplane'")
        desc = LayerDesc(num_experts, d_model, d_ff, top_k, renorm, max_tokens,
                         PW_MASTER_F16 if master_dtype == "f16" else PW_MASTER_F32,
                         PW_LAYOUT_BITPLANE if layout == "bitplane" else PW_LAYOUT_EQ2)
        self.layout = layout
        ctx = _P()
        _check(lib().pw_create(ctypes.byref(desc), ctypes.byref(ctx)))
        self._ctx = ctx
        self.E, self.d, self.F, self.k = num_experts, d_model, d_ff, top_k
        self.max_tokens = max_tokens
        self.master_dtype = torch.float16 if master_dtype == "f16" else torch.float32
        self._keep = {}

    def __del__(self):
        if getattr(self, "_ctx", None) and _lib is not None:
            _lib.pw_destroy(self._ctx)
            self._ctx = None

    # ---- binding of caller-owned memory ----
    def bind_masters(self, w1: torch.Tensor, w3: torch.Tensor, w2: torch.Tensor):
        E, d, F = self.E, self.d, self.F
        if tuple(w1.shape) != (E, F, d) or tuple(w3.shape) != (E, F, d) or tuple(w2.shape) != (E, d, F):
            raise ValueError("masters must be w1, w3 [E, F, d] and w2 [E, d, F]")
        ptrs = [_dev(t, self.master_dtype, n) for t, n in ((w1, "w1"), (w3, "w3"), (w2, "w2"))]
        _check(lib().pw_bind_masters(self._ctx, *ptrs), self._ctx)
        self._keep["masters"] = (w1, w3, w2)

    def pool_bytes_for_bits(self, bits) -> int:
        b = _host_array(bits, np.uint8, self.E, "bits")
        return int(lib().pw_pool_bytes_for_bits(self._ctx, b.ctypes.data))

    def bind_pool(self, pool: torch.Tensor):
        _check(lib().pw_bind_pool(self._ctx, _dev(pool, torch.uint8, "pool"), pool.numel()), self._ctx)
        self._keep["pool"] = pool

    def bind_host_tier(self, host: Optional[torch.Tensor]):
        """Pages in pinned host memory, the pool a cache of page slots
        (pw_bind_host_tier); None goes back to pages in the pool."""
        if host is None:
            _check(lib().pw_bind_host_tier(self._ctx, None, 0), self._ctx)
            self._keep.pop("host", None)
            return
        if host.device.type != "cpu" or not host.is_pinned() or host.dtype != torch.uint8 or not host.is_contiguous():
            raise ValueError("host tier must be a contiguous pinned uint8 CPU tensor")
        _check(lib().pw_bind_host_tier(self._ctx, host.data_ptr(), host.numel()), self._ctx)
        self._keep["host"] = host

    def pool_used_bytes(self) -> int:
        """pw_pool_used_bytes: bytes of the pool the pages span (from its start)."""
        return int(lib().pw_pool_used_bytes(self._ctx))

    def slot_bytes(self) -> int:
        """Bytes of one page slot of the host tier's device cache (an 8-bit page)."""
        return (3 * self.d * self.F + 255) // 256 * 256

    def residency(self, stream=None):
        """pw_get_residency: (slot of each expert, -1 none; dict of hits,
        pages copied in, pages read from the host tier)."""
        slots = np.zeros(self.E, dtype=np.int32)
        stats = np.zeros(3, dtype=np.uint64)
        _check(lib().pw_get_residency(self._ctx, slots.ctypes.data, stats.ctypes.data, _stream(stream)),
               self._ctx)
        return slots, dict(hits=int(stats[0]), copies=int(stats[1]), host_reads=int(stats[2]))

    def workspace_bytes(self) -> int:
        return int(lib().pw_workspace_bytes(self._ctx))

    def bind_workspace(self, ws: torch.Tensor):
        _check(lib().pw_bind_workspace(self._ctx, _dev(ws, torch.uint8, "workspace"), ws.numel()),
               self._ctx)
        self._keep["workspace"] = ws

    # ---- the hot path ----
    def quantize_experts(self, bits, stream=None):
        b = _host_array(bits, np.uint8, self.E, "bits")
        _check(lib().pw_quantize_experts(self._ctx, b.ctypes.data, _stream(stream)), self._ctx)

    def set_budget(self, budget_bits: int, importance, loss=None, stream=None) -> np.ndarray:
        p = _host_array(importance, np.float64, self.E, "importance")
        L = None if loss is None else np.ascontiguousarray(np.asarray(loss, dtype=np.float64).reshape(self.E * 3))
        out = np.zeros(self.E, dtype=np.uint8)
        _check(lib().pw_set_budget(self._ctx, int(budget_bits), p.ctypes.data,
                                   None if L is None else L.ctypes.data, out.ctypes.data,
                                   _stream(stream)), self._ctx)
        return out

    def budget_step(self, memory_bytes: int, reserve_bytes: int, headroom: float, min_interval: int,
                    kv_used_bytes: int, importance, loss=None, stream=None):
        """pw_budget_step: one KV-pressure scheduler step (re-quantizes on
        INIT, SHRINK and GROW). Returns (action, budget_bits, pressure)."""
        p = _host_array(importance, np.float64, self.E, "importance")
        L = None if loss is None else np.ascontiguousarray(np.asarray(loss, dtype=np.float64).reshape(self.E * 3))
        pol = _policy(memory_bytes, reserve_bytes, headroom, min_interval)
        act, press = ctypes.c_int32(0), ctypes.c_int32(0)
        out = ctypes.c_uint64(0)
        _check(lib().pw_budget_step(self._ctx, ctypes.byref(pol), int(kv_used_bytes), p.ctypes.data,
                                    None if L is None else L.ctypes.data, ctypes.byref(act),
                                    ctypes.byref(out), ctypes.byref(press), _stream(stream)), self._ctx)
        return act.value, out.value, bool(press.value)

    def moe_forward(self, x: torch.Tensor, logits: torch.Tensor, y: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
        T = x.shape[0]
        if x.dim() != 2 or x.shape[1] != self.d or tuple(logits.shape) != (T, self.E):
            raise ValueError("x must be [T, d] and logits [T, E]")
        if y is None:
            y = torch.empty((T, self.d), dtype=torch.float32, device=x.device)
        elif tuple(y.shape) != (T, self.d):
            raise ValueError("y must be [T, d]")
        _check(lib().pw_moe_forward(self._ctx, _dev(x, torch.bfloat16, "x"),
                                    _dev(logits, torch.float32, "logits"), T,
                                    _dev(y, torch.float32, "y"), _stream(stream)), self._ctx)
        return y

    def moe_forward_noalloc(self, x: torch.Tensor, logits: torch.Tensor, y: torch.Tensor,
                            stream=None) -> torch.Tensor:
        """pw_moe_forward_noalloc: the forward with the library's static
        device scratch instead of the workspace (y is the caller's)."""
        T = x.shape[0]
        if x.dim() != 2 or x.shape[1] != self.d or tuple(logits.shape) != (T, self.E):
            raise ValueError("x must be [T, d] and logits [T, E]")
        if tuple(y.shape) != (T, self.d):
            raise ValueError("y must be [T, d]")
        _check(lib().pw_moe_forward_noalloc(self._ctx, _dev(x, torch.bfloat16, "x"),
                                            _dev(logits, torch.float32, "logits"), T,
                                            _dev(y, torch.float32, "y"), _stream(stream)), self._ctx)
        return y

    def route(self, logits: torch.Tensor, stream=None):
        T = logits.shape[0]
        ids = torch.empty((T, self.k), dtype=torch.int32, device=logits.device)
        g = torch.empty((T, self.k), dtype=torch.float32, device=logits.device)
        counts = torch.empty((self.E,), dtype=torch.int32, device=logits.device)
        _check(lib().pw_route(self._ctx, _dev(logits, torch.float32, "logits"), T,
                              ids.data_ptr(), g.data_ptr(), counts.data_ptr(), _stream(stream)),
               self._ctx)
        return ids, g, counts

    def route_gated(self, logits: torch.Tensor, score: str = "softmax", bias: Optional[torch.Tensor] = None,
                    n_group: int = 1, topk_group: int = 1, group_score: str = "max", renorm: bool = False,
                    scale: float = 1.0, mask: Optional[torch.Tensor] = None, with_counts: bool = True, stream=None):
        """pw_route_gated: (ids int32 [T, k], weights fp32 [T, k], pairs per
        expert int32 [E] or None). logits [T, E] fp32, bf16 or fp16 (rows may
        be strided); score "softmax" or "sigmoid"; bias fp32 [E] counts in
        the choice only; group_score "max" or "top2"; mask bool or uint8 [T],
        0 for padded tokens."""
        side = _other_stream(stream)
        if side is not None:
            return _call_on(side, (logits, bias, mask), lambda: self.route_gated(
                logits, score, bias, n_group, topk_group, group_score, renorm, scale, mask, with_counts))
        if score not in SCORES or group_score not in GROUP_SCORES:
            raise ValueError("score must be 'softmax' or 'sigmoid', group_score 'max' or 'top2'")
        if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
            raise ValueError("logits must be [T, E]")
        T, E, k = logits.shape[0], self.E, self.k
        dev, raw = _here(logits, "logits")
        lp, ld = _rows(logits, _DTYPES, (T, E), dev, "logits")
        bp = None if bias is None else _whole(bias, torch.float32, (E,), dev, "bias")
        mp = None
        if mask is not None:
            if mask.dtype not in (torch.bool, torch.uint8):
                raise ValueError(f"mask must be bool or uint8 [{T}]")
            mp = _whole(mask, mask.dtype, (T,), dev, "mask")
        ids = logits.new_empty((T, k), dtype=torch.int32)
        g = logits.new_empty((T, k), dtype=torch.float32)
        counts = logits.new_empty((E,), dtype=torch.int32) if with_counts else None
        desc = GateDesc(SCORES[score], n_group, topk_group, GROUP_SCORES[group_score], 1 if renorm else 0, scale)
        status = lib().pw_route_gated(self._ctx, ctypes.byref(desc), lp, _DTYPES[logits.dtype], ld, bp, mp, T,
                                      ids.data_ptr(), g.data_ptr(), None if counts is None else counts.data_ptr(), raw)
        if status:
            _check(status, self._ctx)
        return ids, g, counts

    def moe_forward_routed(self, x: torch.Tensor, ids: torch.Tensor, g: torch.Tensor,
                           residual: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                           out_dtype: Optional[torch.dtype] = None, stream=None) -> torch.Tensor:
        """pw_moe_forward_routed: the experts' products for given ids int32
        [T, k] (-1: no expert) and weights fp32 [T, k], added to residual
        [T, d] if given. y and residual are float32 or bfloat16 (out_dtype;
        default: y's or residual's type, else float32); residual may be y."""
        side = _other_stream(stream)
        if side is not None:
            return _call_on(side, (x, ids, g, residual, y),
                            lambda: self.moe_forward_routed(x, ids, g, residual, y, out_dtype))
        if x.dim() != 2 or x.shape[1] != self.d or ids.shape != (x.shape[0], self.k) or g.shape != ids.shape:
            raise ValueError("x must be [T, d], ids and g [T, k]")
        if out_dtype is None:
            out_dtype = y.dtype if y is not None else (residual.dtype if residual is not None else torch.float32)
        if out_dtype not in (torch.float32, torch.bfloat16):
            raise ValueError(f"out_dtype must be float32 or bfloat16, got {out_dtype}")
        T = x.shape[0]
        dev, raw = _here(x, "x")
        xp = _whole(x, torch.bfloat16, (T, self.d), dev, "x")
        ip = _whole(ids, torch.int32, (T, self.k), dev, "ids")
        gp = _whole(g, torch.float32, (T, self.k), dev, "g")
        rp = None if residual is None else _whole(residual, out_dtype, (T, self.d), dev, "residual")
        if y is None:
            y = torch.empty((T, self.d), dtype=out_dtype, device=x.device)
            yp = y.data_ptr()
        else:
            yp = _whole(y, out_dtype, (T, self.d), dev, "y")
        status = lib().pw_moe_forward_routed(self._ctx, xp, ip, gp, T, rp, yp, _DTYPES[out_dtype], raw)
        if status:
            _check(status, self._ctx)
        return y

    def moe_block(self, x: torch.Tensor, gate_w: torch.Tensor, gate_logit_bias: Optional[torch.Tensor] = None,
                  shared: Optional[Sequence] = None, residual: Optional[torch.Tensor] = None,
                  y: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16, stream=None,
                  norm: Optional[Tuple[Optional[torch.Tensor], float]] = None, experts: Optional[Sequence] = None, **gate):
        """A whole mixture-of-experts block on x bf16 [T, d]: router logits
        (linear with gate_w [E, d], in fp32), route_gated with the arguments
        in `gate`, the shared expert if given (w_gate_up [2 F, d] and w_down
        [d, F], any F; bf16, or Fp8 pairs as linear_fp8 takes them) and the
        routed experts, all added to residual, which has out_dtype as y has.
        norm (weight or None, eps): the block works on rms_norm of x + residual
        (of x, if there is none) and is added to that sum (to x; x has
        out_dtype then). experts (w_gate_up [E, 2 F, d], w_down [E, d, F]: bf16
        or Fp8): the routed experts from these (moe_experts) instead of the
        layer's pages, which need not exist. Rounded on the way: with a norm the
        sum to residual's type and its norm to bf16, the shared expert's SwiGLU
        rows to bf16 (8-bit weights: it and x to e4m3), residual + shared expert
        to out_dtype (float32 keeps that sum), y. Returns (y, ids, weights,
        pairs per expert)."""
        side = _other_stream(stream)
        if side is not None:
            args = (x, gate_w, gate_logit_bias, shared, residual, y, norm, experts, tuple(gate.values()))
            return _call_on(side, args, lambda: self.moe_block(x, gate_w, gate_logit_bias, shared, residual, y,
                                                                  out_dtype, None, norm, experts, **gate))
        if norm is not None:
            weight, eps = norm
            if residual is None:
                x, residual = rms_norm(x, weight, eps, out_dtype=torch.bfloat16), x
            else:
                x, residual = rms_norm(x, weight, eps, residual=residual, out_dtype=torch.bfloat16)
        logits = linear(x, gate_w, gate_logit_bias, out_dtype=torch.float32)
        ids, g, counts = self.route_gated(logits, **gate)
        base = residual
        if shared is not None:
            w_gate_up, w_down = shared
            if _is_pair(w_gate_up):
                h = linear_fp8(quantize_fp8(x), w_gate_up, act="swiglu")
                base = linear_fp8(quantize_fp8(h), w_down, residual=residual, out_dtype=out_dtype)
            else:
                base = linear(linear(x, w_gate_up, act="swiglu"), w_down, residual=residual, out_dtype=out_dtype)
        if experts is not None:
            return moe_experts(x, ids, g, *experts, residual=base, y=y, out_dtype=out_dtype), ids, g, counts
        return self.moe_forward_routed(x, ids, g, base, y, out_dtype), ids, g, counts

    # ---- inspection ----
    def get_page_table(self):
        arr = (PageEntry * self.E)()
        _check(lib().pw_get_page_table(self._ctx, arr), self._ctx)
        return [dict(offset=int(e.offset), nbytes=int(e.nbytes), scale=float(e.scale),
                     bits=int(e.bits)) for e in arr]

    def get_loss_table(self, stream=None) -> np.ndarray:
        out = np.zeros(self.E * 3, dtype=np.float64)
        _check(lib().pw_get_loss_table(self._ctx, out.ctypes.data, _stream(stream)), self._ctx)
        return out.reshape(self.E, 3)

    def profile(self, mask):
        """Per-kernel timing: mask bits 0 router, 1 gate/up, 2 down, 3 combine
        (True = all, False/0 = off)."""
        m = 15 if mask is True else (0 if mask is False else int(mask))
        _check(lib().pw_profile(self._ctx, m), self._ctx)

    def profile_read(self) -> dict:
        d = ProfileData()
        _check(lib().pw_profile_read(self._ctx, ctypes.byref(d)), self._ctx)
        return dict(route_ms=d.route_ms, gate_up_ms=d.gate_up_ms, down_ms=d.down_ms,
                    combine_ms=d.combine_ms, forwards=d.forwards)

    # ---- convenience: caller-owned buffers allocated with torch ----
    def alloc_pool(self, nbytes: int, device="cuda") -> torch.Tensor:
        pool = torch.zeros(max(256, int(nbytes)), dtype=torch.uint8, device=device)
        self.bind_pool(pool)
        return pool

    def alloc_host_tier(self, nbytes: int) -> torch.Tensor:
        host = torch.zeros(max(256, int(nbytes)), dtype=torch.uint8, pin_memory=True)
        self.bind_host_tier(host)
        return host

    def alloc_workspace(self, device="cuda") -> torch.Tensor:
        ws = torch.empty(max(256, self.workspace_bytes()), dtype=torch.uint8, device=device)
        self.bind_workspace(ws)
        return ws
