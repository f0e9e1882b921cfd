"""Thin ctypes binding of libmoonep.so (include/moonep.h), same names as the C ABI.

Argument marshalling only: torch tensors give device pointers, torch's current
stream gives the HIP stream. Every computation runs in the library's HIP
kernels; there is no fallback, and a missing library raises at import of the
first call.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoonep.so")

TRAIN, INFER = 0, 1
BF16, FP32 = 0, 1
FWD, DGRAD, WGRAD = 0, 1, 2
SOFTMAX, SIGMOID = 0, 1
ERR_ID_RANGE, ERR_ID_DUP = 1, 2
OK, EINVAL, EWORKSPACE, EHIP, EMODE, ELIMIT = 0, -1, -2, -3, -4, -5

# every symbol the header declares
EXPORTS = (
    "moonep_version", "moonep_strerror", "moonep_validate_shape", "moonep_workspace_bytes",
    "moonep_workspace_init", "moonep_plan", "moonep_prefetch_weight", "moonep_dispatch",
    "moonep_grouped_gemm", "moonep_grouped_gemm_noalloc", "moonep_combine", "moonep_reduce_grad", "moonep_get_error",
    "moonep_swiglu", "moonep_grouped_gemm_swiglu", "moonep_swiglu_backward",
    "moonep_route", "moonep_route_backward", "moonep_gate_grad",
    "moonep_checkpoint_quantize", "moonep_checkpoint_dispatch", "moonep_swiglu_checkpoint",
    "moonep_grouped_gemm_swiglu_checkpoint", "moonep_swiglu_backward_checkpoint",
    "moonep_mx_quantize", "moonep_mx_quantize_weight", "moonep_mx_prefetch_weight",
    "moonep_mx_grouped_gemm",
    "moonep_vm_granularity", "moonep_pool_create", "moonep_pool_bytes", "moonep_pool_destroy",
    "moonep_view_create", "moonep_view_destroy",
)
SWIGLU_BLOCK = 32


class Shape(ctypes.Structure):
    """moonep_shape."""
    _fields_ = [(n, ctypes.c_int32) for n in ("R", "S", "E", "K", "B", "H", "Hp", "mode", "dtype")]

    @classmethod
    def of(cls, cfg) -> "Shape":
        """From a LayerConfig-like object (R, S, E, K, B, H, Hp, mode, dtype strings)."""
        return cls(cfg.R, cfg.S, cfg.E, cfg.K, cfg.B, cfg.H, cfg.Hp,
                   TRAIN if cfg.mode == "train" else INFER,
                   BF16 if cfg.dtype == "bf16" else FP32)


class Router(ctypes.Structure):
    """moonep_router."""
    _fields_ = [(n, ctypes.c_int32) for n in ("score", "dtype", "groups", "top_groups",
                                              "group_top", "renorm")] + [("scale", ctypes.c_float)]


class MoonepError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {status} ({strerror(status)})")
        self.status = status


_lib = None
_vp = ctypes.c_void_p
_sp = ctypes.POINTER(Shape)
_rp = ctypes.POINTER(Router)


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with "
                              "`python -m redundant_expert_balancing_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        sig = {
            "moonep_version": ([], ctypes.c_int),
            "moonep_strerror": ([ctypes.c_int], ctypes.c_char_p),
            "moonep_validate_shape": ([_sp], ctypes.c_int),
            "moonep_workspace_bytes": ([_sp], ctypes.c_size_t),
            "moonep_workspace_init": ([_sp, _vp, ctypes.c_size_t, _vp], ctypes.c_int),
            "moonep_plan": ([_sp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp], ctypes.c_int),
            "moonep_prefetch_weight": ([_sp, _vp, _vp, _vp], ctypes.c_int),
            "moonep_dispatch": ([_sp, ctypes.c_int32, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
            "moonep_grouped_gemm": ([_sp, ctypes.c_int32, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                     ctypes.c_size_t, _vp], ctypes.c_int),
            "moonep_grouped_gemm_noalloc": ([_sp, ctypes.c_int32, _vp, _vp, _vp, _vp, _vp, _vp,
                                             _vp], ctypes.c_int),
            "moonep_combine": ([_sp, ctypes.c_int32, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
            "moonep_reduce_grad": ([_sp, _vp, _vp, _vp, _vp], ctypes.c_int),
            "moonep_get_error": ([_sp, _vp, ctypes.c_size_t, ctypes.POINTER(ctypes.c_int32),
                                  ctypes.c_int32], ctypes.c_int),
            "moonep_swiglu": ([_sp, _vp, _vp, _vp, _vp], ctypes.c_int),
            "moonep_grouped_gemm_swiglu": ([_sp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                                            _vp], ctypes.c_int),
            "moonep_swiglu_backward": ([_sp, _vp, _vp, _vp, _vp], ctypes.c_int),
            "moonep_route": ([_sp, _rp, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
            "moonep_route_backward": ([_sp, _rp] + [_vp] * 7, ctypes.c_int),
            "moonep_gate_grad": ([_sp, ctypes.c_int32, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
            "moonep_checkpoint_quantize": ([_sp, ctypes.c_int32, _vp, _vp, _vp, _vp], ctypes.c_int),
            "moonep_checkpoint_dispatch": ([_sp, ctypes.c_int32, _vp, _vp, _vp, _vp, _vp],
                                           ctypes.c_int),
            "moonep_swiglu_checkpoint": ([_sp, _vp, _vp, _vp, _vp, _vp], ctypes.c_int),
            "moonep_grouped_gemm_swiglu_checkpoint": ([_sp] + [_vp] * 7 + [ctypes.c_size_t, _vp],
                                                      ctypes.c_int),
            "moonep_swiglu_backward_checkpoint": ([_sp] + [_vp] * 9, ctypes.c_int),
            "moonep_mx_quantize": ([_sp, ctypes.c_int64, ctypes.c_int32, _vp, _vp, _vp, _vp],
                                   ctypes.c_int),
            "moonep_mx_quantize_weight": ([_sp, _vp, _vp, _vp, _vp], ctypes.c_int),
            "moonep_mx_prefetch_weight": ([_sp, _vp, _vp, _vp, _vp], ctypes.c_int),
            "moonep_mx_grouped_gemm": ([_sp] + [_vp] * 8 + [ctypes.c_size_t, _vp], ctypes.c_int),
            "moonep_vm_granularity": ([], ctypes.c_size_t),
            "moonep_pool_create": ([_sp, ctypes.c_int32, ctypes.POINTER(_vp)], ctypes.c_int),
            "moonep_pool_bytes": ([_vp], ctypes.c_size_t),
            "moonep_pool_destroy": ([_vp], ctypes.c_int),
            "moonep_view_create": ([_sp, _vp, ctypes.c_int32, ctypes.POINTER(_vp),
                                    ctypes.POINTER(_vp)], ctypes.c_int),
            "moonep_view_destroy": ([_vp], ctypes.c_int),
        }
        for name, (args, res) in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def strerror(status: int) -> str:
    return lib().moonep_strerror(status).decode()


def _p(t, nbytes: int = 0, name: str = "buffer", dtype=None):
    """Device pointer of a tensor (None -> NULL). The tensor must be a contiguous GPU
    tensor of at least `nbytes` bytes (and of `dtype`, if given): anything else raises
    here, before a kernel could read or write past it."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name}: a GPU tensor is required, got one on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: the tensor must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{name}: {have} bytes, the call needs at least {nbytes}")
    return _vp(t.data_ptr())


def _dims(shape: Shape):
    """(elements per token row N, slots N*K, slots per rank SK, bytes per element)."""
    N = shape.R * shape.S
    return N, N * shape.K, shape.S * shape.K, 2 if shape.dtype == BF16 else 4


def _i32():
    import torch
    return torch.int32


def _f32():
    import torch
    return torch.float32


def _act(shape: Shape):
    """torch dtype of the layer's activations and weights."""
    import torch
    return torch.bfloat16 if shape.dtype == BF16 else torch.float32


def _s(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return _vp(getattr(stream, "cuda_stream", stream))


def _check(fn: str, st: int) -> int:
    if st != OK:
        raise MoonepError(fn, st)
    return st


def _nbytes(t) -> int:
    return t.numel() * t.element_size()


def moonep_version() -> int:
    return lib().moonep_version()


def moonep_validate_shape(shape: Shape) -> int:
    return lib().moonep_validate_shape(ctypes.byref(shape))


def moonep_workspace_bytes(shape: Shape) -> int:
    return lib().moonep_workspace_bytes(ctypes.byref(shape))


def moonep_workspace_init(shape, ws, stream=None):
    _check("moonep_workspace_init", lib().moonep_workspace_init(
        ctypes.byref(shape), _p(ws, moonep_workspace_bytes(shape), "ws"), _nbytes(ws), _s(stream)))


def moonep_plan(shape, topk_idx, cu_seqlens, replica_expert, slot_map, src_index, ws, stream=None):
    N, NK, _, _ = _dims(shape)
    i32, R, B = _i32(), shape.R, shape.B
    _check("moonep_plan", lib().moonep_plan(
        ctypes.byref(shape), _p(topk_idx, 4 * NK, "topk_idx", i32),
        _p(cu_seqlens, 4 * R * (shape.E + B + 1), "cu_seqlens", i32),
        _p(replica_expert, 4 * R * B, "replica_expert", i32),
        _p(slot_map, 4 * NK, "slot_map", i32), _p(src_index, 4 * NK, "src_index", i32),
        _p(ws, moonep_workspace_bytes(shape), "ws"), _nbytes(ws), _s(stream)))


def _w_all_bytes(shape: Shape) -> int:
    return (shape.E + shape.R * shape.B) * shape.H * shape.Hp * _dims(shape)[3]


def moonep_prefetch_weight(shape, replica_expert, w_all, stream=None):
    _check("moonep_prefetch_weight", lib().moonep_prefetch_weight(
        ctypes.byref(shape), _p(replica_expert, 4 * shape.R * shape.B, "replica_expert", _i32()),
        _p(w_all, _w_all_bytes(shape), "w_all", _act(shape)), _s(stream)))


def moonep_dispatch(shape, width, src, slot_map, gates, dst, stream=None):
    N, NK, _, eb = _dims(shape)
    w = int(width)
    _check("moonep_dispatch", lib().moonep_dispatch(
        ctypes.byref(shape), w, _p(src, N * w * eb, "src", _act(shape)),
        _p(slot_map, 4 * NK, "slot_map", _i32()), _p(gates, 4 * NK, "gates", _f32()),
        _p(dst, NK * w * eb, "dst", _act(shape)), _s(stream)))


def _gemm_operands(shape, op, a, b, c, grad_home, reduce_buf):
    _, NK, _, eb = _dims(shape)
    H, Hp, act = shape.H, shape.Hp, _act(shape)
    wsz = 4 * H * Hp
    if int(op) == FWD:
        args = (_p(a, NK * H * eb, "a (xp)", act), _p(b, _w_all_bytes(shape), "b (w_all)", act),
                _p(c, 4 * NK * Hp, "c (out)", _f32()), None, None)
    elif int(op) == DGRAD:
        args = (_p(a, NK * Hp * eb, "a (dyp)", act), _p(b, _w_all_bytes(shape), "b (w_all)", act),
                _p(c, 4 * NK * H, "c (dxp)", _f32()), None, None)
    elif int(op) == WGRAD:
        args = (_p(a, NK * H * eb, "a (xp)", act), _p(b, NK * Hp * eb, "b (dyp)", act), None,
                _p(grad_home, shape.E * wsz, "grad_home", _f32()),
                _p(reduce_buf, shape.R * shape.B * wsz, "reduce_buf", _f32()))
    else:
        args = (_p(a), _p(b), _p(c), _p(grad_home), _p(reduce_buf))   # the library refuses op
    return args


def moonep_grouped_gemm(shape, op, a, b, cu_seqlens, c, grad_home, reduce_buf, ws, stream=None):
    args = _gemm_operands(shape, op, a, b, c, grad_home, reduce_buf)
    _check("moonep_grouped_gemm", lib().moonep_grouped_gemm(
        ctypes.byref(shape), int(op), args[0], args[1],
        _p(cu_seqlens, 4 * shape.R * (shape.E + shape.B + 1), "cu_seqlens", _i32()),
        args[2], args[3], args[4], _p(ws, moonep_workspace_bytes(shape), "ws"), _nbytes(ws),
        _s(stream)))


def moonep_grouped_gemm_noalloc(shape, op, a, b, cu_seqlens, c, grad_home, reduce_buf,
                                stream=None):
    args = _gemm_operands(shape, op, a, b, c, grad_home, reduce_buf)
    _check("moonep_grouped_gemm_noalloc", lib().moonep_grouped_gemm_noalloc(
        ctypes.byref(shape), int(op), args[0], args[1],
        _p(cu_seqlens, 4 * shape.R * (shape.E + shape.B + 1), "cu_seqlens", _i32()),
        args[2], args[3], args[4], _s(stream)))


def moonep_combine(shape, width, src, slot_map, gates, dst, stream=None):
    N, NK, _, _ = _dims(shape)
    w = int(width)
    _check("moonep_combine", lib().moonep_combine(
        ctypes.byref(shape), w, _p(src, 4 * NK * w, "src", _f32()),
        _p(slot_map, 4 * NK, "slot_map", _i32()), _p(gates, 4 * NK, "gates", _f32()),
        _p(dst, 4 * N * w, "dst", _f32()), _s(stream)))


def moonep_reduce_grad(shape, replica_expert, reduce_buf, grad_home, stream=None):
    wsz = 4 * shape.H * shape.Hp
    _check("moonep_reduce_grad", lib().moonep_reduce_grad(
        ctypes.byref(shape), _p(replica_expert, 4 * shape.R * shape.B, "replica_expert", _i32()),
        _p(reduce_buf, shape.R * shape.B * wsz, "reduce_buf", _f32()),
        _p(grad_home, shape.E * wsz, "grad_home", _f32()), _s(stream)))


def moonep_swiglu(shape, h, act, h_saved=None, stream=None):
    _, NK, _, eb = _dims(shape)
    Hp = shape.Hp
    _check("moonep_swiglu", lib().moonep_swiglu(
        ctypes.byref(shape), _p(h, 4 * NK * 2 * Hp, "h", _f32()),
        _p(act, NK * Hp * eb, "act", _act(shape)),
        _p(h_saved, NK * 2 * Hp * eb, "h_saved", _act(shape)), _s(stream)))


def moonep_grouped_gemm_swiglu(shape, xp, w1_all, cu_seqlens, act, h_saved, ws, stream=None):
    _, NK, _, eb = _dims(shape)
    H, Hp, a = shape.H, shape.Hp, _act(shape)
    _check("moonep_grouped_gemm_swiglu", lib().moonep_grouped_gemm_swiglu(
        ctypes.byref(shape), _p(xp, NK * H * eb, "xp", a),
        _p(w1_all, (shape.E + shape.R * shape.B) * H * 2 * Hp * eb, "w1_all", a),
        _p(cu_seqlens, 4 * shape.R * (shape.E + shape.B + 1), "cu_seqlens", _i32()),
        _p(act, NK * Hp * eb, "act", a), _p(h_saved, NK * 2 * Hp * eb, "h_saved", a),
        _p(ws, moonep_workspace_bytes(shape), "ws"), _nbytes(ws), _s(stream)))


def moonep_swiglu_backward(shape, h_saved, da, dh, stream=None):
    _, NK, _, eb = _dims(shape)
    Hp, a = shape.Hp, _act(shape)
    _check("moonep_swiglu_backward", lib().moonep_swiglu_backward(
        ctypes.byref(shape), _p(h_saved, NK * 2 * Hp * eb, "h_saved", a),
        _p(da, 4 * NK * Hp, "da", _f32()), _p(dh, NK * 2 * Hp * eb, "dh", a), _s(stream)))


# ---- router, gates' gradient, 8-bit checkpoints, 4-bit experts
#
# These calls serve single tokens too, so the checks of _p are made in one expression per
# tensor and the stream is asked for as a handle (a whole call's marshalling: 4-6 us).
_torch = None


def _device() -> int:
    """Index of the current device."""
    global _torch
    if _torch is None:
        import torch
        _torch = torch
    if _torch.cuda.is_initialized():
        return _torch._C._cuda_getDevice()
    return _torch.cuda.current_device() if _torch.cuda.is_available() else -2


def _q(t, nbytes, name, dtype, dev, optional=False):
    """Address of a contiguous tensor of `dtype` (None: any) with at least `nbytes` bytes on
    device `dev` (the current one, whose stream the call goes to); raises otherwise."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name}: a tensor is required")
    if (t.get_device() == dev and (dtype is None or t.dtype is dtype) and t.is_contiguous()
            and t.nbytes >= nbytes):
        return t.data_ptr()
    _p(t, nbytes, name, dtype)
    raise ValueError(f"{name}: on {t.device}, the current device is cuda:{dev}")


def _h(stream, dev):
    """hipStream_t of `stream` (None: torch's current one on `dev`)."""
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(dev) if dev >= 0 else None
    return getattr(stream, "cuda_stream", stream)


def _logit(router: Router):
    return (_torch.bfloat16, 2) if router.dtype == BF16 else (_torch.float32, 4)


def _types(shape: Shape):
    """(activation type, its bytes) of the layer."""
    return (_torch.bfloat16, 2) if shape.dtype == BF16 else (_torch.float32, 4)


def moonep_route(shape, router, logits, bias, topk_idx, gates, stream=None):
    d = _device()
    N, E = shape.R * shape.S, shape.E
    b = 4 * N * shape.K
    dt, lb = _logit(router)
    f32 = _torch.float32
    st = lib().moonep_route(
        shape, router, _q(logits, N * E * lb, "logits", dt, d), _q(bias, 4 * E, "bias", f32, d, True),
        _q(topk_idx, b, "topk_idx", _torch.int32, d), _q(gates, b, "gates", f32, d), _h(stream, d))
    if st:
        raise MoonepError("moonep_route", st)


def moonep_route_backward(shape, router, logits, bias, topk_idx, gates, dgates, dlogits,
                          stream=None):
    d = _device()
    N, E = shape.R * shape.S, shape.E
    b = 4 * N * shape.K
    dt, lb = _logit(router)
    f32 = _torch.float32
    st = lib().moonep_route_backward(
        shape, router, _q(logits, N * E * lb, "logits", dt, d), _q(bias, 4 * E, "bias", f32, d, True),
        _q(topk_idx, b, "topk_idx", _torch.int32, d), _q(gates, b, "gates", f32, d),
        _q(dgates, b, "dgates", f32, d), _q(dlogits, N * E * lb, "dlogits", dt, d), _h(stream, d))
    if st:
        raise MoonepError("moonep_route_backward", st)


def moonep_gate_grad(shape, width, src, slot_map, dy, dgates, stream=None):
    d = _device()
    N, w = shape.R * shape.S, int(width)
    NK = N * shape.K
    act, eb = _types(shape)
    f32 = _torch.float32
    st = lib().moonep_gate_grad(
        shape, w, _q(src, 4 * NK * w, "src", f32, d), _q(slot_map, 4 * NK, "slot_map", _torch.int32, d),
        _q(dy, N * w * eb, "dy", act, d), _q(dgates, 4 * NK, "dgates", f32, d), _h(stream, d))
    if st:
        raise MoonepError("moonep_gate_grad", st)


def checkpoint_scale_bytes(width: int) -> int:
    """Bytes of a checkpoint row's scales."""
    return 4 * -(-width // 128)


def moonep_checkpoint_quantize(shape, width, src, q, scales, stream=None):
    d = _device()
    N, w = shape.R * shape.S, int(width)
    act, eb = _types(shape)
    u8 = _torch.uint8
    st = lib().moonep_checkpoint_quantize(
        shape, w, _q(src, N * w * eb, "src", act, d), _q(q, N * w, "q", u8, d),
        _q(scales, N * checkpoint_scale_bytes(w), "scales", u8, d), _h(stream, d))
    if st:
        raise MoonepError("moonep_checkpoint_quantize", st)


def moonep_checkpoint_dispatch(shape, width, q, scales, slot_map, dst, stream=None):
    d = _device()
    N, w = shape.R * shape.S, int(width)
    NK = N * shape.K
    act, eb = _types(shape)
    u8 = _torch.uint8
    st = lib().moonep_checkpoint_dispatch(
        shape, w, _q(q, N * w, "q", u8, d), _q(scales, N * checkpoint_scale_bytes(w), "scales", u8, d),
        _q(slot_map, 4 * NK, "slot_map", _torch.int32, d), _q(dst, NK * w * eb, "dst", act, d),
        _h(stream, d))
    if st:
        raise MoonepError("moonep_checkpoint_dispatch", st)


def _checkpoint_h(shape, q, scales, d):
    NK, w = shape.R * shape.S * shape.K, 2 * shape.Hp
    return (_q(q, NK * w, "q", _torch.uint8, d),
            _q(scales, NK * checkpoint_scale_bytes(w), "scales", _torch.uint8, d))


def moonep_swiglu_checkpoint(shape, h, act, q, scales, stream=None):
    d = _device()
    n = shape.R * shape.S * shape.K * shape.Hp
    at, eb = _types(shape)
    st = lib().moonep_swiglu_checkpoint(
        shape, _q(h, 8 * n, "h", _torch.float32, d), _q(act, n * eb, "act", at, d),
        *_checkpoint_h(shape, q, scales, d), _h(stream, d))
    if st:
        raise MoonepError("moonep_swiglu_checkpoint", st)


def _ws(ws, d):
    """(address, bytes) of a workspace, whose size the library checks."""
    return _q(ws, 0, "ws", None, d), ws.nbytes


def moonep_grouped_gemm_swiglu_checkpoint(shape, xp, w1_all, cu_seqlens, act, q, scales, ws,
                                          stream=None):
    d = _device()
    NK, H, Hp = shape.R * shape.S * shape.K, shape.H, shape.Hp
    at, eb = _types(shape)
    st = lib().moonep_grouped_gemm_swiglu_checkpoint(
        shape, _q(xp, NK * H * eb, "xp", at, d),
        _q(w1_all, (shape.E + shape.R * shape.B) * H * 2 * Hp * eb, "w1_all", at, d),
        _q(cu_seqlens, 4 * shape.R * (shape.E + shape.B + 1), "cu_seqlens", _torch.int32, d),
        _q(act, NK * Hp * eb, "act", at, d), *_checkpoint_h(shape, q, scales, d),
        *_ws(ws, d), _h(stream, d))
    if st:
        raise MoonepError("moonep_grouped_gemm_swiglu_checkpoint", st)


def moonep_swiglu_backward_checkpoint(shape, q, scales, da, src_index, gates, act, dh, dgates,
                                      stream=None):
    d = _device()
    NK, Hp = shape.R * shape.S * shape.K, shape.Hp
    at, eb = _types(shape)
    f32 = _torch.float32
    st = lib().moonep_swiglu_backward_checkpoint(
        shape, *_checkpoint_h(shape, q, scales, d), _q(da, 4 * NK * Hp, "da", f32, d),
        _q(src_index, 4 * NK, "src_index", _torch.int32, d, True),
        _q(gates, 4 * NK, "gates", f32, d, True), _q(act, NK * Hp * eb, "act", at, d),
        _q(dh, NK * 2 * Hp * eb, "dh", at, d), _q(dgates, 4 * NK, "dgates", f32, d, True),
        _h(stream, d))
    if st:
        raise MoonepError("moonep_swiglu_backward_checkpoint", st)


def mx_row_bytes(width: int):
    """Bytes of one token row's values and of its scales."""
    return 64 * -(-width // 128), 16 * -(-width // 512)


def mx_weight_bytes(H: int, Hp: int):
    """Bytes of one expert's values and of its scales."""
    q, s = mx_row_bytes(H)
    return Hp * q, Hp * s


def moonep_mx_quantize(shape, rows, width, src, q, scales, stream=None):
    d = _device()
    rows, w = int(rows), int(width)
    act, eb = _types(shape)
    qb, sb = mx_row_bytes(w)
    st = lib().moonep_mx_quantize(
        shape, rows, w, _q(src, rows * w * eb, "src", act, d), _q(q, rows * qb, "q", _torch.uint8, d),
        _q(scales, rows * sb, "scales", _torch.uint8, d), _h(stream, d))
    if st:
        raise MoonepError("moonep_mx_quantize", st)


def moonep_mx_quantize_weight(shape, w, wq, wscales, stream=None):
    d = _device()
    E = shape.E
    act, eb = _types(shape)
    qb, sb = mx_weight_bytes(shape.H, shape.Hp)
    st = lib().moonep_mx_quantize_weight(
        shape, _q(w, E * shape.H * shape.Hp * eb, "w", act, d), _q(wq, E * qb, "wq", _torch.uint8, d),
        _q(wscales, E * sb, "wscales", _torch.uint8, d), _h(stream, d))
    if st:
        raise MoonepError("moonep_mx_quantize_weight", st)


def _mx_weights(shape, wq, wscales, d):
    rows = shape.E + shape.R * shape.B
    qb, sb = mx_weight_bytes(shape.H, shape.Hp)
    return (_q(wq, rows * qb, "wq", _torch.uint8, d),
            _q(wscales, rows * sb, "wscales", _torch.uint8, d))


def moonep_mx_prefetch_weight(shape, replica_expert, wq, wscales, stream=None):
    d = _device()
    st = lib().moonep_mx_prefetch_weight(
        shape, _q(replica_expert, 4 * shape.R * shape.B, "replica_expert", _torch.int32, d),
        *_mx_weights(shape, wq, wscales, d), _h(stream, d))
    if st:
        raise MoonepError("moonep_mx_prefetch_weight", st)


def moonep_mx_grouped_gemm(shape, xq, xscales, src_index, wq, wscales, cu_seqlens, c, ws,
                           stream=None):
    d = _device()
    N = shape.R * shape.S
    NK = N * shape.K
    rows = NK if src_index is None else N
    qb, sb = mx_row_bytes(shape.H)
    i32, u8 = _torch.int32, _torch.uint8
    st = lib().moonep_mx_grouped_gemm(
        shape, _q(xq, rows * qb, "xq", u8, d), _q(xscales, rows * sb, "xscales", u8, d),
        _q(src_index, 4 * NK, "src_index", i32, d, True), *_mx_weights(shape, wq, wscales, d),
        _q(cu_seqlens, 4 * shape.R * (shape.E + shape.B + 1), "cu_seqlens", i32, d),
        _q(c, 4 * NK * shape.Hp, "c", _torch.float32, d), *_ws(ws, d), _h(stream, d))
    if st:
        raise MoonepError("moonep_mx_grouped_gemm", st)


def moonep_vm_granularity() -> int:
    return lib().moonep_vm_granularity()


def moonep_pool_create(shape, nsets: int) -> int:
    """Opaque pool handle (an int address)."""
    h = _vp()
    _check("moonep_pool_create", lib().moonep_pool_create(ctypes.byref(shape), int(nsets),
                                                          ctypes.byref(h)))
    return h.value


def moonep_pool_bytes(pool) -> int:
    return lib().moonep_pool_bytes(_vp(pool))


def moonep_pool_destroy(pool):
    _check("moonep_pool_destroy", lib().moonep_pool_destroy(_vp(pool)))


def moonep_view_create(shape, pool, set_index: int):
    """(view handle, device address of the [E+R*B, H, Hp] view)."""
    v, w = _vp(), _vp()
    _check("moonep_view_create", lib().moonep_view_create(
        ctypes.byref(shape), _vp(pool), int(set_index), ctypes.byref(v), ctypes.byref(w)))
    return v.value, w.value


def moonep_view_destroy(view):
    _check("moonep_view_destroy", lib().moonep_view_destroy(_vp(view)))


def moonep_get_error(shape, ws, clear: bool = False) -> int:
    flags = ctypes.c_int32(0)
    _check("moonep_get_error", lib().moonep_get_error(
        ctypes.byref(shape), _p(ws, moonep_workspace_bytes(shape), "ws"), _nbytes(ws),
        ctypes.byref(flags), int(clear)))
    return flags.value
