"""Python binding of the KDA C ABI (include/kda.h), by ctypes.

Argument marshalling only: every function forwards to the entry point of the
same name in libkda.so; all arithmetic runs in the CUDA kernels behind it.
Device tensors are torch tensors (used for device memory and streams only).
There is no fallback: if libkda.so is missing or the call fails, an exception
is raised.
"""
from __future__ import annotations

import ctypes
import os
import struct
from array import array

import numpy as np
import torch

KDA_OK, KDA_ERR_INVALID, KDA_ERR_OOM, KDA_ERR_CUDA, KDA_ERR_BLOB, KDA_ERR_TIMEOUT, KDA_ERR_DEVICE, KDA_ERR_IO = range(8)
KDA_F32, KDA_BF16 = 0, 1
KDA_BLOB_MAGIC = 0x3141444B
KDA_BLOB_VERSION = 1
KDA_DECODE_MAX_TOKENS = 8  # most tokens per row in one kda_decode_tokens call
STATUS_NAMES = {0: "KDA_OK", 1: "KDA_ERR_INVALID", 2: "KDA_ERR_OOM", 3: "KDA_ERR_CUDA",
                4: "KDA_ERR_BLOB", 5: "KDA_ERR_TIMEOUT", 6: "KDA_ERR_DEVICE",
                7: "KDA_ERR_IO"}

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libkda.so")


class KdaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status
        self.message = message


class kda_config_t(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("conv_kernel", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("chunk_size", ctypes.c_int32),
                ("gate_lower_bound", ctypes.c_float), ("l2_eps", ctypes.c_float),
                ("rms_eps", ctypes.c_float), ("q_scale", ctypes.c_float)]


class kda_layer_params(ctypes.Structure):
    _fields_ = [("conv_w", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p),
                ("A_log", ctypes.c_void_p), ("norm_w", ctypes.c_void_p)]


class kda_gdr_config_t(ctypes.Structure):
    _fields_ = [("num_heads", ctypes.c_int32), ("num_qk_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("io_dtype", ctypes.c_int32), ("qk_l2norm", ctypes.c_int32), ("l2_eps", ctypes.c_float),
                ("q_scale", ctypes.c_float)]


class kda_gdr_params(ctypes.Structure):
    _fields_ = [("A_log", ctypes.c_void_p), ("dt_bias", ctypes.c_void_p)]
    heads, device = 0, None  # set by kda_gdr_params_from; without them a call refuses the parameters


class kda_gdr_rows(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("q", "k", "v", "a", "b", "out")] + \
        [(n + "_stride", ctypes.c_int64) for n in ("q", "k", "v", "a", "b", "out")]


class kda_glr_config_t(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("io_dtype", ctypes.c_int32)]


class kda_glr_params(ctypes.Structure):
    _fields_ = [("A_log", ctypes.c_void_p), ("a_bias", ctypes.c_void_p), ("b_bias", ctypes.c_void_p)]
    dim, device = 0, None  # set by kda_glr_params_from; without them a call refuses the parameters


_GLR_ROWS, _GLR_GRADS = ("x", "a", "b", "g", "out"), ("x", "a", "b", "g", "dout", "dx", "da", "db", "dg")


_PACK_GLR_ROWS, _PACK_GLR_GRADS = struct.Struct("5P5q").pack, struct.Struct("9P9q").pack


class kda_glr_rows(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _GLR_ROWS] + [(n + "_stride", ctypes.c_int64) for n in _GLR_ROWS]


class kda_glr_grad_rows(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _GLR_GRADS] + [(n + "_stride", ctypes.c_int64) for n in _GLR_GRADS]


class kda_block_norm_config_t(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("io_dtype", ctypes.c_int32), ("eps", ctypes.c_float)]


class kda_block_norm_params(ctypes.Structure):
    _fields_ = [("post_w", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("pre_w", ctypes.c_void_p)]
    dim, device = 0, None  # set by kda_block_norm_params_from; without them a call refuses the parameters


class kda_block_norm_rows(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("x", "y", "g", "x_out", "h", "hs")] + \
        [(n + "_stride", ctypes.c_int64) for n in ("x", "y", "g", "x_out", "h")]


_NORM_ROWS = ("x", "y", "g", "x_out", "h")
_PACK_NORM_ROWS, _PACK_NORM_GRADS = struct.Struct("6P5q").pack, struct.Struct("8P8q").pack
_PACK_NORM_ROWS5 = struct.Struct("5P8x5q").pack  # without hs
_NORM_GRADS = ("x_out", "dh", "dx1", "y", "g", "dx", "dy", "dg")


class kda_block_norm_grad_rows(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in _NORM_GRADS] + [(n + "_stride", ctypes.c_int64) for n in _NORM_GRADS]


class kda_blob_header(ctypes.Structure):
    _fields_ = [("magic", ctypes.c_uint32), ("version", ctypes.c_uint32),
                ("num_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("conv_kernel", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
                ("n_slots", ctypes.c_int32), ("reserved0", ctypes.c_int32),
                ("state_bytes_per_slot", ctypes.c_uint64), ("tail_bytes_per_slot", ctypes.c_uint64),
                ("reserved", ctypes.c_uint8 * 16)]


_VP = ctypes.c_void_p
_I32 = ctypes.c_int32
_PI32 = ctypes.POINTER(ctypes.c_int32)
_lib = None

# (name, restype, argtypes) for every entry point of include/kda.h
SIGNATURES = [
    ("kda_config", _I32, [ctypes.POINTER(kda_config_t), _I32, _I32, _I32]),
    ("kda_state_alloc", _I32, [ctypes.POINTER(kda_config_t), _I32, ctypes.POINTER(_VP)]),
    ("kda_state_free", _I32, [_VP]),
    ("kda_state_reset", _I32, [_VP, _PI32, _I32, _VP]),
    ("kda_state_max_slots", _I32, [_VP]),
    ("kda_state_blob_bytes", ctypes.c_size_t, [_VP, _I32]),
    ("kda_state_snapshot", _I32, [_VP, _PI32, _I32, _VP, _I32, _VP]),
    ("kda_state_restore", _I32, [_VP, _PI32, _I32, _VP, _I32, _VP]),
    ("kda_decode_token", _I32, [ctypes.POINTER(kda_config_t), ctypes.POINTER(kda_layer_params), _VP, _VP, _I32,
                                _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    ("kda_decode_tokens", _I32, [ctypes.POINTER(kda_config_t), ctypes.POINTER(kda_layer_params), _VP, _VP, _I32,
                                 _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    ("kda_prefill", _I32, [ctypes.POINTER(kda_config_t), ctypes.POINTER(kda_layer_params), _VP, _VP, _VP, _PI32,
                           _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    ("kda_prefill_noalloc", _I32, [ctypes.POINTER(kda_config_t), ctypes.POINTER(kda_layer_params), _VP, _VP, _I32,
                                   _VP, _VP, _VP, _PI32, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    ("kda_state_poll_error", _I32, [_VP, _PI32]),
    ("kda_gate_proj_workspace_bytes", ctypes.c_size_t, [ctypes.POINTER(kda_config_t), _I32, ctypes.c_int64]),
    ("kda_gate_proj", _I32, [ctypes.POINTER(kda_config_t), _I32, ctypes.c_int64, _VP, _VP, _VP, _VP, _VP, _VP,
                             _VP, ctypes.c_size_t, _VP]),
    ("kda_gate_proj_in", _I32, [ctypes.POINTER(kda_config_t), _I32, ctypes.c_int64, _VP, _VP, _VP, _VP, _VP, _VP,
                                ctypes.c_size_t, _VP]),
    ("kda_prefill_gate_fused", _I32, [ctypes.POINTER(kda_config_t), ctypes.POINTER(kda_layer_params), _VP, _VP, _VP,
                                      _PI32, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP]),
    ("kda_linear_workspace_bytes", ctypes.c_size_t, [_I32, _I32, _I32]),
    ("kda_linear", _I32, [_I32, _I32, _I32, _VP, _VP, _VP, _VP, _I32, _VP, ctypes.c_size_t, _VP]),
    ("kda_quant_fp8", _I32, [ctypes.c_int64, _I32, _VP, ctypes.c_int64, _I32, _I32, _VP, _VP, _VP]),
    ("kda_linear_fp8_workspace_bytes", ctypes.c_size_t, [_I32, _I32, _I32]),
    ("kda_linear_fp8", _I32, [_I32, _I32, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _VP, ctypes.c_size_t, _VP]),
    ("kda_gdr_config", _I32, [ctypes.POINTER(kda_gdr_config_t), _I32, _I32, _I32, _I32]),
    ("kda_gdr_decode", _I32, [ctypes.POINTER(kda_gdr_config_t), ctypes.POINTER(kda_gdr_params), _VP, _I32, _VP, _VP,
                              _I32, _I32, ctypes.POINTER(kda_gdr_rows), _VP, _VP]),
    ("kda_gdr_workspace_bytes", ctypes.c_size_t, [ctypes.POINTER(kda_gdr_config_t), _PI32, _I32]),
    ("kda_gdr_prefill", _I32, [ctypes.POINTER(kda_gdr_config_t), ctypes.POINTER(kda_gdr_params), _VP, _I32, _VP, _VP,
                               _VP, _VP, _I32, ctypes.POINTER(kda_gdr_rows), _VP, ctypes.c_size_t, _VP, _VP]),
    ("kda_glr_config", _I32, [ctypes.POINTER(kda_glr_config_t), _I32, _I32]),
    ("kda_glr_decode", _I32, [ctypes.POINTER(kda_glr_config_t), ctypes.POINTER(kda_glr_params), _VP, _I32, _VP, _VP, _I32, _I32,
                              _VP, _VP, _VP]),
    ("kda_glr_workspace_bytes", ctypes.c_size_t, [ctypes.POINTER(kda_glr_config_t), _PI32, _I32]),
    ("kda_glr_chunks", ctypes.c_int64, [_VP, _I32]),
    ("kda_glr_prefill", _I32, [ctypes.POINTER(kda_glr_config_t), ctypes.POINTER(kda_glr_params), _VP, _I32, _VP, _VP, _VP, _VP, _I32,
                               _VP, _VP, _VP, ctypes.c_size_t, _VP, _VP]),
    ("kda_glr_backward", _I32, [ctypes.POINTER(kda_glr_config_t), ctypes.POINTER(kda_glr_params), _VP, _VP, _I32, _VP,
                                _VP, _VP, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP, _VP]),
    ("kda_block_norm_config", _I32, [ctypes.POINTER(kda_block_norm_config_t), _I32, _I32]),
    ("kda_block_norm", _I32, [ctypes.POINTER(kda_block_norm_config_t), ctypes.POINTER(kda_block_norm_params), ctypes.c_int64,
                              _VP, _VP]),
    ("kda_block_norm_workspace_bytes", ctypes.c_size_t, [ctypes.POINTER(kda_block_norm_config_t), ctypes.c_int64]),
    ("kda_block_norm_backward", _I32, [ctypes.POINTER(kda_block_norm_config_t), ctypes.POINTER(kda_block_norm_params), ctypes.c_int64,
                                       _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
    ("kda_photo_store_create", _I32, [_I32, ctypes.c_char_p, ctypes.POINTER(_VP)]),
    ("kda_photo_store_free", _I32, [_VP]),
    ("kda_photo_count", _I32, [_VP]),
    ("kda_photo_capacity", _I32, [_VP]),
    ("kda_photo_take", _I32, [_VP, ctypes.POINTER(_VP), _I32, _I32, _PI32, ctypes.c_int64, _PI32, _VP]),
    ("kda_photo_find", _I32, [_VP, _PI32, ctypes.c_int64, _PI32, ctypes.POINTER(ctypes.c_int64)]),
    ("kda_photo_restore", _I32, [_VP, _I32, ctypes.POINTER(_VP), _I32, _I32, _VP]),
    ("kda_last_error", ctypes.c_char_p, []),
]


def lib() -> ctypes.CDLL:
    """Load libkda.so from the package directory (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"the KDA CUDA library is not built ({LIB_PATH} missing); "
                               "run linear_attention_mixer_gb300.build.build()")
        L = ctypes.CDLL(LIB_PATH)
        for name, res, args in SIGNATURES:
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def kda_last_error() -> str:
    return lib().kda_last_error().decode()


def _check(status: int):
    if status != KDA_OK:
        raise KdaError(status, kda_last_error())


def _stream(stream):
    if stream is None:
        return _VP(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return _VP(stream.cuda_stream)
    return _VP(int(stream))


# A call's host time is most of what a small one costs, so the entry points from here on ask torch's C layer
# for the current device and stream.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)


def _raw_stream(stream, device: int) -> int:
    if stream is None:
        return _current_raw_stream(device)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _torch_io_dtype(cfg: kda_config_t):
    return torch.bfloat16 if cfg.io_dtype == KDA_BF16 else torch.float32


def _dev(t: torch.Tensor, dtype=None, name: str = "tensor"):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return _VP(t.data_ptr())


def _i32_array(x) -> np.ndarray:
    """x as a contiguous int32 array; refused where that would change a number."""
    if isinstance(x, (list, tuple)):
        try:
            return np.frombuffer(array("i", x), dtype=np.int32) if x else np.zeros(0, np.int32)
        except OverflowError:
            raise ValueError("slots and lengths must be 32-bit whole numbers") from None
        except TypeError:  # other numbers than Python's own
            pass
    a = np.asarray(x)
    if a.dtype != np.int32:
        with np.errstate(invalid="ignore"):
            b = a.astype(np.int32)
        if (a != b).any():
            raise ValueError("slots and lengths must be 32-bit whole numbers")
        a = b
    return np.ascontiguousarray(a)


def _host_i32(x):
    a = _i32_array(x)
    return a, a.ctypes.data_as(_PI32)


# ---------------------------------------------------------------- entry points

def kda_config(num_heads: int, head_dim: int = 128, io_dtype: int = KDA_BF16) -> kda_config_t:
    cfg = kda_config_t()
    _check(lib().kda_config(ctypes.byref(cfg), num_heads, head_dim, io_dtype))
    return cfg


def kda_state_alloc(cfg: kda_config_t, max_slots: int) -> ctypes.c_void_p:
    h = _VP()
    _check(lib().kda_state_alloc(ctypes.byref(cfg), max_slots, ctypes.byref(h)))
    return h


def kda_state_free(st) -> None:
    _check(lib().kda_state_free(st))


def kda_state_max_slots(st) -> int:
    return int(lib().kda_state_max_slots(st))


def kda_state_blob_bytes(st, n_slots: int) -> int:
    return int(lib().kda_state_blob_bytes(st, n_slots))


def kda_state_reset(st, slots, stream=None) -> None:
    arr, p = _host_i32(slots)
    _check(lib().kda_state_reset(st, p, len(arr), _stream(stream)))


def _buf(t: torch.Tensor, need: int, name: str):
    if not isinstance(t, torch.Tensor) or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous torch tensor")
    if t.numel() * t.element_size() < need:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, {need} needed")
    return _VP(t.data_ptr()), int(t.is_cuda)


def kda_state_snapshot(st, slots, dst: torch.Tensor, stream=None) -> None:
    arr, p = _host_i32(slots)
    ptr, on_dev = _buf(dst, kda_state_blob_bytes(st, len(arr)), "dst")
    _check(lib().kda_state_snapshot(st, p, len(arr), ptr, on_dev, _stream(stream)))


def kda_state_restore(st, slots, src: torch.Tensor, stream=None) -> None:
    arr, p = _host_i32(slots)
    ptr, on_dev = _buf(src, kda_state_blob_bytes(st, len(arr)), "src")
    _check(lib().kda_state_restore(st, p, len(arr), ptr, on_dev, _stream(stream)))


def kda_layer_params_from(conv_w: torch.Tensor, dt_bias: torch.Tensor, A_log: torch.Tensor,
                          norm_w: torch.Tensor) -> kda_layer_params:
    p = kda_layer_params(_dev(conv_w, torch.float32, "conv_w"), _dev(dt_bias, torch.float32, "dt_bias"),
                         _dev(A_log, torch.float32, "A_log"), _dev(norm_w, torch.float32, "norm_w"))
    p._keep = (conv_w, dt_bias, A_log, norm_w)
    return p


def kda_decode_token(cfg: kda_config_t, params: kda_layer_params, st, slots: torch.Tensor,
                     q, k, v, z, b, g, out, stream=None) -> None:
    dt = _torch_io_dtype(cfg)
    B = int(slots.numel())
    D = cfg.num_heads * cfg.head_dim
    for name, t, width in (("q", q, D), ("k", k, D), ("v", v, D), ("z", z, D), ("g", g, D),
                           ("b", b, cfg.num_heads), ("out", out, D)):
        if t.numel() != B * width:
            raise ValueError(f"{name} must hold {B} x {width} elements, got {tuple(t.shape)}")
    _check(lib().kda_decode_token(ctypes.byref(cfg), ctypes.byref(params), st, _dev(slots, torch.int32, "slots"), B,
                                  _dev(q, dt, "q"), _dev(k, dt, "k"), _dev(v, dt, "v"), _dev(z, dt, "z"),
                                  _dev(b, dt, "b"), _dev(g, dt, "g"), _dev(out, dt, "out"), _stream(stream)))


def kda_decode_tokens(cfg: kda_config_t, params: kda_layer_params, st, slots: torch.Tensor, n: int,
                      q, k, v, z, b, g, out, stream=None) -> None:
    """n consecutive decode tokens per row: q,k,v,z,g,out [B][n][H*d], b [B][n][H]."""
    dt = _torch_io_dtype(cfg)
    B = int(slots.numel())
    D = cfg.num_heads * cfg.head_dim
    for name, t, width in (("q", q, D), ("k", k, D), ("v", v, D), ("z", z, D), ("g", g, D),
                           ("b", b, cfg.num_heads), ("out", out, D)):
        if t.numel() != B * n * width:
            raise ValueError(f"{name} must hold {B} x {n} x {width} elements, got {tuple(t.shape)}")
    _check(lib().kda_decode_tokens(ctypes.byref(cfg), ctypes.byref(params), st, _dev(slots, torch.int32, "slots"),
                                   B, int(n), _dev(q, dt, "q"), _dev(k, dt, "k"), _dev(v, dt, "v"),
                                   _dev(z, dt, "z"), _dev(b, dt, "b"), _dev(g, dt, "g"), _dev(out, dt, "out"),
                                   _stream(stream)))


def kda_prefill(cfg: kda_config_t, params: kda_layer_params, st, slots: torch.Tensor, cu_seqlens: torch.Tensor,
                cu_seqlens_host, q, k, v, z, b, g, out, stream=None) -> None:
    dt = _torch_io_dtype(cfg)
    N = int(slots.numel())
    cu_h, cu_p = _host_i32(cu_seqlens_host)
    if len(cu_h) != N + 1 or cu_seqlens.numel() != N + 1:
        raise ValueError("cu_seqlens must hold N + 1 entries")
    T = int(cu_h[-1]) if N > 0 else 0
    D = cfg.num_heads * cfg.head_dim
    for name, t, width in (("q", q, D), ("k", k, D), ("v", v, D), ("z", z, D), ("g", g, D),
                           ("b", b, cfg.num_heads), ("out", out, D)):
        if t.numel() != T * width:
            raise ValueError(f"{name} must hold {T} x {width} elements, got {tuple(t.shape)}")
    _check(lib().kda_prefill(ctypes.byref(cfg), ctypes.byref(params), st, _dev(slots, torch.int32, "slots"),
                             _dev(cu_seqlens, torch.int32, "cu_seqlens"), cu_p, N,
                             _dev(q, dt, "q"), _dev(k, dt, "k"), _dev(v, dt, "v"), _dev(z, dt, "z"),
                             _dev(b, dt, "b"), _dev(g, dt, "g"), _dev(out, dt, "out"), _stream(stream)))


def kda_prefill_noalloc(cfg: kda_config_t, params: kda_layer_params, S: torch.Tensor, tail: torch.Tensor,
                        err, slots: torch.Tensor, cu_seqlens: torch.Tensor, cu_seqlens_host,
                        q, k, v, z, b, g, out, stream=None) -> None:
    """kda_prefill on caller-owned state buffers with the library's static workspace.

    S: FP32 [max_slots, H, d, d]; tail: io dtype [max_slots, 3, K-1, H*d]; err: int32
    device tensor of one element, or None.
    """
    dt = _torch_io_dtype(cfg)
    H, d, Kc = cfg.num_heads, cfg.head_dim, cfg.conv_kernel
    if S.dim() != 4 or tuple(S.shape[1:]) != (H, d, d):
        raise ValueError(f"S must be [max_slots, {H}, {d}, {d}]")
    max_slots = int(S.shape[0])
    if tuple(tail.shape) != (max_slots, 3, Kc - 1, H * d):
        raise ValueError(f"tail must be [{max_slots}, 3, {Kc - 1}, {H * d}]")
    N = int(slots.numel())
    cu_h, cu_p = _host_i32(cu_seqlens_host)
    if len(cu_h) != N + 1 or cu_seqlens.numel() != N + 1:
        raise ValueError("cu_seqlens must hold N + 1 entries")
    T = int(cu_h[-1]) if N > 0 else 0
    D = H * d
    for name, t, width in (("q", q, D), ("k", k, D), ("v", v, D), ("z", z, D), ("g", g, D),
                           ("b", b, H), ("out", out, D)):
        if t.numel() != T * width:
            raise ValueError(f"{name} must hold {T} x {width} elements, got {tuple(t.shape)}")
    errp = _VP(None) if err is None else _dev(err, torch.int32, "err")
    _check(lib().kda_prefill_noalloc(ctypes.byref(cfg), ctypes.byref(params), _dev(S, torch.float32, "S"),
                                     _dev(tail, dt, "tail"), max_slots, errp, _dev(slots, torch.int32, "slots"),
                                     _dev(cu_seqlens, torch.int32, "cu_seqlens"), cu_p, N,
                                     _dev(q, dt, "q"), _dev(k, dt, "k"), _dev(v, dt, "v"), _dev(z, dt, "z"),
                                     _dev(b, dt, "b"), _dev(g, dt, "g"), _dev(out, dt, "out"), _stream(stream)))


def kda_gate_proj_workspace_bytes(cfg: kda_config_t, hidden: int, T: int) -> int:
    return int(lib().kda_gate_proj_workspace_bytes(ctypes.byref(cfg), int(hidden), int(T)))


def kda_gate_proj(cfg: kda_config_t, x, w_fa, w_fb, w_b, z, b, workspace: torch.Tensor, stream=None) -> None:
    """z = W_fb (W_fa x), b = W_b x for x [T, hidden]; every tensor in the config's I/O dtype
    except the workspace (any dtype, at least kda_gate_proj_workspace_bytes bytes)."""
    H, d = cfg.num_heads, cfg.head_dim
    if x.dim() != 2:
        raise ValueError("x must be [T, hidden]")
    T, hidden = int(x.shape[0]), int(x.shape[1])
    for name, t, shape in (("w_fa", w_fa, (d, hidden)), ("w_fb", w_fb, (H * d, d)), ("w_b", w_b, (H, hidden)),
                           ("z", z, (T, H * d)), ("b", b, (T, H))):
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    bf = _torch_io_dtype(cfg)
    ws = _dev(workspace, None, "workspace")
    _check(lib().kda_gate_proj(ctypes.byref(cfg), hidden, T, _dev(x, bf, "x"), _dev(w_fa, bf, "w_fa"),
                               _dev(w_fb, bf, "w_fb"), _dev(w_b, bf, "w_b"), _dev(z, bf, "z"), _dev(b, bf, "b"),
                               ws, workspace.numel() * workspace.element_size(), _stream(stream)))


def kda_gate_proj_in(cfg: kda_config_t, x, w_fa, w_b, f, b, workspace: torch.Tensor, stream=None) -> None:
    """f = W_fa x [T, d] and b = W_b x [T, H] (BF16), the inputs of kda_prefill_gate_fused."""
    H, d = cfg.num_heads, cfg.head_dim
    if x.dim() != 2:
        raise ValueError("x must be [T, hidden]")
    T, hidden = int(x.shape[0]), int(x.shape[1])
    for name, t, shape in (("w_fa", w_fa, (d, hidden)), ("w_b", w_b, (H, hidden)), ("f", f, (T, d)), ("b", b, (T, H))):
        if tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    bf = torch.bfloat16
    _check(lib().kda_gate_proj_in(ctypes.byref(cfg), hidden, T, _dev(x, bf, "x"), _dev(w_fa, bf, "w_fa"),
                                  _dev(w_b, bf, "w_b"), _dev(f, bf, "f"), _dev(b, bf, "b"),
                                  _dev(workspace, None, "workspace"), workspace.numel() * workspace.element_size(),
                                  _stream(stream)))


def kda_prefill_gate_fused(cfg: kda_config_t, params: kda_layer_params, st, slots: torch.Tensor,
                           cu_seqlens: torch.Tensor, cu_seqlens_host, q, k, v, f, w_fb, b, g, out, stream=None) -> None:
    """kda_prefill with z = W_fb f formed inside (f = W_fa x [T, d], w_fb [H d, d]; BF16)."""
    bf = torch.bfloat16
    N = int(slots.numel())
    cu_h, cu_p = _host_i32(cu_seqlens_host)
    if len(cu_h) != N + 1 or cu_seqlens.numel() != N + 1:
        raise ValueError("cu_seqlens must hold N + 1 entries")
    T = int(cu_h[-1]) if N > 0 else 0
    H, d = cfg.num_heads, cfg.head_dim
    D = H * d
    for name, t, width in (("q", q, D), ("k", k, D), ("v", v, D), ("f", f, d), ("g", g, D), ("b", b, H),
                           ("out", out, D)):
        if t.numel() != T * width:
            raise ValueError(f"{name} must hold {T} x {width} elements, got {tuple(t.shape)}")
    if tuple(w_fb.shape) != (D, d):
        raise ValueError(f"w_fb must be [{D}, {d}]")
    _check(lib().kda_prefill_gate_fused(ctypes.byref(cfg), ctypes.byref(params), st, _dev(slots, torch.int32, "slots"),
                                        _dev(cu_seqlens, torch.int32, "cu_seqlens"), cu_p, N, _dev(q, bf, "q"),
                                        _dev(k, bf, "k"), _dev(v, bf, "v"), _dev(f, bf, "f"), _dev(w_fb, bf, "w_fb"),
                                        _dev(b, bf, "b"), _dev(g, bf, "g"), _dev(out, bf, "out"), _stream(stream)))


def kda_linear_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().kda_linear_workspace_bytes(int(M), int(N), int(K)))


def kda_linear(x, w, y, workspace: torch.Tensor, r=None, ysplit: int = 0, stream=None) -> None:
    """y = x w^T (+ r), BF16: x [M, K], w [N, K], y [M, N] (or [N / ysplit, M, ysplit] with ysplit)."""
    bf = torch.bfloat16
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x must be [M, K] and w [N, K]")
    M, K = int(x.shape[0]), int(x.shape[1])
    N = int(w.shape[0])
    if y.numel() != M * N:
        raise ValueError(f"y must hold {M} x {N} elements, got {tuple(y.shape)}")
    if r is not None and r.numel() != M * N:
        raise ValueError(f"r must hold {M} x {N} elements, got {tuple(r.shape)}")
    _check(lib().kda_linear(M, N, K, _dev(x, bf, "x"), _dev(w, bf, "w"),
                            _VP(None) if r is None else _dev(r, bf, "r"), _dev(y, bf, "y"), int(ysplit),
                            _dev(workspace, None, "workspace"), workspace.numel() * workspace.element_size(),
                            _stream(stream)))


def _bad_tensor(name: str, t, dtype, dev: int, shape=None) -> None:
    """Why a tensor was not taken: not of dtype (None: any), contiguous, on CUDA device dev and (if given) of shape."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must have dtype {dtype}, got {t.dtype}")
    if t.device.index != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _ptr(name: str, t, dtype, dev: int, shape=None) -> int:
    """The address of a tensor that passes (the tests in the order of their cost)."""
    try:
        if (dtype is None or t.dtype is dtype) and t.get_device() == dev and (shape is None or t.shape == shape) and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _bad_tensor(name, t, dtype, dev, shape)


_BF16, _F32, _F8, _I32T = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.int32


def kda_quant_fp8(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, block_rows: int = 1, stream=None) -> None:
    """q [M, K] (float8_e4m3fn) and s [ceil(M / block_rows), ceil(K / 128)] (FP32) from x [M, K] (BF16 or
    FP32, contiguous within a row): one power-of-two scale for each 1 x 128 or 128 x 128 block."""
    dev = _current_device()
    dt = x.dtype
    if x.dim() != 2 or not x.is_cuda or not (dt is _BF16 or dt is _F32):
        raise TypeError("x must be a CUDA tensor [M, K] of bfloat16 or float32")
    M, K = x.shape
    if block_rows < 1:
        raise ValueError("block_rows must be 1 or 128")
    if M > 0 and K > 1 and x.stride(1) != 1:
        raise ValueError("x must be contiguous within a row")
    if x.get_device() != dev:
        raise ValueError(f"x is on {x.device}, the current device is cuda:{dev}")
    st = lib().kda_quant_fp8(M, K, x.data_ptr(), x.stride(0) if M > 1 else K, KDA_BF16 if dt is _BF16 else KDA_F32, block_rows,
                             _ptr("q", q, _F8, dev, (M, K)), _ptr("s", s, _F32, dev, (-(-M // block_rows), -(-K // 128))),
                             _raw_stream(stream, dev))
    if st:
        _check(st)


def kda_linear_fp8_workspace_bytes(M: int, N: int, K: int) -> int:
    need = int(lib().kda_linear_fp8_workspace_bytes(int(M), int(N), int(K)))
    if need == 0:
        raise KdaError(KDA_ERR_INVALID, kda_last_error())
    return need


def kda_linear_fp8(xq, xs, wq, ws, y, workspace: torch.Tensor, r=None, ysplit: int = 0, stream=None) -> None:
    """y = x w^T (+ r) in BF16 from E4M3 xq [M, K], wq [N, K] and their scales xs [M, ceil(K / 128)],
    ws [ceil(N / 128), ceil(K / 128)]; y [M, N] (or [N / ysplit, M, ysplit] with ysplit)."""
    dev = _current_device()
    if xq.dim() != 2 or wq.dim() != 2 or xq.shape[1] != wq.shape[1]:
        raise ValueError("xq must be [M, K] and wq [N, K]")
    M, K = xq.shape
    N = wq.shape[0]
    nk = -(-K // 128)
    if y.numel() != M * N or (r is not None and r.numel() != M * N):
        raise ValueError(f"y and r must hold {M} x {N} elements")
    st = lib().kda_linear_fp8(M, N, K, _ptr("xq", xq, _F8, dev), _ptr("xs", xs, _F32, dev, (M, nk)), _ptr("wq", wq, _F8, dev),
                              _ptr("ws", ws, _F32, dev, (-(-N // 128), nk)), None if r is None else _ptr("r", r, _BF16, dev),
                              _ptr("y", y, _BF16, dev), ysplit, _ptr("workspace", workspace, None, dev), workspace.nbytes,
                              _raw_stream(stream, dev))
    if st:
        _check(st)


def kda_gdr_config(num_heads: int, num_qk_heads: int | None = None, head_dim: int = 128,
                   io_dtype: int = KDA_BF16) -> kda_gdr_config_t:
    cfg = kda_gdr_config_t()
    _check(lib().kda_gdr_config(ctypes.byref(cfg), num_heads, num_heads if num_qk_heads is None else num_qk_heads,
                                head_dim, io_dtype))
    return cfg


def kda_gdr_params_from(A_log: torch.Tensor, dt_bias: torch.Tensor) -> kda_gdr_params:
    if A_log.shape != dt_bias.shape or A_log.dim() != 1:
        raise ValueError("A_log and dt_bias must both be [H]")
    p = kda_gdr_params(_dev(A_log, torch.float32, "A_log"), _dev(dt_bias, torch.float32, "dt_bias"))
    if A_log.device != dt_bias.device:
        raise ValueError("A_log and dt_bias must be on one device")
    p._keep = (A_log, dt_bias)
    p.heads, p.device = A_log.numel(), A_log.device.index
    return p


def _check_row(name, t, T, width, dt, dev) -> None:
    """Raise for a row tensor that a call cannot take."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dt:
        raise TypeError(f"{name} must be a CUDA tensor of {dt}")
    if t.device.index != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    if tuple(t.shape) != (T, width):
        raise ValueError(f"{name} must be [{T}, {width}], got {list(t.shape)}")
    if T > 0 and width > 1 and t.stride(1) != 1:
        raise ValueError(f"{name} must be contiguous within a token")


def _gdr_call(cfg, params, S, src_slots, dst_slots, T, q, k, v, a, b, out, err, dev):
    """The checked pointers of a gated delta rule call over T tokens, the current device being dev: S, src,
    dst, rows, err."""
    H, d = cfg.num_heads, cfg.head_dim
    wk, wv = cfg.num_qk_heads * d, H * d
    dt = _BF16 if cfg.io_dtype == KDA_BF16 else _F32
    if S.shape[1:] != (H, d, d):
        raise ValueError(f"S must be [max_slots, {H}, {d}, {d}], got {list(S.shape)}")
    if params.heads != H or params.device != dev:
        raise ValueError(f"A_log and dt_bias must hold {H} elements on cuda:{dev}, got {params.heads} on cuda:{params.device}")
    if src_slots.numel() != dst_slots.numel():
        raise ValueError("src_slots and dst_slots must have the same length")
    qk, vo, ab = (T, wk), (T, wv), (T, H)
    if (q.dtype is dt and k.dtype is dt and v.dtype is dt and a.dtype is dt and b.dtype is dt and out.dtype is dt
            and q.shape == qk and k.shape == qk and v.shape == vo and out.shape == vo and a.shape == ab and b.shape == ab
            and q.get_device() == k.get_device() == v.get_device() == a.get_device() == b.get_device() == out.get_device() == dev
            and (T == 0 or (q.stride(1) == k.stride(1) == v.stride(1) == out.stride(1) == 1
                            and (H == 1 or a.stride(1) == b.stride(1) == 1)))):
        r = kda_gdr_rows(q.data_ptr(), k.data_ptr(), v.data_ptr(), a.data_ptr(), b.data_ptr(), out.data_ptr(),
                         *((q.stride(0), k.stride(0), v.stride(0), a.stride(0), b.stride(0), out.stride(0)) if T > 1 else
                           (wk, wk, wv, H, H, wv)))
        return (_ptr("S", S, _F32, dev), _ptr("src_slots", src_slots, _I32T, dev), _ptr("dst_slots", dst_slots, _I32T, dev),
                r, None if err is None else _ptr("err", err, _I32T, dev))
    for name, t, width in (("q", q, wk), ("k", k, wk), ("v", v, wv), ("a", a, H), ("b", b, H), ("out", out, wv)):
        _check_row(name, t, T, width, dt, dev)


def kda_gdr_decode(cfg: kda_gdr_config_t, params: kda_gdr_params, S: torch.Tensor, src_slots: torch.Tensor,
                   dst_slots: torch.Tensor, n: int, q, k, v, a, b, out, err=None, stream=None) -> None:
    """n tokens for each row: q, k [B n, Hk d], v, out [B n, H d], a, b [B n, H], contiguous within a
    token; S FP32 [max_slots, H, d, d], read at src_slots (-1: zeros) and written at dst_slots."""
    dev = _current_device()
    B = src_slots.numel()
    Sp, sp, dp, r, ep = _gdr_call(cfg, params, S, src_slots, dst_slots, B * n, q, k, v, a, b, out, err, dev)
    st = lib().kda_gdr_decode(cfg, params, Sp, S.shape[0], sp, dp, B, n, r, ep, _raw_stream(stream, dev))
    if st:
        _check(st)


def kda_gdr_workspace_bytes(cfg: kda_gdr_config_t, cu_seqlens_host) -> int:
    cu_h, cu_p = _host_i32(cu_seqlens_host)
    need = int(lib().kda_gdr_workspace_bytes(ctypes.byref(cfg), cu_p, len(cu_h) - 1))
    if need == 0:
        raise KdaError(KDA_ERR_INVALID, kda_last_error())
    return need


def kda_gdr_prefill(cfg: kda_gdr_config_t, params: kda_gdr_params, S: torch.Tensor, src_slots: torch.Tensor,
                    dst_slots: torch.Tensor, cu_seqlens: torch.Tensor, cu_seqlens_host, q, k, v, a, b, out,
                    workspace: torch.Tensor, err=None, stream=None) -> None:
    """Packed sequences, rows as in kda_gdr_decode with T = cu_seqlens[-1]; workspace of at least
    kda_gdr_workspace_bytes(cfg, cu_seqlens_host) bytes."""
    dev = _current_device()
    N = src_slots.numel()
    cu_h = _i32_array(cu_seqlens_host)
    if cu_h.shape != (N + 1,):
        raise ValueError("cu_seqlens_host must hold N + 1 entries")
    Sp, sp, dp, r, ep = _gdr_call(cfg, params, S, src_slots, dst_slots, int(cu_h[N]), q, k, v, a, b, out, err, dev)
    st = lib().kda_gdr_prefill(cfg, params, Sp, S.shape[0], sp, dp, _ptr("cu_seqlens", cu_seqlens, _I32T, dev, (N + 1,)),
                               cu_h.ctypes.data, N, r, _ptr("workspace", workspace, None, dev), workspace.nbytes, ep,
                               _raw_stream(stream, dev))
    if st:
        _check(st)


def kda_glr_config(dim: int, io_dtype: int = KDA_BF16) -> kda_glr_config_t:
    cfg = kda_glr_config_t()
    _check(lib().kda_glr_config(ctypes.byref(cfg), dim, io_dtype))
    return cfg


def _vectors(p, device, **tensors) -> None:
    """Keep a layer's FP32 vectors, all of one length and on one device, in its parameters p."""
    shape = next(iter(tensors.values())).shape
    for name, t in tensors.items():
        if t.dim() != 1 or t.shape != shape or t.device != device:
            raise ValueError(f"{' and '.join(tensors)} must be vectors of one length on one device")
        setattr(p, name, _dev(t, torch.float32, name))
    p._keep = tuple(tensors.values())
    p.dim, p.device = shape[0], device.index


def kda_glr_params_from(A_log: torch.Tensor, a_bias: torch.Tensor, b_bias: torch.Tensor) -> kda_glr_params:
    p = kda_glr_params()
    _vectors(p, A_log.device, A_log=A_log, a_bias=a_bias, b_bias=b_bias)
    return p


def _row_args(pack, names, tensors, T, width, dt, dev):
    """A row struct (as `pack` makes it: bytes), its pointers, then its strides, from checked tensors [T, width] of dt on device
    dev, contiguous within a token (None: not given)."""
    shape, ptrs, strides, many = (T, width), [], [], T > 1
    for name, t in zip(names, tensors):
        if t is None:
            ptrs.append(0)
            strides.append(0)
            continue
        try:
            step, one = t.stride()
            if t.dtype is not dt or t.shape != shape or t.get_device() != dev or one != 1:
                _check_row(name, t, T, width, dt, dev)
        except (AttributeError, ValueError):
            _check_row(name, t, T, width, dt, dev)
            raise
        ptrs.append(t.data_ptr())
        strides.append(step if many else width)
    return pack(*ptrs, *strides)


def _tuple(*v):
    return v


def _f32(name, t, dev, shape):
    return None if t is None else _ptr(name, t, _F32, dev, shape)


def _params_ok(cfg, params, dev) -> None:
    if params.dim != cfg.dim or params.device != dev:
        raise ValueError(f"the parameters must hold {cfg.dim} elements on cuda:{dev}, got {params.dim} on cuda:{params.device}")


def _states(cfg, S, src_slots, dst_slots, dev):
    """The checked addresses of S, src_slots and dst_slots."""
    if src_slots.numel() != dst_slots.numel():
        raise ValueError("src_slots and dst_slots must have the same length")
    if S.dim() != 2 or S.shape[1] != cfg.dim:
        raise ValueError(f"S must be [max_slots, {cfg.dim}], got {list(S.shape)}")
    if (S.dtype is _F32 and src_slots.dtype is _I32T and dst_slots.dtype is _I32T and S.get_device() == src_slots.get_device() == dst_slots.get_device() == dev
            and S.is_contiguous() and src_slots.is_contiguous() and dst_slots.is_contiguous()):
        return S.data_ptr(), src_slots.data_ptr(), dst_slots.data_ptr()
    return _ptr("S", S, _F32, dev), _ptr("src_slots", src_slots, _I32T, dev), _ptr("dst_slots", dst_slots, _I32T, dev)


def kda_glr_decode(cfg: kda_glr_config_t, params: kda_glr_params, S: torch.Tensor, src_slots: torch.Tensor, dst_slots: torch.Tensor,
                   n: int, x, a, b, g, out, err=None, stream=None) -> None:
    """n tokens for each row: x, a, b, g (or None), out [B n, dim], contiguous within a token; S FP32 [max_slots, dim],
    read at src_slots (-1: zeros) and written at dst_slots."""
    dev = _current_device()
    B = src_slots.numel()
    _params_ok(cfg, params, dev)
    Sp, sp, dp = _states(cfg, S, src_slots, dst_slots, dev)
    r = _row_args(_PACK_GLR_ROWS, _GLR_ROWS, (x, a, b, g, out), B * n, cfg.dim, _F32 if cfg.io_dtype == KDA_F32 else _BF16, dev)
    st = lib().kda_glr_decode(cfg, params, Sp, S.shape[0], sp, dp, B, n, r, None if err is None else _ptr("err", err, _I32T, dev),
                              _raw_stream(stream, dev))
    if st:
        _check(st)


def kda_glr_workspace_bytes(cfg: kda_glr_config_t, cu_seqlens_host) -> int:
    cu_h, cu_p = _host_i32(cu_seqlens_host)
    need = int(lib().kda_glr_workspace_bytes(ctypes.byref(cfg), cu_p, len(cu_h) - 1))
    if need == 0:
        raise KdaError(KDA_ERR_INVALID, kda_last_error())
    return need


def _lengths(cu_seqlens_host):
    """A host cu_seqlens as 32-bit numbers: what keeps them, their address, how many, and the last."""
    if isinstance(cu_seqlens_host, (list, tuple)):
        try:
            a = array("i", cu_seqlens_host)
            return a, a.buffer_info()[0], len(a), a[-1] if a else 0
        except (OverflowError, TypeError):  # refused, or taken as other numbers, below
            pass
    a = _i32_array(cu_seqlens_host).reshape(-1)
    return a, a.ctypes.data, len(a), int(a[-1]) if len(a) else 0


def kda_glr_chunks(cu_seqlens_host) -> int:
    """Rows of the `starts` that a kda_glr_prefill of these sequences fills for its backward."""
    keep, at, count, _ = _lengths(cu_seqlens_host)
    n = lib().kda_glr_chunks(at, count - 1)
    if n < 0:
        raise KdaError(KDA_ERR_INVALID, kda_last_error())
    return n


def _glr_starts(cfg, starts, at, N, dev):
    """The address of starts, of as many rows as the sequences' chunks or more."""
    n = lib().kda_glr_chunks(at, N)
    if n < 0:
        raise KdaError(KDA_ERR_INVALID, kda_last_error())
    if starts.dim() != 2 or starts.shape[0] < n or starts.shape[1] != cfg.dim:
        raise ValueError(f"starts must be [{n}, {cfg.dim}] or longer, got {list(starts.shape)}")
    return _ptr("starts", starts, _F32, dev)


def kda_glr_prefill(cfg: kda_glr_config_t, params: kda_glr_params, S: torch.Tensor, src_slots: torch.Tensor, dst_slots: torch.Tensor,
                    cu_seqlens: torch.Tensor, cu_seqlens_host, x, a, b, g, out, workspace: torch.Tensor, starts=None, err=None,
                    stream=None) -> None:
    """Packed sequences, rows as in kda_glr_decode with T = cu_seqlens[-1]; workspace of at least
    kda_glr_workspace_bytes(cfg, cu_seqlens_host) bytes; starts FP32 [kda_glr_chunks(cu_seqlens_host), dim] for a backward."""
    dev = _current_device()
    N = src_slots.numel()
    keep, at, count, T = _lengths(cu_seqlens_host)
    if count != N + 1 or cu_seqlens.numel() != count:
        raise ValueError("cu_seqlens and cu_seqlens_host must hold N + 1 entries")
    _params_ok(cfg, params, dev)
    Sp, sp, dp = _states(cfg, S, src_slots, dst_slots, dev)
    r = _row_args(_PACK_GLR_ROWS, _GLR_ROWS, (x, a, b, g, out), T, cfg.dim, _F32 if cfg.io_dtype == KDA_F32 else _BF16, dev)
    st = lib().kda_glr_prefill(cfg, params, Sp, S.shape[0], sp, dp, _ptr("cu_seqlens", cu_seqlens, _I32T, dev), at, N, r,
                               None if starts is None else _glr_starts(cfg, starts, at, N, dev), _ptr("workspace", workspace, None, dev),
                               workspace.nbytes, None if err is None else _ptr("err", err, _I32T, dev), _raw_stream(stream, dev))
    if st:
        _check(st)


def kda_glr_backward(cfg: kda_glr_config_t, params: kda_glr_params, cu_seqlens: torch.Tensor, cu_seqlens_host, starts: torch.Tensor,
                     x, a, b, g, dout, dx, da, db, dg, work: torch.Tensor, dS_last=None, dS_first=None, dA_log=None, da_bias=None,
                     db_bias=None, err=None, stream=None) -> None:
    """The gradients of a kda_glr_prefill that filled `starts`: rows [T, dim] (dg None where g is), dS_last (None: zeros)
    and dS_first [N, dim], and FP32 sums over all tokens, dA_log, da_bias, db_bias [dim]; work as the prefill's workspace."""
    dev = _current_device()
    keep, at, count, T = _lengths(cu_seqlens_host)
    N = count - 1
    if cu_seqlens.numel() != count:
        raise ValueError("cu_seqlens and cu_seqlens_host must hold N + 1 entries")
    _params_ok(cfg, params, dev)
    r = _row_args(_PACK_GLR_GRADS, _GLR_GRADS, (x, a, b, g, dout, dx, da, db, dg), T, cfg.dim, _F32 if cfg.io_dtype == KDA_F32 else _BF16, dev)
    vec, state = (cfg.dim,), (N, cfg.dim)
    st = lib().kda_glr_backward(cfg, params, _ptr("cu_seqlens", cu_seqlens, _I32T, dev), at, N, _glr_starts(cfg, starts, at, N, dev), r,
                                _f32("dS_last", dS_last, dev, state), _f32("dS_first", dS_first, dev, state), _f32("dA_log", dA_log, dev, vec),
                                _f32("da_bias", da_bias, dev, vec), _f32("db_bias", db_bias, dev, vec), _ptr("work", work, None, dev),
                                work.nbytes, None if err is None else _ptr("err", err, _I32T, dev), _raw_stream(stream, dev))
    if st:
        _check(st)


def kda_block_norm_config(dim: int, io_dtype: int = KDA_BF16) -> kda_block_norm_config_t:
    cfg = kda_block_norm_config_t()
    _check(lib().kda_block_norm_config(ctypes.byref(cfg), dim, io_dtype))
    return cfg


def kda_block_norm_params_from(post_w: torch.Tensor, scale: torch.Tensor, pre_w: torch.Tensor) -> kda_block_norm_params:
    p = kda_block_norm_params()
    _vectors(p, post_w.device, post_w=post_w, scale=scale, pre_w=pre_w)
    return p


def kda_block_norm(cfg: kda_block_norm_config_t, params: kda_block_norm_params, x, y=None, g=None, x_out=None, h=None, hs=None,
                   stream=None) -> None:
    """x_out = x + scale sigmoid(g) post_w y / rms(y) and h = pre_w x_out / rms(x_out) for rows [M, dim], contiguous within
    a row; without y only h of x, without h only x_out. h in the rows' type, or float8_e4m3fn with hs FP32 [M, ceil(dim / 128)]."""
    dev = _current_device()
    _params_ok(cfg, params, dev)
    M, D = x.shape[0], cfg.dim
    dt = _F32 if cfg.io_dtype == KDA_F32 else _BF16
    if hs is None:
        r = _row_args(_PACK_NORM_ROWS5, _NORM_ROWS, (x, y, g, x_out, h), M, D, dt, dev)
    else:
        e = _row_args(_tuple, ("h",), (h,), M, D, _F8, dev)
        p = _row_args(_tuple, _NORM_ROWS, (x, y, g, x_out), M, D, dt, dev)
        r = _PACK_NORM_ROWS(*p[:4], e[0], _f32("hs", hs, dev, (M, -(-D // 128))), *p[4:], e[1])
    st = lib().kda_block_norm(cfg, params, M, r, _raw_stream(stream, dev))
    if st:
        _check(st)


def kda_block_norm_workspace_bytes(cfg: kda_block_norm_config_t, M: int) -> int:
    need = int(lib().kda_block_norm_workspace_bytes(ctypes.byref(cfg), int(M)))
    if need == 0:
        raise KdaError(KDA_ERR_INVALID, kda_last_error())
    return need


def kda_block_norm_backward(cfg: kda_block_norm_config_t, params: kda_block_norm_params, x_out, dh, dx1, dx, work: torch.Tensor, y=None,
                            g=None, dy=None, dg=None, dpost_w=None, dscale=None, dpre_w=None, stream=None) -> None:
    """Gradients of kda_block_norm from its x_out (x where it had no y), the gradient dh of h (None: not used) and that of
    x_out from elsewhere, dx1 (None: zeros): rows dx, dy, dg [M, dim] and sums over the rows dpost_w, dscale, dpre_w FP32
    [dim], each or None; work of at least kda_block_norm_workspace_bytes(cfg, M) bytes."""
    dev = _current_device()
    _params_ok(cfg, params, dev)
    r = _row_args(_PACK_NORM_GRADS, _NORM_GRADS, (x_out, dh, dx1, y, g, dx, dy, dg), dx.shape[0], cfg.dim,
                  _F32 if cfg.io_dtype == KDA_F32 else _BF16, dev)
    vec = (cfg.dim,)
    st = lib().kda_block_norm_backward(cfg, params, dx.shape[0], r, _f32("dpost_w", dpost_w, dev, vec), _f32("dscale", dscale, dev, vec),
                                       _f32("dpre_w", dpre_w, dev, vec), _ptr("work", work, None, dev), work.nbytes,
                                       _raw_stream(stream, dev))
    if st:
        _check(st)


def _layers(layers):
    hs = [layers] if isinstance(layers, _VP) else list(layers)
    arr = (_VP * len(hs))(*[h.value if isinstance(h, _VP) else h for h in hs])
    return arr, len(hs)


def kda_photo_store_create(capacity: int = -1, dir: str | None = None) -> ctypes.c_void_p:
    """A photo store: capacity < 0 means "not given" (2 with a directory, else 0 = off)."""
    h = _VP()
    _check(lib().kda_photo_store_create(capacity, None if dir is None else dir.encode(), ctypes.byref(h)))
    return h


def kda_photo_store_free(ps) -> None:
    _check(lib().kda_photo_store_free(ps))


def kda_photo_count(ps) -> int:
    return int(lib().kda_photo_count(ps))


def kda_photo_capacity(ps) -> int:
    return int(lib().kda_photo_capacity(ps))


def kda_photo_take(ps, layers, slot: int, tokens, stream=None) -> int:
    """Photo of `slot` of each state in `layers` after the host token prefix; returns its id (-1: store off)."""
    arr, n = _layers(layers)
    tok, tp = _host_i32(tokens)
    pid = ctypes.c_int32()
    _check(lib().kda_photo_take(ps, arr, n, slot, tp, len(tok), ctypes.byref(pid), _stream(stream)))
    return int(pid.value)


def kda_photo_find(ps, tokens) -> tuple[int, int]:
    """(photo id, prefix length) of the deepest photo whose prefix starts `tokens`, or (-1, 0)."""
    tok, tp = _host_i32(tokens)
    pid, plen = ctypes.c_int32(), ctypes.c_int64()
    _check(lib().kda_photo_find(ps, tp, len(tok), ctypes.byref(pid), ctypes.byref(plen)))
    return int(pid.value), int(plen.value)


def kda_photo_restore(ps, photo_id: int, layers, slot: int, stream=None) -> None:
    arr, n = _layers(layers)
    _check(lib().kda_photo_restore(ps, photo_id, arr, n, slot, _stream(stream)))


def kda_state_poll_error(st) -> int:
    code = ctypes.c_int32()
    _check(lib().kda_state_poll_error(st, ctypes.byref(code)))
    return int(code.value)
