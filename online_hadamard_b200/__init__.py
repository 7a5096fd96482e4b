"""Python binding of libmacaq: the MACaQ MXFP4 W4A4 linear layer on B200 (sm_100a).

Argument marshalling only: every function below checks tensor placement, dtype and
contiguity, allocates outputs (on the call's stream) when the caller does not pass them, and calls the
C entry point of the same name in ``_build/libmacaq.so`` with the tensors' device made
current, on that device's current CUDA stream (or the stream passed, which must belong to it).  All
arithmetic runs in the library's CUDA kernels; there is no CPU or PyTorch fallback -- if
the library cannot be loaded, every call raises.

Method: "MACaQ: Fast, Model Agnostic Calibrated Quantization for Low-Precision Weights and
Activations", Abstract (per-channel scale and block-Hadamard applied online to the
activations, inverse transforms absorbed into the weights, MXFP4 W4A4).  Layouts and
conventions are documented in include/macaq.h.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import torch

from . import build as _build_mod

__all__ = [
    "load_library", "MacaqError", "scale_bytes", "scale_offset", "linear_workspace_bytes", "gemm_workspace_bytes",
    "macaq_calibrate_scale", "macaq_fold_weights", "macaq_act_transform_quant", "macaq_act_quant_plain",
    "macaq_mxfp4_gemm", "macaq_w4a4_linear", "macaq_mxfp4_linear", "macaq_w4a4_grouped_linear",
    "grouped_workspace_bytes", "macaq_w4a4_linear_noalloc", "macaq_calib_hessian", "macaq_flip_refine",
    "macaq_w4a4_grouped_linear_device", "grouped_device_workspace_bytes", "macaq_scales_to_tiled",
    "macaq_scales_to_rowmajor", "macaq_w4a4_linear_multi", "linear_multi_workspace_bytes",
    "macaq_qk_norm_rope", "macaq_kv4_append", "macaq_kv4_gather", "macaq_kv4_attention", "kv4_page_bytes",
    "kv4_attention_workspace_bytes",
    "macaq_device_status", "status_str", "EXPORTED_SYMBOLS",
]

# Every symbol include/macaq.h declares.
EXPORTED_SYMBOLS = (
    "macaq_status_str", "macaq_scale_bytes", "macaq_scale_offset", "macaq_linear_workspace_bytes",
    "macaq_gemm_workspace_bytes",
    "macaq_calibrate_scale", "macaq_fold_weights", "macaq_act_transform_quant", "macaq_w4a4_linear",
    "macaq_act_quant_plain", "macaq_mxfp4_linear", "macaq_mxfp4_gemm", "macaq_device_status",
    "macaq_grouped_workspace_bytes", "macaq_w4a4_grouped_linear", "macaq_w4a4_linear_noalloc",
    "macaq_hessian_workspace_bytes", "macaq_calib_hessian", "macaq_flip_refine_workspace_bytes",
    "macaq_flip_refine", "macaq_grouped_device_workspace_bytes", "macaq_w4a4_grouped_linear_device",
    "macaq_scales_to_tiled", "macaq_scales_to_rowmajor", "macaq_linear_multi_workspace_bytes",
    "macaq_w4a4_linear_multi", "macaq_kv4_page_bytes", "macaq_qk_norm_rope", "macaq_kv4_append",
    "macaq_kv4_gather", "macaq_kv4_attention_workspace_bytes", "macaq_kv4_attention",
)

MACAQ_OK = 0

_lock = threading.Lock()
_lib = None


class MacaqError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_str(status)} ({status})")
        self.status = status


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load (building first if absent) libmacaq.so and declare its C signatures."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        lib_path = path or _build_mod.LIB_PATH
        if path is None and not os.path.exists(lib_path):
            _build_mod.build()
        lib = ctypes.CDLL(lib_path)
        p, i64, sz, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
        lib.macaq_status_str.argtypes = [i32]
        lib.macaq_status_str.restype = ctypes.c_char_p
        lib.macaq_scale_bytes.argtypes = [i64, i64]
        lib.macaq_scale_bytes.restype = sz
        lib.macaq_scale_offset.argtypes = [i64, i64, i64]
        lib.macaq_scale_offset.restype = i64
        lib.macaq_linear_workspace_bytes.argtypes = [i64, i64, i64]
        lib.macaq_linear_workspace_bytes.restype = sz
        lib.macaq_gemm_workspace_bytes.argtypes = [i64, i64, i64]
        lib.macaq_gemm_workspace_bytes.restype = sz
        lib.macaq_calibrate_scale.argtypes = [p, i64, p, i64, i64, p, p]
        lib.macaq_fold_weights.argtypes = [p, i64, i64, p, p, p, p, p]
        lib.macaq_act_transform_quant.argtypes = [p, i64, i64, p, p, p, p]
        lib.macaq_act_quant_plain.argtypes = [p, i64, i64, p, p, p]
        lib.macaq_mxfp4_gemm.argtypes = [p, p, i64, p, p, i64, i64, p, i32, p, sz, p]
        lib.macaq_w4a4_linear.argtypes = [p, i64, i64, p, p, p, i64, p, p, sz, p]
        lib.macaq_mxfp4_linear.argtypes = [p, i64, i64, p, p, i64, p, p, sz, p]
        lib.macaq_grouped_workspace_bytes.argtypes = [p, i32, i64, i64]
        lib.macaq_grouped_workspace_bytes.restype = sz
        lib.macaq_w4a4_grouped_linear.argtypes = [p, p, i32, i64, p, p, p, i64, p, p, sz, p]
        lib.macaq_device_status.argtypes = [i32]
        lib.macaq_w4a4_linear_noalloc.argtypes = [p, i64, i64, p, p, p, i64, p, p]
        lib.macaq_hessian_workspace_bytes.argtypes = [i64, i64]
        lib.macaq_hessian_workspace_bytes.restype = sz
        lib.macaq_calib_hessian.argtypes = [p, i64, i64, p, p, p, sz, p]
        lib.macaq_flip_refine_workspace_bytes.argtypes = [i64, i64]
        lib.macaq_flip_refine_workspace_bytes.restype = sz
        lib.macaq_flip_refine.argtypes = [p, i64, i64, p, p, p, p, i64, p, p, sz, p]
        lib.macaq_scales_to_tiled.argtypes = [p, i64, i64, p, p]
        lib.macaq_scales_to_rowmajor.argtypes = [p, i64, i64, p, p]
        lib.macaq_grouped_device_workspace_bytes.argtypes = [i64, i32, i64, i64]
        lib.macaq_grouped_device_workspace_bytes.restype = sz
        lib.macaq_w4a4_grouped_linear_device.argtypes = [p, i64, p, i32, i32, i64, i64, p, p, p, i64, p, p, sz, p]
        lib.macaq_linear_multi_workspace_bytes.argtypes = [i64, i32, i64]
        lib.macaq_linear_multi_workspace_bytes.restype = sz
        lib.macaq_w4a4_linear_multi.argtypes = [p, i64, i64, i32, p, p, p, p, p, p, sz, p]
        f32 = ctypes.c_float
        lib.macaq_kv4_page_bytes.argtypes = [i32, i32]
        lib.macaq_kv4_page_bytes.restype = sz
        lib.macaq_qk_norm_rope.argtypes = [p, i64, i64, i32, i32, i32, p, p, f32, p, i64, i32, i32, p, p, p, p]
        lib.macaq_kv4_append.argtypes = [p, i64, i64, i32, i32, i32, p, p, f32, p, i64, i32, i32, p, p, i64, i32, p,
                                         p, p]
        lib.macaq_kv4_gather.argtypes = [p, i64, i32, i32, i32, p, i64, p, p, p]
        lib.macaq_kv4_attention_workspace_bytes.argtypes = [i64, i64, i32, i32, i32, i64]
        lib.macaq_kv4_attention_workspace_bytes.restype = sz
        lib.macaq_kv4_attention.argtypes = [p, i64, i64, i32, i32, i32, p, i64, i32, p, i64, i64, p, p, i64, f32, i64,
                                            p, p, p, sz, p]
        for name in ("macaq_calibrate_scale", "macaq_fold_weights", "macaq_act_transform_quant", "macaq_act_quant_plain",
                     "macaq_mxfp4_gemm", "macaq_w4a4_linear", "macaq_mxfp4_linear", "macaq_device_status",
                     "macaq_w4a4_grouped_linear", "macaq_w4a4_linear_noalloc", "macaq_calib_hessian",
                     "macaq_flip_refine", "macaq_w4a4_grouped_linear_device", "macaq_scales_to_tiled",
                     "macaq_scales_to_rowmajor", "macaq_w4a4_linear_multi", "macaq_qk_norm_rope", "macaq_kv4_append",
                     "macaq_kv4_gather", "macaq_kv4_attention"):
            getattr(lib, name).restype = i32
        if path is None:
            _lib = lib
        return lib


def status_str(status: int) -> str:
    return load_library().macaq_status_str(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != MACAQ_OK:
        raise MacaqError(status, where)


def _ptr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _stream(stream, device: torch.device) -> int:
    """The CUDA stream handle of a call whose tensors live on `device`: the given stream, which
    must belong to that device, or that device's current stream."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)  # without a Stream object around it
    _check_stream_device(stream, device)
    return stream.cuda_stream


def _check_stream_device(stream, device: torch.device) -> None:
    """A stream of another GPU would run the kernels there, on pointers into this one."""
    sdev = torch.device(stream.device)
    if sdev.type != "cuda" or sdev.index != device.index:
        raise ValueError(f"stream belongs to {sdev}, the call's tensors to {device}")


_CURRENT = contextlib.nullcontext()


def _device(device):
    """`device` made current for the library call inside (None: the current device as it is).  Nothing is
    switched where it is current already, which costs a call of a few microseconds two or three of them."""
    if device is None:
        return _CURRENT
    if isinstance(device, torch.device) and device.index == torch.cuda.current_device() and device.type == "cuda":
        return _CURRENT
    return torch.cuda.device(device)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape=None, min_numel=None, device=None) -> None:
    """Argument checks the C ABI cannot make (it sees bare pointers): a contiguous CUDA tensor of
    the right dtype and shape or size, on the device of the call's other tensors.  A buffer
    that is too small or on the wrong device would otherwise reach a kernel."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if min_numel is not None:
        _need_numel(t, name, min_numel)


def _need_numel(t: torch.Tensor, name: str, n: int) -> None:
    if t.numel() < n:
        raise ValueError(f"{name} holds {t.numel()} elements, the call needs at least {n}")


def _empty(shape, dtype: torch.dtype, device: torch.device, stream) -> torch.Tensor:
    """Memory for a call on `stream` (None: the current one).  Of another stream than the current it is that
    stream's own, so the kernels there meet neither what the current stream still does with memory given back before,
    nor what it gets when a workspace is dropped at the end of the call; and a result that the caller drops is not
    used again before the current stream is done with it, too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _check_stream_device(stream, device)
    here = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if here != stream:
        t.record_stream(here)
    return t


def scale_bytes(rows: int, K: int) -> int:
    """Size of an E8M0 scale buffer in the MMA tile layout (include/macaq.h)."""
    return int(load_library().macaq_scale_bytes(rows, K))


def scale_offset(r: int, kb: int, K: int) -> int:
    return int(load_library().macaq_scale_offset(r, kb, K))


def linear_workspace_bytes(M: int, N: int, K: int, device=None) -> int:
    """Scratch bytes macaq_w4a4_linear and macaq_mxfp4_linear need on `device` (default: the
    current CUDA device; the size depends on its SM count)."""
    with _device(device):
        return int(load_library().macaq_linear_workspace_bytes(M, N, K))


def gemm_workspace_bytes(M: int, N: int, K: int, device=None) -> int:
    """Scratch bytes of the GEMM's stream-K schedule on `device` (default: the current one)."""
    with _device(device):
        return int(load_library().macaq_gemm_workspace_bytes(M, N, K))


def macaq_scales_to_tiled(rowmajor: torch.Tensor, K: int, tiled=None, stream=None):
    """Row-major E8M0 scales uint8 [rows, K/32] -> the MMA tile layout (uint8 [scale_bytes(rows, K)])."""
    rows = rowmajor.shape[0]
    _need(rowmajor, "rowmajor", torch.uint8, (rows, K // 32))
    dev = rowmajor.device
    tiled = _empty(scale_bytes(rows, K), torch.uint8, dev, stream) if tiled is None else tiled
    _need(tiled, "tiled", torch.uint8, min_numel=scale_bytes(rows, K), device=dev)
    with torch.cuda.device(dev):
        _check(load_library().macaq_scales_to_tiled(_ptr(rowmajor), rows, K, _ptr(tiled), _stream(stream, dev)),
               "macaq_scales_to_tiled")
    return tiled


def macaq_scales_to_rowmajor(tiled: torch.Tensor, rows: int, K: int, rowmajor=None, stream=None):
    """MMA-tile-layout E8M0 scales -> row-major uint8 [rows, K/32]."""
    _need(tiled, "tiled", torch.uint8, min_numel=scale_bytes(rows, K))
    dev = tiled.device
    rowmajor = _empty((rows, K // 32), torch.uint8, dev, stream) if rowmajor is None else rowmajor
    _need(rowmajor, "rowmajor", torch.uint8, (rows, K // 32), device=dev)
    with torch.cuda.device(dev):
        _check(load_library().macaq_scales_to_rowmajor(_ptr(tiled), rows, K, _ptr(rowmajor), _stream(stream, dev)),
               "macaq_scales_to_rowmajor")
    return rowmajor


def macaq_calibrate_scale(xcal: torch.Tensor, W: torch.Tensor, s=None, stream=None):
    """Per-channel scale s (fp32 [K]) from a bf16 calibration batch [C, K] and fp32 weights [N, K]."""
    C, K = xcal.shape
    _need(xcal, "xcal", torch.bfloat16)
    dev = xcal.device
    _need(W, "W", torch.float32, device=dev)
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError("xcal and W must have the same K")
    s = _empty(K, torch.float32, W.device, stream) if s is None else s
    _need(s, "s", torch.float32, (K,), device=W.device)
    with torch.cuda.device(dev):
        _check(load_library().macaq_calibrate_scale(_ptr(xcal), C, _ptr(W), N, K, _ptr(s), _stream(stream, dev)),
               "macaq_calibrate_scale")
    return s


def macaq_fold_weights(W: torch.Tensor, s: torch.Tensor, Wq=None, Ws=None, act_mult=None, stream=None):
    """Fold diag(s) H/sqrt(32) into W (fp32 [N, K]) and RTN-quantise: (Wq, Ws, act_mult)."""
    N, K = W.shape
    _need(W, "W", torch.float32)
    dev = W.device
    _need(s, "s", torch.float32, (K,), device=dev)
    Wq = _empty((N, K // 2), torch.uint8, dev, stream) if Wq is None else Wq
    Ws = _empty(max(scale_bytes(N, K), 1), torch.uint8, dev, stream) if Ws is None else Ws
    act_mult = _empty(K, torch.float32, dev, stream) if act_mult is None else act_mult
    _need(Wq, "Wq", torch.uint8, (N, K // 2), device=dev)
    _need(Ws, "Ws", torch.uint8, min_numel=scale_bytes(N, K), device=dev)
    _need(act_mult, "act_mult", torch.float32, (K,), device=dev)
    with torch.cuda.device(dev):
        _check(load_library().macaq_fold_weights(_ptr(W), N, K, _ptr(s), _ptr(Wq), _ptr(Ws), _ptr(act_mult),
                                                 _stream(stream, dev)), "macaq_fold_weights")
    return Wq, Ws, act_mult


def macaq_act_transform_quant(x: torch.Tensor, act_mult: torch.Tensor, Aq=None, As=None, stream=None):
    """Scale, FWHT-32 and MXFP4-quantise bf16 activations [M, K]: (Aq, As)."""
    M, K = x.shape
    _need(x, "x", torch.bfloat16)
    dev = x.device
    _need(act_mult, "act_mult", torch.float32, (K,), device=dev)
    Aq = _empty((M, K // 2), torch.uint8, dev, stream) if Aq is None else Aq
    As = _empty(max(scale_bytes(M, K), 1), torch.uint8, dev, stream) if As is None else As
    _need(Aq, "Aq", torch.uint8, (M, K // 2), device=dev)
    _need(As, "As", torch.uint8, min_numel=scale_bytes(M, K), device=dev)
    with torch.cuda.device(dev):
        _check(load_library().macaq_act_transform_quant(_ptr(x), M, K, _ptr(act_mult), _ptr(Aq), _ptr(As),
                                                        _stream(stream, dev)), "macaq_act_transform_quant")
    return Aq, As


def macaq_act_quant_plain(x: torch.Tensor, Aq=None, As=None, stream=None):
    """Plain MXFP4 quantisation of bf16 activations (no scale, no transform): (Aq, As)."""
    M, K = x.shape
    _need(x, "x", torch.bfloat16)
    dev = x.device
    Aq = _empty((M, K // 2), torch.uint8, dev, stream) if Aq is None else Aq
    As = _empty(max(scale_bytes(M, K), 1), torch.uint8, dev, stream) if As is None else As
    _need(Aq, "Aq", torch.uint8, (M, K // 2), device=dev)
    _need(As, "As", torch.uint8, min_numel=scale_bytes(M, K), device=dev)
    with torch.cuda.device(dev):
        _check(load_library().macaq_act_quant_plain(_ptr(x), M, K, _ptr(Aq), _ptr(As), _stream(stream, dev)),
               "macaq_act_quant_plain")
    return Aq, As


def macaq_mxfp4_gemm(Aq, As, Wq, Ws, M: int, N: int, K: int, y=None, out_fp32: bool = False, workspace=None,
                     data_parallel: bool = False, stream=None):
    """y = dec(A) dec(W)^T from MXFP4 operands; bf16 (default) or fp32 [M, N].  A stream-K
    workspace is allocated when not given (the schedule macaq_w4a4_linear uses);
    data_parallel=True passes none (data-parallel schedule)."""
    _need(Aq, "Aq", torch.uint8, (M, K // 2))
    dev = Aq.device
    _need(Wq, "Wq", torch.uint8, (N, K // 2), device=dev)
    _need(As, "As", torch.uint8, min_numel=scale_bytes(M, K), device=dev)
    _need(Ws, "Ws", torch.uint8, min_numel=scale_bytes(N, K), device=dev)
    dt = torch.float32 if out_fp32 else torch.bfloat16
    y = _empty((M, N), dt, dev, stream) if y is None else y
    _need(y, "y", dt, (M, N), device=dev)
    if data_parallel:
        workspace = None
    elif workspace is None:
        workspace = _empty(max(gemm_workspace_bytes(M, N, K, dev), 1), torch.uint8, dev, stream)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, device=dev)
    with torch.cuda.device(dev):
        _check(load_library().macaq_mxfp4_gemm(_ptr(Aq), _ptr(As), M, _ptr(Wq), _ptr(Ws), N, K, _ptr(y),
                                               1 if out_fp32 else 0, _ptr(workspace),
                                               0 if workspace is None else workspace.numel(), _stream(stream, dev)),
               "macaq_mxfp4_gemm")
    return y


def macaq_w4a4_linear(x: torch.Tensor, act_mult: torch.Tensor, Wq: torch.Tensor, Ws: torch.Tensor, N: int,
                      y=None, workspace=None, stream=None):
    """y = x W^T through the online transform, MXFP4 quantisation and the W4A4 GEMM (bf16 [M, N])."""
    M, K = x.shape
    _need(x, "x", torch.bfloat16)
    dev = x.device
    _need(act_mult, "act_mult", torch.float32, (K,), device=dev)
    _need(Wq, "Wq", torch.uint8, (N, K // 2), device=dev)
    _need(Ws, "Ws", torch.uint8, min_numel=scale_bytes(N, K), device=dev)
    y = _empty((M, N), torch.bfloat16, dev, stream) if y is None else y
    _need(y, "y", torch.bfloat16, (M, N), device=dev)
    need = linear_workspace_bytes(M, N, K, dev)
    workspace = _empty(need, torch.uint8, dev, stream) if workspace is None else workspace
    _need(workspace, "workspace", torch.uint8, device=dev)
    with torch.cuda.device(dev):
        _check(load_library().macaq_w4a4_linear(_ptr(x), M, K, _ptr(act_mult), _ptr(Wq), _ptr(Ws), N, _ptr(y),
                                                _ptr(workspace), workspace.numel(), _stream(stream, dev)),
               "macaq_w4a4_linear")
    return y


def macaq_mxfp4_linear(x: torch.Tensor, Wq: torch.Tensor, Ws: torch.Tensor, N: int, y=None, workspace=None,
                       stream=None):
    """Plain MXFP4 linear (no scale, no transform): the baseline of the transform's overhead."""
    M, K = x.shape
    _need(x, "x", torch.bfloat16)
    dev = x.device
    _need(Wq, "Wq", torch.uint8, (N, K // 2), device=dev)
    _need(Ws, "Ws", torch.uint8, min_numel=scale_bytes(N, K), device=dev)
    y = _empty((M, N), torch.bfloat16, dev, stream) if y is None else y
    _need(y, "y", torch.bfloat16, (M, N), device=dev)
    need = linear_workspace_bytes(M, N, K, dev)
    workspace = _empty(need, torch.uint8, dev, stream) if workspace is None else workspace
    _need(workspace, "workspace", torch.uint8, device=dev)
    with torch.cuda.device(dev):
        _check(load_library().macaq_mxfp4_linear(_ptr(x), M, K, _ptr(Wq), _ptr(Ws), N, _ptr(y), _ptr(workspace),
                                                 workspace.numel(), _stream(stream, dev)), "macaq_mxfp4_linear")
    return y


def linear_multi_workspace_bytes(M: int, G: int, K: int, device=None) -> int:
    """Scratch bytes macaq_w4a4_linear_multi needs for G linears on M tokens (default device: the
    current one; the size depends on its SM count)."""
    with _device(device):
        return int(load_library().macaq_linear_multi_workspace_bytes(M, G, K))


def macaq_w4a4_linear_multi(x: torch.Tensor, act_mult, Wq: torch.Tensor, Ws: torch.Tensor, Ns, y=None,
                            workspace=None, stream=None):
    """G linears on the same x [M, K] bf16 (the q, k and v projections, or gate and up), each its own
    folded layer: act_mult fp32 [G, K] (torch.stack of the folds' multipliers; None: plain MXFP4),
    Wq [sum Ns, K/2] and Ws (torch.cat of the folds' codes and scales, in the same order), Ns the
    output features of each (multiples of 128).  Returns y bf16 [M, sum Ns]: linear g's outputs in
    columns sum(Ns[:g]) .. sum(Ns[:g + 1]) - 1."""
    import numpy as np
    M, K = x.shape
    n = np.ascontiguousarray(np.asarray(list(Ns), dtype=np.int64))
    G, Nt = len(n), int(n.sum())
    _need(x, "x", torch.bfloat16)
    dev = x.device
    if act_mult is not None:
        _need(act_mult, "act_mult", torch.float32, (G, K), device=dev)
    _need(Wq, "Wq", torch.uint8, (Nt, K // 2), device=dev)
    _need(Ws, "Ws", torch.uint8, min_numel=sum(scale_bytes(int(v), K) for v in n), device=dev)
    y = _empty((M, Nt), torch.bfloat16, dev, stream) if y is None else y
    _need(y, "y", torch.bfloat16, (M, Nt), device=dev)
    need = linear_multi_workspace_bytes(M, G, K, dev)
    workspace = _empty(need, torch.uint8, dev, stream) if workspace is None else workspace
    _need(workspace, "workspace", torch.uint8, device=dev)
    with torch.cuda.device(dev):
        _check(load_library().macaq_w4a4_linear_multi(_ptr(x), M, K, G, _ptr(act_mult), _ptr(Wq), _ptr(Ws),
                                                      ctypes.c_void_p(n.ctypes.data), _ptr(y), _ptr(workspace),
                                                      workspace.numel(), _stream(stream, dev)),
               "macaq_w4a4_linear_multi")
    return y


def _counts_array(counts):
    import numpy as np
    c = np.ascontiguousarray(np.asarray(counts, dtype=np.int64))
    return c, ctypes.c_void_p(c.ctypes.data)


def grouped_workspace_bytes(counts, N: int, K: int) -> int:
    """Scratch bytes macaq_w4a4_grouped_linear needs for these per-expert token counts."""
    c, cp = _counts_array(counts)
    return int(load_library().macaq_grouped_workspace_bytes(cp, len(c), N, K))


def macaq_w4a4_grouped_linear(x: torch.Tensor, counts, act_mult, Wq: torch.Tensor, Ws: torch.Tensor, N: int,
                              y=None, workspace=None, stream=None):
    """Grouped (mixture-of-experts) linear: x [T, K] bf16 grouped by expert, counts = tokens per
    expert (host ints), act_mult fp32 [E, K] (None: plain MXFP4), Wq [E, N, K/2], Ws the experts'
    scale buffers concatenated.  Returns y bf16 [T, N]."""
    T, K = x.shape
    c, cp = _counts_array(counts)
    E = len(c)
    if int(c.sum()) != T:
        raise ValueError("counts must sum to the rows of x")
    _need(x, "x", torch.bfloat16)
    dev = x.device
    if act_mult is not None:
        _need(act_mult, "act_mult", torch.float32, (E, K), device=dev)
    _need(Wq, "Wq", torch.uint8, (E, N, K // 2), device=dev)
    _need(Ws, "Ws", torch.uint8, min_numel=E * scale_bytes(N, K), device=dev)
    y = _empty((T, N), torch.bfloat16, dev, stream) if y is None else y
    _need(y, "y", torch.bfloat16, (T, N), device=dev)
    need = max(grouped_workspace_bytes(c, N, K), 1)
    workspace = _empty(need, torch.uint8, dev, stream) if workspace is None else workspace
    _need(workspace, "workspace", torch.uint8, device=dev)
    with torch.cuda.device(dev):
        _check(load_library().macaq_w4a4_grouped_linear(_ptr(x), cp, E, K, _ptr(act_mult), _ptr(Wq), _ptr(Ws), N,
                                                        _ptr(y), _ptr(workspace), workspace.numel(), _stream(stream, dev)),
               "macaq_w4a4_grouped_linear")
    return y


def grouped_device_workspace_bytes(T: int, E: int, N: int, K: int, device=None) -> int:
    """Scratch bytes macaq_w4a4_grouped_linear_device needs for T routed rows over E experts."""
    with _device(device):
        return int(load_library().macaq_grouped_device_workspace_bytes(T, E, N, K))


def macaq_w4a4_grouped_linear_device(x: torch.Tensor, counts: torch.Tensor, act_mult, Wq: torch.Tensor,
                                     Ws: torch.Tensor, N: int, capacity: int = 0, y=None, workspace=None, stream=None):
    """Grouped (mixture-of-experts) linear with the per-expert token counts on the DEVICE (int32 or
    int64 CUDA tensor [E], e.g. straight from a GPU router): no host copy, no synchronisation.  x
    [T, K] bf16 grouped by expert, act_mult fp32 [E, K] (None: plain MXFP4), Wq [E, N, K/2], Ws the
    experts' scale buffers concatenated; capacity = the most rows any expert may have (0: T), which
    picks the kernels; rows past it are not computed (reported as MACAQ_ECOUNTS).  Returns y bf16
    [T, N]."""
    T, K = x.shape
    _need(x, "x", torch.bfloat16)
    dev = x.device
    if counts.dtype not in (torch.int32, torch.int64):
        raise ValueError("counts must be int32 or int64")
    _need(counts, "counts", counts.dtype, device=dev)
    E = counts.numel()
    if act_mult is not None:
        _need(act_mult, "act_mult", torch.float32, (E, K), device=dev)
    _need(Wq, "Wq", torch.uint8, (E, N, K // 2), device=dev)
    _need(Ws, "Ws", torch.uint8, min_numel=E * scale_bytes(N, K), device=dev)
    y = _empty((T, N), torch.bfloat16, dev, stream) if y is None else y
    _need(y, "y", torch.bfloat16, (T, N), device=dev)
    need = grouped_device_workspace_bytes(T, E, N, K, dev)
    if need == 0:
        raise ValueError("shape not supported by the grouped linear (1 <= E <= 128, N % 128 == 0, T >= 1)")
    workspace = _empty(need, torch.uint8, dev, stream) if workspace is None else workspace
    _need(workspace, "workspace", torch.uint8, min_numel=need, device=dev)
    with torch.cuda.device(dev):
        _check(load_library().macaq_w4a4_grouped_linear_device(
            _ptr(x), T, _ptr(counts), counts.element_size(), E, int(capacity), K, _ptr(act_mult), _ptr(Wq), _ptr(Ws), N,
            _ptr(y),
            _ptr(workspace), workspace.numel(), _stream(stream, dev)), "macaq_w4a4_grouped_linear_device")
    return y


NOALLOC_SCRATCH_BYTES = 32 << 20  # MACAQ_NOALLOC_SCRATCH_BYTES of include/macaq.h


def macaq_w4a4_linear_noalloc(x: torch.Tensor, act_mult: torch.Tensor, Wq: torch.Tensor, Ws: torch.Tensor,
                              N: int, y=None, stream=None):
    """macaq_w4a4_linear without a workspace: for callers that cannot allocate device memory,
    the library keeps the activation scratch in its own static 32 MiB device array (see
    include/macaq.h for the limit and the ordering rule).  Only y is allocated here, and
    only when the caller does not pass it."""
    M, K = x.shape
    _need(x, "x", torch.bfloat16)
    dev = x.device
    _need(act_mult, "act_mult", torch.float32, (K,), device=dev)
    _need(Wq, "Wq", torch.uint8, (N, K // 2), device=dev)
    _need(Ws, "Ws", torch.uint8, min_numel=scale_bytes(N, K), device=dev)
    y = _empty((M, N), torch.bfloat16, dev, stream) if y is None else y
    _need(y, "y", torch.bfloat16, (M, N), device=dev)
    with torch.cuda.device(dev):
        _check(load_library().macaq_w4a4_linear_noalloc(_ptr(x), M, K, _ptr(act_mult), _ptr(Wq), _ptr(Ws), N, _ptr(y),
                                                        _stream(stream, dev)), "macaq_w4a4_linear_noalloc")
    return y


def macaq_calib_hessian(xcal: torch.Tensor, act_mult: torch.Tensor, Hs=None, workspace=None, stream=None):
    """Hs = Xt^T Xt (fp64 [K, K]) of a bf16 calibration batch [C, K] after the online transform with
    the layer's multipliers (Flip-Refinement's Hessian)."""
    C, K = xcal.shape
    _need(xcal, "xcal", torch.bfloat16)
    dev = xcal.device
    _need(act_mult, "act_mult", torch.float32, (K,), device=dev)
    Hs = _empty((K, K), torch.float64, dev, stream) if Hs is None else Hs
    _need(Hs, "Hs", torch.float64, (K, K), device=dev)
    need = int(load_library().macaq_hessian_workspace_bytes(C, K))
    workspace = _empty(max(need, 1), torch.uint8, dev, stream) if workspace is None else workspace
    _need(workspace, "workspace", torch.uint8, min_numel=need, device=dev)
    with torch.cuda.device(dev):
        _check(load_library().macaq_calib_hessian(_ptr(xcal), C, K, _ptr(act_mult), _ptr(Hs), _ptr(workspace),
                                                  workspace.numel(), _stream(stream, dev)), "macaq_calib_hessian")
    return Hs


def macaq_flip_refine(W: torch.Tensor, s: torch.Tensor, Hs: torch.Tensor, Wq: torch.Tensor, Ws: torch.Tensor,
                      max_moves: int, moves=None, workspace=None, stream=None):
    """Flip-Refinement of the round-to-nearest codes Wq [N, K/2] (from macaq_fold_weights of W and s)
    in place, scales Ws kept; returns the int32 moves applied per row."""
    N, K = W.shape
    _need(W, "W", torch.float32)
    dev = W.device
    _need(s, "s", torch.float32, (K,), device=dev)
    _need(Hs, "Hs", torch.float64, (K, K), device=dev)
    _need(Wq, "Wq", torch.uint8, (N, K // 2), device=dev)
    _need(Ws, "Ws", torch.uint8, min_numel=scale_bytes(N, K), device=dev)
    moves = _empty(N, torch.int32, dev, stream) if moves is None else moves
    _need(moves, "moves", torch.int32, (N,), device=dev)
    need = int(load_library().macaq_flip_refine_workspace_bytes(N, K))
    if need == 0:
        raise ValueError(f"K={K} is not supported by macaq_flip_refine (K <= 12288, K % 32 == 0)")
    workspace = _empty(need, torch.uint8, dev, stream) if workspace is None else workspace
    _need(workspace, "workspace", torch.uint8, min_numel=need, device=dev)
    with torch.cuda.device(dev):
        _check(load_library().macaq_flip_refine(_ptr(W), N, K, _ptr(s), _ptr(Hs), _ptr(Wq), _ptr(Ws), int(max_moves),
                                                _ptr(moves), _ptr(workspace), workspace.numel(),
                                                _stream(stream, dev)), "macaq_flip_refine")
    return moves


def _out(t, name: str, shape, like: torch.Tensor, stream) -> torch.Tensor:
    """A bf16 result on the device of `like`: the caller's tensor after its checks, or a new one."""
    if t is None:
        return _empty(shape, torch.bfloat16, like.device, stream)
    _need(t, name, torch.bfloat16, shape, device=like.device)
    return t


def _need_rows(t: torch.Tensor, name: str, width: int, device=None) -> int:
    """A bf16 CUDA tensor [T, >= width] whose rows are contiguous and may lie further apart (a slice of
    the columns of a stacked output); returns the distance between rows in elements."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, the call's other tensors on {device}")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 2 or t.shape[1] < width:
        raise ValueError(f"{name} must have shape (T, {width} or more), got {tuple(t.shape)}")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    if ld < t.shape[1]:
        raise ValueError(f"the rows of {name} overlap")
    if ld % 8:
        if t.shape[0] > 1:
            raise ValueError(f"the rows of {name} must lie a multiple of 8 elements apart, got {ld}")
        ld += 8 - ld % 8  # a single row: nothing lies behind it
    return ld


def _rope_args(rope, positions, head_dim: int, T: int, device):
    """(rope_rows, rope_dim) after the checks of a rotation table and positions."""
    if rope is None:
        return 0, 0
    _need(rope, "rope", torch.float32, device=device)
    if rope.dim() != 2 or rope.shape[1] not in (head_dim, head_dim // 2):
        raise ValueError(f"rope must have shape (positions, {head_dim} or {head_dim // 2}), got {tuple(rope.shape)}")
    if positions is None:
        raise ValueError("rope needs positions")
    _need(positions, "positions", torch.int64, (T,), device=device)
    return rope.shape[0], rope.shape[1]


def kv4_page_bytes(page_size: int, head_dim: int) -> int:
    """Bytes of one page of one kv head: allocate the cache as uint8 [pages, Hk, kv4_page_bytes(...)]."""
    return int(load_library().macaq_kv4_page_bytes(page_size, head_dim))


def _need_cache(cache, page_size: int, head_dim: int, device=None):
    """(pages, kv heads) of a cache tensor."""
    if page_size not in (16, 32, 64, 128) or head_dim not in (64, 128):
        raise ValueError(f"page_size must be 16, 32, 64 or 128 and head_dim 64 or 128, got {page_size}, {head_dim}")
    pb = page_size * head_dim * 17 // 16  # kv4_page_bytes
    _need(cache, "cache", torch.uint8, device=device)
    if cache.dim() != 3 or cache.shape[2] != pb:
        raise ValueError(f"cache must have shape (pages, kv heads, {pb}), got {tuple(cache.shape)}")
    return cache.shape[0], cache.shape[1]


def macaq_qk_norm_rope(qkv: torch.Tensor, Hq: int, Hk: int, head_dim: int, rope=None, positions=None, q_weight=None,
                       k_weight=None, eps: float = 1e-6, interleaved: bool = False, q=None, k=None, stream=None):
    """Per-head norm (weights fp32 [head_dim], None: none) and position rotation of the query and key
    heads of qkv (bf16 [T, (Hq + Hk) * head_dim or more], e.g. the stacked q/k/v output) in one pass.
    rope fp32 [P, R]: R/2 cosines then R/2 sines of each position, R = head_dim or head_dim/2; positions
    int64 [T].  Returns (q [T, Hq, head_dim], k [T, Hk, head_dim]) in bf16."""
    ld = _need_rows(qkv, "qkv", (Hq + Hk) * head_dim)
    dev, T = qkv.device, qkv.shape[0]
    rows, R = _rope_args(rope, positions, head_dim, T, dev)
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _need(w, name, torch.float32, (head_dim,), device=dev)
    q = _out(q, "q", (T, Hq, head_dim), qkv, stream)
    k = _out(k, "k", (T, Hk, head_dim), qkv, stream)
    with _device(dev):
        _check(load_library().macaq_qk_norm_rope(_ptr(qkv), T, ld, Hq, Hk, head_dim, _ptr(q_weight), _ptr(k_weight),
                                                 eps, _ptr(rope), rows, R, 1 if interleaved else 0, _ptr(positions),
                                                 _ptr(q), _ptr(k), _stream(stream, dev)), "macaq_qk_norm_rope")
    return q, k


def macaq_kv4_append(qkv: torch.Tensor, Hq: int, Hk: int, head_dim: int, cache: torch.Tensor, page_size: int,
                     slots: torch.Tensor, rope=None, positions=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                     interleaved: bool = False, q=None, stream=None):
    """Stores the keys and values of qkv (bf16 [T, (Hq + 2 Hk) * head_dim or more]) in the paged MXFP4
    cache (uint8 [pages, Hk, kv4_page_bytes(page_size, head_dim)]) at slots (int64 [T], page * page_size
    + place; negative: padding, not stored), with norm and rotation (as macaq_qk_norm_rope), transform and
    quantisation on the way.  Returns the normed and rotated queries, bf16 [T, Hq, head_dim] (Hq = 0:
    None)."""
    ld = _need_rows(qkv, "qkv", (Hq + 2 * Hk) * head_dim)
    dev, T = qkv.device, qkv.shape[0]
    pages, heads = _need_cache(cache, page_size, head_dim, dev)
    if heads != Hk:
        raise ValueError(f"cache holds {heads} kv heads, the call names {Hk}")
    _need(slots, "slots", torch.int64, (T,), device=dev)
    rows, R = _rope_args(rope, positions, head_dim, T, dev)
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _need(w, name, torch.float32, (head_dim,), device=dev)
    if Hq:
        q = _out(q, "q", (T, Hq, head_dim), qkv, stream)
    with _device(dev):
        _check(load_library().macaq_kv4_append(_ptr(qkv), T, ld, Hq, Hk, head_dim, _ptr(q_weight), _ptr(k_weight), eps,
                                               _ptr(rope), rows, R, 1 if interleaved else 0, _ptr(positions),
                                               _ptr(cache), pages, page_size, _ptr(slots), _ptr(q) if Hq else None,
                                               _stream(stream, dev)), "macaq_kv4_append")
    return q if Hq else None


def macaq_kv4_gather(cache: torch.Tensor, head_dim: int, page_size: int, slots: torch.Tensor, k=None, v=None,
                     stream=None):
    """Reads tokens back from the cache: (k, v) bf16 [T, Hk, head_dim], the values it holds for slots
    (int64 [T]); zeros for negative slots."""
    pages, Hk = _need_cache(cache, page_size, head_dim)
    dev = cache.device
    _need(slots, "slots", torch.int64, device=dev)
    T = slots.numel()
    if slots.dim() != 1:
        raise ValueError(f"slots must have shape ({T},), got {tuple(slots.shape)}")
    k = _out(k, "k", (T, Hk, head_dim), cache, stream)
    v = _out(v, "v", (T, Hk, head_dim), cache, stream)
    with _device(dev):
        _check(load_library().macaq_kv4_gather(_ptr(cache), pages, page_size, Hk, head_dim, _ptr(slots), T, _ptr(k),
                                               _ptr(v), _stream(stream, dev)), "macaq_kv4_gather")
    return k, v


def kv4_attention_workspace_bytes(T: int, B: int, Hq: int, Hk: int, head_dim: int, max_q: int, device=None) -> int:
    """Scratch bytes macaq_kv4_attention needs for T query rows of B sequences on `device` (default: the
    current one; the size depends on its SM count)."""
    with _device(device):
        return int(load_library().macaq_kv4_attention_workspace_bytes(T, B, Hq, Hk, head_dim, max_q))


def macaq_kv4_attention(q: torch.Tensor, cache: torch.Tensor, page_size: int, tables: torch.Tensor,
                        kv_lens: torch.Tensor, cu_q=None, max_q: int = 1, scale: float | None = None, window: int = 0,
                        out=None, lse=None, workspace=None, stream=None):
    """Attention of q (bf16 [T, Hq, head_dim], rows may lie further apart) over the paged MXFP4 cache,
    causal: tables int32 [B, pages of a sequence], kv_lens int32 [B] keys of each sequence, cu_q int32
    [B + 1] its query rows (None: one query each), max_q the most queries of any sequence, scale (default
    head_dim ** -0.5), window (0: none) the newest keys a query sees.  Returns out bf16 [T, Hq, head_dim];
    lse, if given (fp32 [T, Hq]), receives the logarithms of the softmax sums."""
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a CUDA tensor of shape (T, heads, head_dim)")
    T, Hq, D = q.shape
    if q.is_cuda and q.dtype == torch.bfloat16 and q.is_contiguous():
        ld = Hq * D
    else:
        if T and (q.stride(2) != 1 or (Hq > 1 and q.stride(1) != D)):
            raise ValueError("the rows of q must be contiguous")
        ld = _need_rows(q.as_strided((T, Hq * D), (q.stride(0), 1)), "q", Hq * D)
    dev = q.device
    pages, Hk = _need_cache(cache, page_size, D, dev)
    if not isinstance(tables, torch.Tensor) or tables.dim() != 2:
        raise ValueError("tables must be a CUDA tensor of shape (sequences, pages)")
    B, width = tables.shape
    _need(tables, "tables", torch.int32, device=dev)
    _need(kv_lens, "kv_lens", torch.int32, (B,), device=dev)
    if cu_q is not None:
        _need(cu_q, "cu_q", torch.int32, (B + 1,), device=dev)
    elif B != T or max_q != 1:
        raise ValueError("without cu_q every sequence has one query: T = B and max_q = 1")
    out = _out(out, "out", (T, Hq, D), q, stream)
    if lse is not None:
        _need(lse, "lse", torch.float32, (T, Hq), device=dev)
    need = kv4_attention_workspace_bytes(T, B, Hq, Hk, D, max_q, dev)
    if need == 0:
        raise ValueError("shape not supported by the attention (Hq a multiple of Hk, at most 1024; max_q >= 1)")
    if workspace is None:
        workspace = _empty(need, torch.uint8, dev, stream)
    else:
        _need(workspace, "workspace", torch.uint8, min_numel=need, device=dev)
    with _device(dev):
        _check(load_library().macaq_kv4_attention(
            _ptr(q), T, ld, Hq, Hk, D, _ptr(cache), pages, page_size, _ptr(tables), B, width, _ptr(kv_lens), _ptr(cu_q),
            int(max_q), D ** -0.5 if scale is None else float(scale), int(window), _ptr(out), _ptr(lse),
            _ptr(workspace), workspace.numel(), _stream(stream, dev)), "macaq_kv4_attention")
    return out


def macaq_device_status(clear: bool = False) -> int:
    """MACAQ_OK, or the last device-side event: MACAQ_ETIMEOUT (a bounded wait gave up), MACAQ_ECOUNTS
    (device routing counts were corrected) or MACAQ_EINDEX (an index of a cache call was out of range).
    Synchronises."""
    return int(load_library().macaq_device_status(1 if clear else 0))
