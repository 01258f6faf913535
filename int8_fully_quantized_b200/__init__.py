"""Python binding of the per-block INT8 data-flow library (``libjetfire.so``, C ABI in
``include/jetfire.h``).

The binding only marshals arguments: tensors are torch CUDA tensors (torch provides device memory
and streams), every step of the computation runs in the library's sm_100a kernels. There is no
fallback: importing works without a GPU (so the C ABI can be inspected), but every compute call
raises if the library is missing or no B200 is current.

A quantized tensor is a pair ``QTensor(q, s)``: ``q`` int8 [rows, cols] codes and ``s`` fp32
[rows/32, cols/32] block scales, both contiguous on the device. Block (I, J) covers rows
32I..32I+31 and columns 32J..32J+31 (Jetfire summary, "Approach": per-block scales, B = 32).
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
import os
from typing import NamedTuple, Optional

import torch

from . import build_lib
from .build_lib import LIB_PATH

__all__ = [
    "QTensor", "JetfireError", "load_library", "empty_qtensor", "EXPORTED_SYMBOLS", "JF_F32", "JF_BF16", "JF_F16",
    "GRANULARITY", "ACTIVATIONS", "ROPE_LAYOUTS", "QKVRope",
    # C ABI, one wrapper per entry point
    "jf_quantize_block", "jf_dequantize_block", "jf_linear_fwd", "jf_linear_fwd_gelu", "jf_linear_dgrad",
    "jf_linear_wgrad", "jf_gelu_i8", "jf_layernorm_i8", "jf_gelu_i8_bwd", "jf_layernorm_i8_bwd",
    "jf_quantize_block_rowstats", "jf_layernorm_i8_rowstats", "quantize_block_rowstats", "layernorm_i8_rowstats",
    "jf_layernorm_i8_bwd_workspace_bytes", "jf_layernorm_i8_bwd_noalloc", "jf_quantize_granular",
    "jf_dequantize_granular", "jf_quantization_error", "jf_granular_scale_count", "jf_mx_quantize",
    "jf_mx_linear_fwd", "jf_gemm_i8_s32", "jf_selftest_wait_timeout", "jf_strerror",
    "jf_device_status", "jf_sm_count", "jf_linear_fwd_epilogue", "jf_linear_dgrad_epilogue", "jf_bias_grad",
    "jf_rope_table", "jf_qkv_rope_fwd", "jf_qkv_rope_bwd", "jf_qkv_rope_bwd_workspace_bytes",
    # allocating helpers
    "quantize_block", "dequantize_block", "linear_fwd", "linear_fwd_gelu", "linear_dgrad", "linear_wgrad",
    "gelu_i8", "layernorm_i8", "gelu_i8_bwd", "layernorm_i8_bwd", "quantize_granular", "quantization_mse",
    "mx_quantize", "mx_linear_fwd", "linear_fwd_epilogue", "linear_dgrad_epilogue", "bias_grad", "rope_frequencies",
    "rope_table", "qkv_rope", "qkv_rope_bwd",
]

JF_F32, JF_BF16, JF_F16 = 0, 1, 2
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
ROPE_LAYOUTS = {"half": 0, "interleaved": 1}
GRANULARITY = {"block": 0, "token": 1, "channel": 2, "tensor": 3}
_DTYPES = {torch.float32: JF_F32, torch.bfloat16: JF_BF16, torch.float16: JF_F16}

EXPORTED_SYMBOLS = (
    "jf_quantize_block", "jf_quantize_block_rowstats", "jf_layernorm_i8_rowstats", "jf_dequantize_block", "jf_linear_fwd", "jf_linear_fwd_gelu", "jf_linear_dgrad",
    "jf_linear_wgrad",
    "jf_gelu_i8", "jf_layernorm_i8", "jf_gelu_i8_bwd", "jf_layernorm_i8_bwd", "jf_layernorm_i8_bwd_workspace_bytes",
    "jf_layernorm_i8_bwd_noalloc", "jf_quantize_granular", "jf_dequantize_granular", "jf_quantization_error",
    "jf_granular_scale_count", "jf_mx_quantize", "jf_mx_linear_fwd", "jf_gemm_i8_s32", "jf_selftest_wait_timeout",
    "jf_linear_fwd_epilogue", "jf_linear_dgrad_epilogue", "jf_bias_grad", "jf_rope_table", "jf_qkv_rope_fwd",
    "jf_qkv_rope_bwd", "jf_qkv_rope_bwd_workspace_bytes",
    "jf_strerror",
    "jf_device_status",
    "jf_sm_count",
)


class _CQ(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class _Q(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class _Matrix(ctypes.Structure):   # jf_cmatrix and jf_matrix
    _fields_ = [("p", ctypes.c_void_p), ("dt", ctypes.c_int), ("ld", ctypes.c_int64)]


class _Heads(ctypes.Structure):    # jf_cheads and jf_heads
    _fields_ = [("p", ctypes.c_void_p), ("stride_b", ctypes.c_int64), ("stride_s", ctypes.c_int64),
                ("stride_h", ctypes.c_int64)]


class _Rope(ctypes.Structure):     # jf_qkv_rope
    _fields_ = [("batch", ctypes.c_int64), ("seq", ctypes.c_int64), ("q_heads", ctypes.c_int64),
                ("kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("rot_dim", ctypes.c_int64),
                ("layout", ctypes.c_int), ("cos_table", ctypes.c_void_p), ("sin_table", ctypes.c_void_p),
                ("table_len", ctypes.c_int64), ("positions", ctypes.c_void_p), ("gamma_q", ctypes.c_void_p),
                ("gamma_k", ctypes.c_void_p), ("eps", ctypes.c_float)]


class JetfireError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {jf_strerror(status)} (status {status})")


_lib = None


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load ``libjetfire.so`` (built by ``build_lib``) once and declare its prototypes."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or os.environ.get("JETFIRE_LIB", LIB_PATH)
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m int8_fully_quantized_b200.build_lib`")
    if path == LIB_PATH and not build_lib.up_to_date():
        raise RuntimeError(f"{path} was not built from the current sources: rebuild it with "
                           "`python -m int8_fully_quantized_b200.build_lib`")
    lib = ctypes.CDLL(path)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    lib.jf_quantize_block.argtypes = [vp, i32, i64, i64, vp, vp, vp]
    lib.jf_dequantize_block.argtypes = [vp, vp, i64, i64, vp, i32, vp]
    for name in ("jf_linear_fwd", "jf_linear_dgrad", "jf_linear_wgrad"):
        getattr(lib, name).argtypes = [_CQ, _CQ, _Q, vp, vp]
    lib.jf_linear_fwd_gelu.argtypes = [_CQ, _CQ, _Q, _Q, vp]
    lib.jf_gelu_i8.argtypes = [_CQ, _Q, vp]
    lib.jf_layernorm_i8.argtypes = [_CQ, vp, vp, ctypes.c_float, _Q, vp]
    lib.jf_quantize_block_rowstats.argtypes = [vp, i32, i64, i64, vp, vp, vp, vp]
    lib.jf_layernorm_i8_rowstats.argtypes = [_CQ, vp, vp, vp, ctypes.c_float, _Q, vp]
    lib.jf_gelu_i8_bwd.argtypes = [_CQ, _CQ, _Q, vp]
    lib.jf_layernorm_i8_bwd.argtypes = [_CQ, _CQ, vp, ctypes.c_float, _Q, vp, vp, vp, i64, vp]
    lib.jf_layernorm_i8_bwd_workspace_bytes.argtypes = [i64, i64]
    lib.jf_layernorm_i8_bwd_noalloc.argtypes = [_CQ, _CQ, vp, ctypes.c_float, _Q, vp, vp, vp]
    lib.jf_quantize_granular.argtypes = [vp, i32, i64, i64, i32, vp, vp, vp]
    lib.jf_dequantize_granular.argtypes = [vp, vp, i64, i64, i32, vp, i32, vp]
    lib.jf_quantization_error.argtypes = [vp, i32, vp, vp, i64, i64, i32, vp, vp]
    lib.jf_granular_scale_count.argtypes = [i64, i64, i32]
    lib.jf_mx_quantize.argtypes = [vp, i32, i64, i64, vp, vp, vp]
    lib.jf_mx_linear_fwd.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, vp]
    lib.jf_gemm_i8_s32.argtypes = [vp, vp, vp, i64, i64, i64, vp]
    lib.jf_selftest_wait_timeout.argtypes = [i64, vp]
    lib.jf_linear_fwd_epilogue.argtypes = [_CQ, _CQ, vp, i32, _CQ, _Matrix, _Q, _Matrix, _Q, vp]
    lib.jf_linear_dgrad_epilogue.argtypes = [_CQ, _CQ, _CQ, i32, _CQ, _Matrix, _Q, _Matrix, vp]
    lib.jf_bias_grad.argtypes = [_CQ, vp, vp]
    lib.jf_rope_table.argtypes = [ctypes.POINTER(ctypes.c_double), i64, ctypes.c_double, i64, vp, vp, vp]
    rope = ctypes.POINTER(_Rope)
    lib.jf_qkv_rope_fwd.argtypes = [_CQ, rope, _Heads, _Heads, _Heads, i32, vp]
    lib.jf_qkv_rope_bwd.argtypes = [_CQ, rope, _Heads, _Heads, _Heads, i32, _Q, vp, vp, vp, i64, vp]
    lib.jf_qkv_rope_bwd_workspace_bytes.argtypes = [i64, rope]
    lib.jf_strerror.argtypes = [i32]
    lib.jf_strerror.restype = ctypes.c_char_p
    lib.jf_device_status.argtypes = [vp]
    lib.jf_sm_count.argtypes = []
    for name in EXPORTED_SYMBOLS:
        if name != "jf_strerror":
            getattr(lib, name).restype = ctypes.c_int
    lib.jf_layernorm_i8_bwd_workspace_bytes.restype = i64
    lib.jf_granular_scale_count.restype = i64
    lib.jf_qkv_rope_bwd_workspace_bytes.restype = i64
    _lib = lib
    return lib


class QTensor(NamedTuple):
    q: torch.Tensor
    s: torch.Tensor

    @property
    def rows(self) -> int:
        return self.q.shape[0]

    @property
    def cols(self) -> int:
        return self.q.shape[1]


def empty_qtensor(rows: int, cols: int, device="cuda") -> QTensor:
    return QTensor(torch.empty((rows, cols), dtype=torch.int8, device=device),
                   torch.empty((rows // 32, cols // 32), dtype=torch.float32, device=device))


def _on(stream, device: torch.device):
    """The context of a stream in which a helper allocates: memory the caching allocator hands out belongs to one
    stream, and what the call frees again (a workspace) may still be in use there."""
    if not _has_cuda():
        return contextlib.nullcontext()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device)
    elif device.type == "cuda" and device.index is not None and stream.device_index != device.index:
        raise ValueError(f"a stream of cuda:{stream.device_index} for tensors on {device}")
    return torch.cuda.stream(stream)


def _empty_like(t: QTensor, rows: int, cols: int) -> QTensor:
    return QTensor(t.q.new_empty((rows, cols)), t.s.new_empty((rows // 32, cols // 32)))


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return t.data_ptr() if t.numel() else None


@functools.lru_cache(None)
def _has_cuda() -> bool:
    return torch.cuda.is_available()


def _stream(stream, device: int = -1) -> Optional[int]:
    """The handle of ``stream``, by default the current stream of the device (-1: the current one)."""
    if stream is None:
        if not _has_cuda():
            return None
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if device < 0 else device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _cq(t: QTensor) -> _CQ:
    return _CQ(_ptr(t.q), _ptr(t.s), t.q.shape[0], t.q.shape[1])


def _q(t: Optional[QTensor], rows: int, cols: int) -> _Q:
    if t is None:
        return _Q(None, None, rows, cols)
    return _Q(_ptr(t.q), _ptr(t.s), t.q.shape[0], t.q.shape[1])


def _check(status: int, where: str) -> None:
    if status != 0:
        raise JetfireError(status, where)


# --------------------------------------------------------------------------- C ABI, same names
def jf_quantize_block(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, stream=None) -> None:
    lib = load_library()
    if x.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {x.dtype}")
    _check(lib.jf_quantize_block(_ptr(x), _DTYPES[x.dtype], x.shape[0], x.shape[1], _ptr(q), _ptr(s),
                                 _stream(stream)), "jf_quantize_block")


def jf_quantize_block_rowstats(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, stats: torch.Tensor,
                               stream=None) -> None:
    lib = load_library()
    _check(lib.jf_quantize_block_rowstats(_ptr(x), _DTYPES[x.dtype], x.shape[0], x.shape[1], _ptr(q), _ptr(s),
                                          _ptr(stats), _stream(stream)), "jf_quantize_block_rowstats")


def jf_dequantize_block(q: torch.Tensor, s: torch.Tensor, y: torch.Tensor, stream=None) -> None:
    lib = load_library()
    if y.dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {y.dtype}")
    _check(lib.jf_dequantize_block(_ptr(q), _ptr(s), q.shape[0], q.shape[1], _ptr(y), _DTYPES[y.dtype],
                                   _stream(stream)), "jf_dequantize_block")


def jf_linear_fwd(X: QTensor, W: QTensor, Y: Optional[QTensor], y_f32: Optional[torch.Tensor] = None,
                  stream=None) -> None:
    lib = load_library()
    _check(lib.jf_linear_fwd(_cq(X), _cq(W), _q(Y, X.rows, W.rows), _ptr(y_f32), _stream(stream)), "jf_linear_fwd")


def jf_linear_fwd_gelu(X: QTensor, W: QTensor, Y: QTensor, Ypre: Optional[QTensor] = None, stream=None) -> None:
    lib = load_library()
    _check(lib.jf_linear_fwd_gelu(_cq(X), _cq(W), _q(Y, X.rows, W.rows), _q(Ypre, X.rows, W.rows), _stream(stream)),
           "jf_linear_fwd_gelu")


def jf_linear_dgrad(dY: QTensor, W: QTensor, dX: Optional[QTensor], dx_f32: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    lib = load_library()
    _check(lib.jf_linear_dgrad(_cq(dY), _cq(W), _q(dX, dY.rows, W.cols), _ptr(dx_f32), _stream(stream)),
           "jf_linear_dgrad")


def jf_linear_wgrad(dY: QTensor, X: QTensor, dW: Optional[QTensor], dw_f32: Optional[torch.Tensor] = None,
                    stream=None) -> None:
    lib = load_library()
    _check(lib.jf_linear_wgrad(_cq(dY), _cq(X), _q(dW, dY.cols, X.cols), _ptr(dw_f32), _stream(stream)),
           "jf_linear_wgrad")


def jf_gelu_i8(X: QTensor, Y: QTensor, stream=None) -> None:
    lib = load_library()
    _check(lib.jf_gelu_i8(_cq(X), _q(Y, X.rows, X.cols), _stream(stream)), "jf_gelu_i8")


def jf_layernorm_i8(X: QTensor, gamma: torch.Tensor, beta: torch.Tensor, eps: float, Y: QTensor,
                    stream=None) -> None:
    lib = load_library()
    _check(lib.jf_layernorm_i8(_cq(X), _ptr(gamma), _ptr(beta), ctypes.c_float(eps), _q(Y, X.rows, X.cols),
                               _stream(stream)), "jf_layernorm_i8")


def jf_layernorm_i8_rowstats(X: QTensor, stats: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor, eps: float,
                             Y: QTensor, stream=None) -> None:
    lib = load_library()
    _check(lib.jf_layernorm_i8_rowstats(_cq(X), _ptr(stats), _ptr(gamma), _ptr(beta), ctypes.c_float(eps),
                                        _q(Y, X.rows, X.cols), _stream(stream)), "jf_layernorm_i8_rowstats")


def jf_gelu_i8_bwd(X: QTensor, dY: QTensor, dX: QTensor, stream=None) -> None:
    lib = load_library()
    _check(lib.jf_gelu_i8_bwd(_cq(X), _cq(dY), _q(dX, X.rows, X.cols), _stream(stream)), "jf_gelu_i8_bwd")


def jf_layernorm_i8_bwd_workspace_bytes(rows: int, cols: int) -> int:
    return int(load_library().jf_layernorm_i8_bwd_workspace_bytes(rows, cols))


def jf_layernorm_i8_bwd(X: QTensor, dY: QTensor, gamma: torch.Tensor, eps: float, dX: QTensor,
                        dgamma: Optional[torch.Tensor] = None, dbeta: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    lib = load_library()
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib.jf_layernorm_i8_bwd(_cq(X), _cq(dY), _ptr(gamma), ctypes.c_float(eps), _q(dX, X.rows, X.cols),
                                   _ptr(dgamma), _ptr(dbeta), _ptr(workspace), nbytes, _stream(stream)),
           "jf_layernorm_i8_bwd")


def jf_layernorm_i8_bwd_noalloc(X: QTensor, dY: QTensor, gamma: torch.Tensor, eps: float, dX: QTensor,
                                dgamma: Optional[torch.Tensor] = None, dbeta: Optional[torch.Tensor] = None,
                                stream=None) -> None:
    lib = load_library()
    _check(lib.jf_layernorm_i8_bwd_noalloc(_cq(X), _cq(dY), _ptr(gamma), ctypes.c_float(eps), _q(dX, X.rows, X.cols),
                                           _ptr(dgamma), _ptr(dbeta), _stream(stream)), "jf_layernorm_i8_bwd_noalloc")


def jf_granular_scale_count(rows: int, cols: int, g: int) -> int:
    return int(load_library().jf_granular_scale_count(rows, cols, g))


def jf_quantize_granular(x: torch.Tensor, g: int, q: torch.Tensor, s: torch.Tensor, stream=None) -> None:
    lib = load_library()
    _check(lib.jf_quantize_granular(_ptr(x), _DTYPES[x.dtype], x.shape[0], x.shape[1], g, _ptr(q), _ptr(s),
                                    _stream(stream)), "jf_quantize_granular")


def jf_dequantize_granular(q: torch.Tensor, s: torch.Tensor, g: int, y: torch.Tensor, stream=None) -> None:
    lib = load_library()
    _check(lib.jf_dequantize_granular(_ptr(q), _ptr(s), q.shape[0], q.shape[1], g, _ptr(y), _DTYPES[y.dtype],
                                      _stream(stream)), "jf_dequantize_granular")


def jf_quantization_error(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, g: int, sums: torch.Tensor,
                          stream=None) -> None:
    lib = load_library()
    _check(lib.jf_quantization_error(_ptr(x), _DTYPES[x.dtype], _ptr(q), _ptr(s), x.shape[0], x.shape[1], g,
                                     _ptr(sums), _stream(stream)), "jf_quantization_error")


def quantize_granular(x: torch.Tensor, granularity: str, stream=None):
    """(codes, scales) of x at one granularity: "block", "token", "channel" or "tensor"."""
    g = GRANULARITY[granularity]
    q = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    s = torch.empty(jf_granular_scale_count(x.shape[0], x.shape[1], g), dtype=torch.float32, device=x.device)
    jf_quantize_granular(x, g, q, s, stream)
    return q, s


def quantization_mse(x: torch.Tensor, granularity: str, stream=None) -> float:
    """Mean squared error of quantize -> dequantize at one granularity, computed on the GPU."""
    q, s = quantize_granular(x, granularity, stream)
    sums = torch.empty(3, dtype=torch.float64, device=x.device)
    jf_quantization_error(x, q, s, GRANULARITY[granularity], sums, stream)
    if stream is not None:   # .item() below is ordered after the current stream only
        stream.synchronize() if hasattr(stream, "synchronize") else torch.cuda.synchronize()
    return float(sums[2].item())


def jf_mx_quantize(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, stream=None) -> None:
    lib = load_library()
    _check(lib.jf_mx_quantize(_ptr(x), _DTYPES[x.dtype], x.shape[0], x.shape[1], _ptr(codes), _ptr(scales),
                              _stream(stream)), "jf_mx_quantize")


def jf_mx_linear_fwd(a_codes, a_scales, b_codes, b_scales, y: torch.Tensor, stream=None) -> None:
    lib = load_library()
    M, K = a_codes.shape
    N = b_codes.shape[0]
    _check(lib.jf_mx_linear_fwd(_ptr(a_codes), _ptr(a_scales), _ptr(b_codes), _ptr(b_scales), M, N, K, _ptr(y),
                                _stream(stream)), "jf_mx_linear_fwd")


def mx_quantize(x: torch.Tensor, stream=None):
    """MXFP8 (E4M3 codes as uint8, E8M0 scale bytes per 1x32 block of a row) of x [rows, cols]."""
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scales = torch.empty((x.shape[0], x.shape[1] // 32), dtype=torch.uint8, device=x.device)
    jf_mx_quantize(x, codes, scales, stream)
    return codes, scales


def mx_linear_fwd(a_codes, a_scales, b_codes, b_scales, stream=None) -> torch.Tensor:
    """fp32 Y = A B^T of two MXFP8 tensors on the tensor core's block-scaled MMA."""
    y = torch.empty((a_codes.shape[0], b_codes.shape[0]), dtype=torch.float32, device=a_codes.device)
    jf_mx_linear_fwd(a_codes, a_scales, b_codes, b_scales, y, stream)
    return y


def jf_gemm_i8_s32(a: torch.Tensor, b: torch.Tensor, c: torch.Tensor, stream=None) -> None:
    """c (int32 [M, N]) = a (int8 [M, K]) @ b (int8 [N, K])^T on the tensor core, no scales."""
    lib = load_library()
    M, K = a.shape
    N = b.shape[0]
    _check(lib.jf_gemm_i8_s32(_ptr(a), _ptr(b), _ptr(c), M, N, K, _stream(stream)), "jf_gemm_i8_s32")


# ---- a transformer block around the linear layer: epilogues, bias gradient, QKV norm and rotation
def _device(where: str, first: torch.Tensor, *rest: Optional[torch.Tensor]) -> int:
    """The device index that all the tensors (Nones apart) share; -1 for host memory."""
    d = first.get_device()
    for t in rest:
        if t is not None and t.get_device() != d:
            raise ValueError(f"{where}: tensors on {first.device} and {t.device} in one call")
    return d


def _run(where: str, fn, args: tuple, device: int, stream) -> None:
    """fn(*args, stream) with the tensors' device current."""
    if not _has_cuda():   # the call refuses by itself
        status = fn(*args, None)
    elif device < 0:
        raise ValueError(f"{where}: the kernels take device memory, got CPU tensors")
    elif device == torch.cuda.current_device():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _stream(stream, device))
    if status != 0:
        raise JetfireError(status, where)


def _parts(t) -> tuple:
    return t if type(t) is QTensor else (t,) if t is not None else ()


_I8, _F32 = torch.int8, torch.float32


def _operand(t: QTensor, what: str, kind=_CQ):
    """The C struct of a QTensor whose types, shapes and layout have been checked."""
    q, s = t
    if q.dtype is not _I8 or s.dtype is not _F32:
        raise ValueError(f"{what}: codes must be int8 and scales float32")
    shape = q.shape
    if len(shape) != 2 or s.shape != (shape[0] // 32, shape[1] // 32):
        raise ValueError(f"{what}: scales of shape {tuple(s.shape)} do not belong to codes of shape {tuple(shape)}")
    if not (q.is_contiguous() and s.is_contiguous()):
        raise ValueError(f"{what}: codes and scales must be contiguous")
    return kind(q.data_ptr(), s.data_ptr(), shape[0], shape[1])


def _f32_vector(t: Optional[torch.Tensor], n: int, what: str) -> Optional[int]:
    if t is None:
        return None
    if t.dtype is not _F32 or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous, float32 and of shape ({n},), got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _matrix(t: Optional[torch.Tensor], rows: int, cols: int, what: str) -> _Matrix:
    """A dense matrix whose rows may be strided (the last dimension is contiguous)."""
    if t is None:
        return _NO_M
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"{what}: unsupported dtype {t.dtype}")
    if t.shape != (rows, cols):
        raise ValueError(f"{what} must have shape ({rows}, {cols}), got {tuple(t.shape)}")
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return _Matrix(t.data_ptr() if t.numel() else None, dt, ld if rows > 1 else max(cols, 1))


_NO_CQ, _NO_Q, _NO_M = _CQ(None, None, 0, 0), _Q(None, None, 0, 0), _Matrix(None, 0, 0)


def _residual(residual, rows: int, cols: int):
    if type(residual) is QTensor:
        return _operand(residual, "residual"), _NO_M
    return _NO_CQ, _matrix(residual, rows, cols, "residual")


def _activation(act: str) -> int:
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"unknown activation {act!r}: one of {', '.join(ACTIVATIONS)}")
    return code


def jf_linear_fwd_epilogue(X: QTensor, W: QTensor, Y: Optional[QTensor] = None, y: Optional[torch.Tensor] = None,
                           bias: Optional[torch.Tensor] = None, act: str = "none", residual=None,
                           P: Optional[QTensor] = None, stream=None) -> None:
    """Z = act(X W^T + bias) + residual into Y (INT8 blocks) and / or y (dense fp32, bf16 or fp16, rows may be
    strided); P receives the re-quantized pre-activation. The residual is a QTensor or a dense matrix; y
    may be the dense residual itself."""
    lib = load_library()
    cx, cw = _operand(X, "X"), _operand(W, "W")
    rows, cols = cx.rows, cw.rows
    Rq, R = _residual(residual, rows, cols)
    _run("jf_linear_fwd_epilogue", lib.jf_linear_fwd_epilogue,
         (cx, cw, _f32_vector(bias, cols, "bias"), _activation(act), Rq, R, _NO_Q if Y is None else _operand(Y, "Y", _Q),
          _matrix(y, rows, cols, "y"), _NO_Q if P is None else _operand(P, "P", _Q)),
         _device("jf_linear_fwd_epilogue", *X, *W, y, bias, *_parts(Y), *_parts(P), *_parts(residual)), stream)


def jf_linear_dgrad_epilogue(dY: QTensor, W: QTensor, dX: Optional[QTensor] = None, dx: Optional[torch.Tensor] = None,
                             pre: Optional[QTensor] = None, act: str = "none", residual=None, stream=None) -> None:
    """Z = (dY W) * act'(pre) + residual into dX (INT8 blocks) and / or dx (dense); pre is the INT8
    pre-activation the forward saved."""
    lib = load_library()
    cy, cw = _operand(dY, "dY"), _operand(W, "W")
    rows, cols = cy.rows, cw.cols
    Rq, R = _residual(residual, rows, cols)
    _run("jf_linear_dgrad_epilogue", lib.jf_linear_dgrad_epilogue,
         (cy, cw, _NO_CQ if pre is None else _operand(pre, "pre"), _activation(act), Rq, R,
          _NO_Q if dX is None else _operand(dX, "dX", _Q), _matrix(dx, rows, cols, "dx")),
         _device("jf_linear_dgrad_epilogue", *dY, *W, dx, *_parts(dX), *_parts(pre), *_parts(residual)), stream)


def jf_bias_grad(dY: QTensor, db: torch.Tensor, stream=None) -> None:
    """db (float32 [cols]) = the column sums of dY."""
    lib = load_library()
    cy = _operand(dY, "dY")
    _run("jf_bias_grad", lib.jf_bias_grad, (cy, _f32_vector(db, cy.cols, "db")), _device("jf_bias_grad", *dY, db), stream)


def jf_rope_table(inv_freq, cos: torch.Tensor, sin: torch.Tensor, magnitude: float = 1.0, stream=None) -> None:
    """Fills the float32 tables cos and sin [length, len(inv_freq)] of the angles position * inv_freq[j]."""
    lib = load_library()
    half = len(inv_freq)
    for t, what in ((cos, "cos"), (sin, "sin")):
        if t.dtype != torch.float32 or t.dim() != 2 or t.shape[1] != half or t.shape != cos.shape:
            raise ValueError(f"{what} must be float32 of shape (length, {half})")
    freq = (ctypes.c_double * max(half, 1))(*[float(f) for f in inv_freq])
    _run("jf_rope_table", lib.jf_rope_table, (freq, half, float(magnitude), cos.shape[0], _ptr(cos), _ptr(sin)),
         _device("jf_rope_table", cos, sin), stream)


class QKVRope(NamedTuple):
    """Heads, rotary tables and norm weights of a QKV tensor (struct jf_qkv_rope). The INT8 tensor's columns
    are q_heads, then kv_heads key and kv_heads value heads of head_dim columns; row b * seq + s is token s of
    sequence b, rows past batch * seq are padding. cos and sin are [table_len, rot_dim / 2] (see rope_table);
    positions, int64 with batch * seq elements, defaults to each token's place in its sequence."""
    batch: int
    seq: int
    q_heads: int
    kv_heads: int
    head_dim: int
    cos: Optional[torch.Tensor] = None
    sin: Optional[torch.Tensor] = None
    positions: Optional[torch.Tensor] = None
    gamma_q: Optional[torch.Tensor] = None
    gamma_k: Optional[torch.Tensor] = None
    eps: float = 1e-6
    layout: str = "half"


def _rope(a: QKVRope) -> _Rope:
    batch, seq, q_heads, kv_heads, d, cos, sin, positions, gamma_q, gamma_k, eps, layout = a
    code = ROPE_LAYOUTS.get(layout)
    if code is None:
        raise ValueError(f"unknown layout {layout!r}: one of {', '.join(ROPE_LAYOUTS)}")
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin belong together")
    half = length = 0
    pc = ps = None
    if cos is not None:
        if cos.dtype is not _F32 or sin.dtype is not _F32 or cos.dim() != 2 or cos.shape != sin.shape:
            raise ValueError("cos and sin must be float32 tables of one shape (length, rot_dim / 2)")
        length, half = cos.shape
        pc, ps = _ptr(cos), _ptr(sin)
    if positions is not None and (positions.dtype is not torch.int64 or positions.numel() != batch * seq):
        raise ValueError(f"positions must be int64 with {batch * seq} elements")
    return _Rope(batch, seq, q_heads, kv_heads, d, 2 * half, code, pc, ps, length,
                 None if positions is None else _ptr(positions), _f32_vector(gamma_q, d, "gamma_q"),
                 _f32_vector(gamma_k, d, "gamma_k"), eps)


_NO_HEADS = _Heads(None, 0, 0, 0)


def _heads(t: Optional[torch.Tensor], a: QKVRope, heads: int, heads_first: bool, dtype, what: str) -> _Heads:
    if t is None:
        if heads * a.batch * a.seq:
            raise ValueError(f"{what} is missing")
        return _NO_HEADS
    shape = (a.batch, heads, a.seq, a.head_dim) if heads_first else (a.batch, a.seq, heads, a.head_dim)
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{what} must be {dtype} of shape {shape}, got {t.dtype} {tuple(t.shape)}")
    b, x, y, step = t.stride()
    if step != 1 and t.numel():
        raise ValueError(f"{what}: the last dimension must be contiguous")
    return _Heads(t.data_ptr(), b, y, x) if heads_first else _Heads(t.data_ptr(), b, x, y)


def _qkv_dtype(*tensors) -> torch.dtype:
    dtype = next((t.dtype for t in tensors if t is not None), _F32)
    if dtype not in _DTYPES:
        raise ValueError(f"unsupported dtype {dtype}")
    return dtype


def jf_qkv_rope_fwd(qkv: QTensor, a: QKVRope, q: Optional[torch.Tensor], k: Optional[torch.Tensor],
                    v: Optional[torch.Tensor], heads_first: bool = False, stream=None) -> None:
    """q, k and v ([batch, seq, heads, head_dim], with heads_first [batch, heads, seq, head_dim]; strided views
    allowed) of the INT8 tensor qkv, queries and keys normed per head and rotated."""
    lib = load_library()
    dtype = _qkv_dtype(q, k, v)
    _run("jf_qkv_rope_fwd", lib.jf_qkv_rope_fwd,
         (_operand(qkv, "qkv"), _rope(a), _heads(q, a, a.q_heads, heads_first, dtype, "q"),
          _heads(k, a, a.kv_heads, heads_first, dtype, "k"), _heads(v, a, a.kv_heads, heads_first, dtype, "v"), _DTYPES[dtype]),
         _device("jf_qkv_rope_fwd", *qkv, q, k, v, a.cos, a.sin, a.positions, a.gamma_q, a.gamma_k), stream)


def jf_qkv_rope_bwd_workspace_bytes(rows: int, a: QKVRope) -> int:
    return int(load_library().jf_qkv_rope_bwd_workspace_bytes(rows, _rope(a)))


def jf_qkv_rope_bwd(qkv: QTensor, a: QKVRope, dq, dk, dv, dqkv: QTensor, dgamma_q: Optional[torch.Tensor] = None,
                    dgamma_k: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    heads_first: bool = False, stream=None) -> None:
    """The gradient of jf_qkv_rope_fwd: dq, dk, dv to INT8 dqkv and the norm weights' gradients."""
    _qkv_rope_bwd(load_library(), _rope(a), qkv, a, dq, dk, dv, dqkv, dgamma_q, dgamma_k, workspace, heads_first, stream)


def _qkv_rope_bwd(lib, rope: _Rope, qkv, a, dq, dk, dv, dqkv, dgamma_q, dgamma_k, workspace, heads_first, stream) -> None:
    dtype = _qkv_dtype(dq, dk, dv)
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _run("jf_qkv_rope_bwd", lib.jf_qkv_rope_bwd,
         (_operand(qkv, "qkv"), rope, _heads(dq, a, a.q_heads, heads_first, dtype, "dq"),
          _heads(dk, a, a.kv_heads, heads_first, dtype, "dk"), _heads(dv, a, a.kv_heads, heads_first, dtype, "dv"), _DTYPES[dtype],
          _operand(dqkv, "dqkv", _Q), _f32_vector(dgamma_q, a.head_dim, "dgamma_q"),
          _f32_vector(dgamma_k, a.head_dim, "dgamma_k"), None if workspace is None else _ptr(workspace), nbytes),
         _device("jf_qkv_rope_bwd", *qkv, dq, dk, dv, *dqkv, dgamma_q, dgamma_k, workspace, a.cos, a.sin, a.positions, a.gamma_q,
                 a.gamma_k), stream)


def jf_selftest_wait_timeout(limit_ns: int, stream=None) -> None:
    lib = load_library()
    _check(lib.jf_selftest_wait_timeout(limit_ns, _stream(stream)), "jf_selftest_wait_timeout")


def jf_strerror(status: int) -> str:
    return load_library().jf_strerror(int(status)).decode()


def jf_device_status(stream=None) -> int:
    return int(load_library().jf_device_status(_stream(stream)))


def jf_sm_count() -> int:
    return int(load_library().jf_sm_count())


# --------------------------------------------------------------------------- allocating helpers
def quantize_block(x: torch.Tensor, stream=None) -> QTensor:
    out = empty_qtensor(x.shape[0], x.shape[1], x.device)
    jf_quantize_block(x, out.q, out.s, stream)
    return out


def dequantize_block(t: QTensor, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    y = torch.empty(t.q.shape, dtype=dtype, device=t.q.device)
    jf_dequantize_block(t.q, t.s, y, stream)
    return y


def linear_fwd(X: QTensor, W: QTensor, want_f32: bool = False, stream=None):
    Y = empty_qtensor(X.rows, W.rows, X.q.device)
    yf = torch.empty((X.rows, W.rows), dtype=torch.float32, device=X.q.device) if want_f32 else None
    jf_linear_fwd(X, W, Y, yf, stream)
    return (Y, yf) if want_f32 else Y


def linear_fwd_gelu(X: QTensor, W: QTensor, want_pre: bool = False, stream=None):
    """Y = requant(GELU(X W^T)) with GELU applied on chip; with ``want_pre`` also the re-quantized
    pre-activation (the same tensor linear_fwd returns)."""
    Y = empty_qtensor(X.rows, W.rows, X.q.device)
    P = empty_qtensor(X.rows, W.rows, X.q.device) if want_pre else None
    jf_linear_fwd_gelu(X, W, Y, P, stream)
    return (Y, P) if want_pre else Y


def linear_dgrad(dY: QTensor, W: QTensor, want_f32: bool = False, stream=None):
    dX = empty_qtensor(dY.rows, W.cols, dY.q.device)
    xf = torch.empty((dY.rows, W.cols), dtype=torch.float32, device=dY.q.device) if want_f32 else None
    jf_linear_dgrad(dY, W, dX, xf, stream)
    return (dX, xf) if want_f32 else dX


def linear_wgrad(dY: QTensor, X: QTensor, want_f32: bool = False, stream=None):
    dW = empty_qtensor(dY.cols, X.cols, dY.q.device)
    wf = torch.empty((dY.cols, X.cols), dtype=torch.float32, device=dY.q.device) if want_f32 else None
    jf_linear_wgrad(dY, X, dW, wf, stream)
    return (dW, wf) if want_f32 else dW


def gelu_i8(X: QTensor, stream=None) -> QTensor:
    Y = empty_qtensor(X.rows, X.cols, X.q.device)
    jf_gelu_i8(X, Y, stream)
    return Y


def gelu_i8_bwd(X: QTensor, dY: QTensor, stream=None) -> QTensor:
    """dX = requant(dY * GELU'(X)) on INT8 blocks; X is the saved pre-activation."""
    dX = empty_qtensor(X.rows, X.cols, X.q.device)
    jf_gelu_i8_bwd(X, dY, dX, stream)
    return dX


def layernorm_i8_bwd(X: QTensor, dY: QTensor, gamma: torch.Tensor, eps: float = 1e-5, stream=None):
    """(dX, dgamma, dbeta) of LayerNorm_i8; the workspace is allocated here, per call."""
    dX = empty_qtensor(X.rows, X.cols, X.q.device)
    dgamma = torch.empty(X.cols, dtype=torch.float32, device=X.q.device)
    dbeta = torch.empty_like(dgamma)
    ws = torch.empty(jf_layernorm_i8_bwd_workspace_bytes(X.rows, X.cols), dtype=torch.uint8, device=X.q.device)
    jf_layernorm_i8_bwd(X, dY, gamma, eps, dX, dgamma, dbeta, ws, stream)
    return dX, dgamma, dbeta


def layernorm_i8(X: QTensor, gamma: torch.Tensor, beta: torch.Tensor, eps: float = 1e-5, stream=None) -> QTensor:
    Y = empty_qtensor(X.rows, X.cols, X.q.device)
    jf_layernorm_i8(X, gamma, beta, eps, Y, stream)
    return Y



def quantize_block_rowstats(x: torch.Tensor, stream=None):
    """(QTensor, stats): the per-block quantization of x and, per row and block, the int32 sums of q
    and q^2 ([rows, cols/32, 2]) that layernorm_i8_rowstats takes in place of a pass over the codes."""
    out = empty_qtensor(x.shape[0], x.shape[1], x.device)
    stats = torch.empty((x.shape[0], x.shape[1] // 32, 2), dtype=torch.int32, device=x.device)
    jf_quantize_block_rowstats(x, out.q, out.s, stats, stream)
    return out, stats


def layernorm_i8_rowstats(X: QTensor, stats: torch.Tensor, gamma: torch.Tensor, beta: torch.Tensor,
                          eps: float = 1e-5, stream=None) -> QTensor:
    Y = empty_qtensor(X.rows, X.cols, X.q.device)
    jf_layernorm_i8_rowstats(X, stats, gamma, beta, eps, Y, stream)
    return Y


def linear_fwd_epilogue(X: QTensor, W: QTensor, bias: Optional[torch.Tensor] = None, act: str = "none", residual=None,
                        want_pre: bool = False, out_dtype: Optional[torch.dtype] = None, stream=None):
    """act(X W^T + bias) + residual as INT8 blocks, or as a dense matrix of out_dtype; with ``want_pre`` also
    the re-quantized pre-activation X W^T + bias, for linear_dgrad_epilogue. The residual is a QTensor or a
    dense matrix of any supported dtype."""
    if stream is not None:
        with _on(stream, X.q.device):
            return linear_fwd_epilogue(X, W, bias, act, residual, want_pre, out_dtype)
    rows, cols = X.rows, W.rows
    Y = _empty_like(X, rows, cols) if out_dtype is None else None
    y = X.q.new_empty((rows, cols), dtype=out_dtype) if out_dtype is not None else None
    P = _empty_like(X, rows, cols) if want_pre else None
    jf_linear_fwd_epilogue(X, W, Y, y, bias, act, residual, P)
    out = Y if y is None else y
    return (out, P) if want_pre else out


def linear_dgrad_epilogue(dY: QTensor, W: QTensor, pre: Optional[QTensor] = None, act: str = "none", residual=None,
                          out_dtype: Optional[torch.dtype] = None, stream=None):
    """(dY W) * act'(pre) + residual as INT8 blocks, or as a dense matrix of out_dtype."""
    if stream is not None:
        with _on(stream, dY.q.device):
            return linear_dgrad_epilogue(dY, W, pre, act, residual, out_dtype)
    rows, cols = dY.rows, W.cols
    dX = _empty_like(dY, rows, cols) if out_dtype is None else None
    dx = dY.q.new_empty((rows, cols), dtype=out_dtype) if out_dtype is not None else None
    jf_linear_dgrad_epilogue(dY, W, dX, dx, pre, act, residual)
    return dX if dx is None else dx


def bias_grad(dY: QTensor, stream=None) -> torch.Tensor:
    """The bias gradient (float32 [cols]): the column sums of the INT8 gradient dY."""
    if stream is not None:
        with _on(stream, dY.q.device):
            return bias_grad(dY)
    db = dY.s.new_empty(dY.cols)
    jf_bias_grad(dY, db)
    return db


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     original_length: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(inv_freq, magnitude) of rotary positions over rot_dim dimensions, for rope_table.

    scaling "none": f_j = base^(-2 j / rot_dim). "linear": positions divided by ``factor``. "ntk": the base
    raised to base * factor^(rot_dim / (rot_dim - 2)), which leaves the fastest frequency and divides the
    slowest by ``factor``. "yarn": frequencies that turn more than beta_fast times over original_length stay,
    those that turn less than beta_slow times are divided by ``factor``, a linear ramp over j between; the
    tables are multiplied by 0.1 ln(factor) + 1."""
    if rot_dim <= 0 or rot_dim % 2:
        raise ValueError("rot_dim must be positive and even")
    if scaling not in ("none", "linear", "ntk", "yarn"):
        raise ValueError(f"unknown scaling {scaling!r}: one of none, linear, ntk, yarn")
    if factor <= 0.0 or (scaling == "ntk" and rot_dim == 2):
        raise ValueError("factor must be positive (and ntk needs rot_dim above 2)")
    half = rot_dim // 2
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freq = [base ** (-2.0 * j / rot_dim) for j in range(half)]
    if scaling == "linear":
        return [f / factor for f in freq], 1.0
    if scaling == "yarn":
        if original_length <= 0 or not beta_fast > beta_slow > 0:
            raise ValueError("yarn needs original_length > 0 and beta_fast > beta_slow > 0")

        def index_of(turns: float) -> float:   # the j whose frequency turns that often over original_length
            return half * math.log(original_length / (2.0 * math.pi * turns)) / math.log(base)

        low, high = max(math.floor(index_of(beta_fast)), 0), min(math.ceil(index_of(beta_slow)), rot_dim - 1)
        ramp = [min(max((j - low) / max(high - low, 1e-3), 0.0), 1.0) for j in range(half)]
        return [f * (1.0 - r) + f / factor * r for f, r in zip(freq, ramp)], 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    return freq, 1.0


def rope_table(length: int, inv_freq, magnitude: float = 1.0, device="cuda", stream=None):
    """(cos, sin): the float32 tables [length, len(inv_freq)] of a program's rotary positions, kept for all calls."""
    if stream is not None:
        with _on(stream, torch.device(device)):
            return rope_table(length, inv_freq, magnitude, device)
    cos = torch.empty((length, len(inv_freq)), dtype=torch.float32, device=device)
    sin = torch.empty_like(cos)
    jf_rope_table(inv_freq, cos, sin, magnitude)
    return cos, sin


def qkv_rope(qkv: QTensor, a: QKVRope, dtype: torch.dtype = torch.bfloat16, heads_first: bool = False, stream=None):
    """(q, k, v) for attention from the INT8 output of the QKV projection, [batch, seq, heads, head_dim] (with
    heads_first [batch, heads, seq, head_dim]): queries and keys normed per head (where ``a`` has weights) and
    rotated, values dequantized."""
    if stream is not None:
        with _on(stream, qkv.q.device):
            return qkv_rope(qkv, a, dtype, heads_first)
    out = [qkv.q.new_empty((a.batch, n, a.seq, a.head_dim) if heads_first else (a.batch, a.seq, n, a.head_dim), dtype=dtype)
           for n in (a.q_heads, a.kv_heads, a.kv_heads)]
    jf_qkv_rope_fwd(qkv, a, *out, heads_first)
    return tuple(out)


def qkv_rope_bwd(qkv: QTensor, a: QKVRope, dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor, heads_first: bool = False,
                 stream=None):
    """(dqkv, dgamma_q, dgamma_k) of qkv_rope: an INT8 gradient for the projection's backward, and the norm
    weights' gradients (None where there is no norm). The workspace is allocated here, per call."""
    if stream is not None:
        with _on(stream, qkv.q.device):
            return qkv_rope_bwd(qkv, a, dq, dk, dv, heads_first)
    lib, rope = load_library(), _rope(a)
    dqkv = _empty_like(qkv, qkv.rows, qkv.cols)
    dgq = qkv.s.new_empty(a.head_dim) if a.gamma_q is not None else None
    dgk = qkv.s.new_empty(a.head_dim) if a.gamma_k is not None else None
    ws = None
    if dgq is not None or dgk is not None:
        ws = qkv.q.new_empty(max(lib.jf_qkv_rope_bwd_workspace_bytes(qkv.rows, rope), 0), dtype=torch.uint8)
    _qkv_rope_bwd(lib, rope, qkv, a, dq, dk, dv, dqkv, dgq, dgk, ws, heads_first, None)
    return dqkv, dgq, dgk
