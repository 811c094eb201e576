"""ctypes binding of ``libfp8q.so`` -- argument marshalling only.

Two layers with the C names:

* ``lib()`` returns the loaded ``ctypes.CDLL`` whose functions take the exact
  C arguments (device pointers as ints, sizes, enums, a stream handle).
* ``fp8_quantize_per_tensor``, ``fp8_quantize_blockwise``, ``fp8_dequantize``,
  ``fp8_quantize_mx``, ``fp8_dequantize_mx``, ``fp8_amax_history_update`` and
  the other wrappers below, the ``fp8q_*`` operators of the feed-forward block
  among them, take torch CUDA tensors, allocate any
  output the caller did not pass (``torch.empty`` on the input's device), pass
  pointers and the current stream to the C function, and raise ``FP8Error`` on
  a nonzero status.  All computation happens in the library's kernels; there
  is no CPU fallback, and a missing library raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import NamedTuple

import torch

E4M3, E5M2 = 0, 1
F32, BF16 = 0, 1

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libfp8q.so")
_lib = None

class FP8BlockTensor(ctypes.Structure):
    """struct fp8_block_tensor of include/fp8q.h."""
    _fields_ = [("x", ctypes.c_void_p), ("q", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class FP8CurrentTensor(ctypes.Structure):
    """struct fp8_current_tensor of include/fp8q.h."""
    _fields_ = [("x", ctypes.c_void_p), ("q", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("scale_out", ctypes.c_void_p), ("amax_out", ctypes.c_void_p)]


class FP8DelayedTensor(ctypes.Structure):
    """struct fp8_delayed_tensor of include/fp8q.h."""
    _fields_ = [("x", ctypes.c_void_p), ("q", ctypes.c_void_p), ("n", ctypes.c_int64), ("scale", ctypes.c_void_p),
                ("history", ctypes.c_void_p), ("state", ctypes.c_void_p), ("scale_used", ctypes.c_void_p),
                ("amax_out", ctypes.c_void_p)]


# Declared in include/fp8q.h: name -> (restype, argtypes)
_c_int, _i64, _vp = ctypes.c_int, ctypes.c_int64, ctypes.c_void_p
SIGNATURES = {
    "fp8_quantize_per_tensor": (_c_int, [_vp, _c_int, _i64, _c_int, _vp, _vp, _vp, _vp, _vp]),
    "fp8_quantize_blockwise": (_c_int, [_vp, _c_int, _i64, _i64, _c_int, _c_int, _c_int, _vp, _vp, _vp]),
    "fp8_dequantize": (_c_int, [_vp, _c_int, _i64, _i64, _c_int, _c_int, _vp, _vp, _c_int, _vp]),
    "fp8_amax_history_update": (_c_int, [_vp, _vp, _c_int, _vp, _c_int, _vp, _vp]),
    "fp8_amax_history_update_ex": (_c_int, [_vp, _vp, _c_int, _vp, _c_int, _vp, _c_int, ctypes.c_float,
                                            ctypes.c_float, _vp]),
    "fp8_quantize_per_tensor_fused": (_c_int, [_vp, _c_int, _i64, _c_int, _vp, _vp, _vp, _vp, _vp]),
    "fp8_quantize_per_tensor_fused_noalloc": (_c_int, [_vp, _c_int, _i64, _c_int, _vp, _vp, _vp, _vp]),
    "fp8_amax": (_c_int, [_vp, _c_int, _i64, _vp, _vp]),
    "fp8_scale_from_amax": (_c_int, [_vp, _c_int, _vp, _vp]),
    "fp8_fake_quantize": (_c_int, [_vp, _c_int, _i64, _i64, _c_int, _c_int, _c_int, _vp, _vp, _vp, _vp]),
    "fp8_quantize_per_tensor_transpose": (_c_int, [_vp, _c_int, _i64, _i64, _c_int, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fp8_gemm_blockwise_ex": (_c_int, [_vp, _vp, _c_int, _vp, _vp, _c_int, _c_int, _i64, _i64, _i64, _vp, _c_int,
                                       _vp]),
    "fp8_quantize_blockwise_transpose": (_c_int, [_vp, _c_int, _i64, _i64, _c_int, _c_int, _c_int, _vp, _vp, _vp,
                                                  _vp, _vp]),
    "fp8_quantize_mx": (_c_int, [_vp, _c_int, _i64, _i64, _c_int, _c_int, _vp, _vp, _vp]),
    "fp8_dequantize_mx": (_c_int, [_vp, _c_int, _i64, _i64, _vp, _vp, _c_int, _vp]),
    "fp8_gemm_blockwise": (_c_int, [_vp, _vp, _c_int, _vp, _vp, _c_int, _i64, _i64, _i64, _vp, _c_int, _vp]),
    "fp8_quantize_delayed_step": (_c_int, [_vp, _c_int, _i64, _c_int, _vp, _vp, _vp, _c_int, _c_int, ctypes.c_float,
                                           ctypes.c_float, _vp, _vp, _vp, _vp, _vp]),
    "fp8_quantize_blockwise_grouped": (_c_int, [ctypes.POINTER(FP8BlockTensor), _c_int, _c_int, _c_int, _c_int,
                                                _c_int, _vp]),
    "fp8_quantize_delayed_step_grouped": (_c_int, [ctypes.POINTER(FP8DelayedTensor), _c_int, _c_int, _c_int, _c_int,
                                                   _c_int, ctypes.c_float, ctypes.c_float, _vp, _vp]),
    "fp8_quantize_per_tensor_grouped": (_c_int, [ctypes.POINTER(FP8CurrentTensor), _c_int, _c_int, _c_int, _vp]),
    "fp8_status_string": (ctypes.c_char_p, [_c_int]),
    "fp8_device_status": (_c_int, [_vp, _c_int, _vp]),
    "fp8_selftest_wait_timeout": (_c_int, [ctypes.c_uint32, _vp]),
}
# Declared in include/fp8q_ffn.h (the feed-forward operators)
FFN_SIGNATURES = {
    "fp8q_rmsnorm_quantize": (_c_int, [_vp, _c_int, _vp, _vp, _c_int, _i64, _i64, ctypes.c_float, _c_int, _vp, _vp, _vp,
                                       _vp, _vp, _vp]),
    "fp8q_rmsnorm_backward": (_c_int, [_vp, _vp, _c_int, _vp, _vp, _c_int, _vp, _i64, _i64, _vp, _vp, _vp, _i64, _vp]),
    "fp8q_rmsnorm_backward_workspace": (_i64, [_i64, _i64]),
    "fp8q_gemm_gated": (_c_int, [_vp, _vp, _c_int, _vp, _vp, _c_int, _i64, _i64, _i64, _c_int, _c_int, _vp, _vp, _vp,
                                 _c_int, _vp]),
    "fp8q_gated_backward": (_c_int, [_vp, _vp, _c_int, _i64, _i64, _c_int, _c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "fp8q_moe_sort": (_c_int, [_vp, _i64, _i64, _c_int, _c_int, _i64, _vp, _vp, _vp, _vp, _vp, _i64, _vp]),
    "fp8q_moe_rows": (_i64, [_i64, _i64, _c_int, _c_int]),
    "fp8q_moe_sort_workspace": (_i64, [_i64, _i64, _c_int]),
    "fp8q_moe_dispatch": (_c_int, [_vp, _c_int, _i64, _vp, _c_int, _vp, _vp, _i64, _i64, _i64, _c_int, _vp, _vp, _vp, _vp,
                                   _vp]),
    "fp8q_moe_dispatch_codes": (_c_int, [_vp, _vp, _c_int, _i64, _vp, _c_int, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp]),
    "fp8q_moe_combine": (_c_int, [_vp, _c_int, _i64, _i64, _vp, _vp, _vp, _i64, _i64, _vp, _vp]),
    "fp8q_moe_combine_backward": (_c_int, [_vp, _vp, _c_int, _i64, _vp, _c_int, _vp, _vp, _i64, _i64, _i64, _vp, _c_int, _vp,
                                           _vp, _vp, _vp, _vp, _vp]),
    "fp8q_gemm_grouped": (_c_int, [_vp, _vp, _c_int, _vp, _vp, _c_int, _vp, _c_int, _i64, _i64, _i64, _vp, _c_int, _vp]),
    "fp8q_gemm_gated_grouped": (_c_int, [_vp, _vp, _c_int, _vp, _vp, _c_int, _vp, _c_int, _i64, _i64, _i64, _c_int, _c_int,
                                         _vp, _vp, _vp, _c_int, _vp]),
    "fp8q_gemm_grouped_wgrad": (_c_int, [_vp, _vp, _c_int, _vp, _vp, _c_int, _vp, _c_int, _i64, _i64, _i64, _vp, _c_int,
                                         _vp]),
}
DEVICE_STATUS_WAIT_TIMEOUT = 0x1
ACT_SILU, ACT_GELU_TANH = 0, 1
AMAX_WINDOW_MAX, AMAX_EMA = 0, 1
MX_FIT, MX_OCP = 0, 1
FUSED_WORKSPACE_BYTES = 16


class FP8Error(RuntimeError):
    """A libfp8q call returned an error status."""

    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: status {status} ({fp8_status_string(status)})")


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libfp8q.so (raises if it has not been built)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(
            f"{p} is missing: build it with `python -m fine_grained_block_b200.build` "
            "(there is no fallback implementation)")
    L = ctypes.CDLL(p)
    for name, (res, args) in (*SIGNATURES.items(), *FFN_SIGNATURES.items()):
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = L
    return L


lib = load_library


def fp8_status_string(status: int) -> str:
    return load_library().fp8_status_string(int(status)).decode()


# -- marshalling helpers ----------------------------------------------------------

_DTYPE_CODE = {torch.float32: F32, torch.bfloat16: BF16}


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libfp8q works on CUDA tensors only")
        if t is not None and not t.is_contiguous():
            raise ValueError("libfp8q needs contiguous tensors")


def _check(fn: str, status: int):
    if status != 0:
        raise FP8Error(fn, status)


# -- entry points -------------------------------------------------------------------

def fp8_quantize_per_tensor(x: torch.Tensor, fmt: int = E4M3, scale_in: torch.Tensor | None = None,
                            q: torch.Tensor | None = None, scale_out: torch.Tensor | None = None,
                            amax_out: torch.Tensor | None = None, want_amax: bool = True, stream=None):
    """Per-tensor quantize.  scale_in None = current scaling, else delayed (a 1-element fp32 CUDA tensor).

    Returns (q uint8 like x, scale_out [1] fp32, amax_out [1] fp32 or None)."""
    _need_cuda(x, scale_in, q, scale_out, amax_out)
    dev = x.device
    q = torch.empty(x.shape, dtype=torch.uint8, device=dev) if q is None else q
    scale_out = torch.empty(1, dtype=torch.float32, device=dev) if scale_out is None else scale_out
    if amax_out is None and (want_amax or scale_in is None):
        amax_out = torch.empty(1, dtype=torch.float32, device=dev)
    st = load_library().fp8_quantize_per_tensor(_ptr(x), _DTYPE_CODE[x.dtype], x.numel(), fmt, _ptr(scale_in),
                                                _ptr(q), _ptr(scale_out), _ptr(amax_out), _stream(stream))
    _check("fp8_quantize_per_tensor", st)
    return q, scale_out, amax_out


def fp8_quantize_per_tensor_transpose(x: torch.Tensor, fmt: int = E4M3, scale_in: torch.Tensor | None = None,
                                      with_q: bool = True, q: torch.Tensor | None = None,
                                      qt: torch.Tensor | None = None, scale_out: torch.Tensor | None = None,
                                      amax_out: torch.Tensor | None = None, stream=None):
    """Per-tensor quantize of a 2-D tensor with a transposed copy.  Returns (q or None, qt [C, R], scale, amax)."""
    _need_cuda(x, scale_in, q, qt, scale_out, amax_out)
    if x.dim() != 2:
        raise ValueError("the transposing quantize takes a 2-D tensor")
    R, C = x.shape
    dev = x.device
    if q is None and with_q:
        q = torch.empty((R, C), dtype=torch.uint8, device=dev)
    qt = torch.empty((C, R), dtype=torch.uint8, device=dev) if qt is None else qt
    scale_out = torch.empty(1, dtype=torch.float32, device=dev) if scale_out is None else scale_out
    amax_out = torch.empty(1, dtype=torch.float32, device=dev) if amax_out is None else amax_out
    st = load_library().fp8_quantize_per_tensor_transpose(_ptr(x), _DTYPE_CODE[x.dtype], R, C, fmt, _ptr(scale_in),
                                                          _ptr(q), _ptr(qt), _ptr(scale_out), _ptr(amax_out),
                                                          _stream(stream))
    _check("fp8_quantize_per_tensor_transpose", st)
    return q, qt, scale_out, amax_out


def fused_workspace(device="cuda") -> torch.Tensor:
    """A zeroed workspace for fp8_quantize_per_tensor_fused (one per stream)."""
    return torch.zeros(FUSED_WORKSPACE_BYTES // 4, dtype=torch.int32, device=device)


def fp8_quantize_per_tensor_fused(x: torch.Tensor, fmt: int = E4M3, workspace: torch.Tensor | None = None,
                                  q: torch.Tensor | None = None, scale_out: torch.Tensor | None = None,
                                  amax_out: torch.Tensor | None = None, stream=None):
    """Per-tensor current scaling in one pass when x fits on chip (else the two-pass path).

    Returns (q, scale_out [1], amax_out [1])."""
    _need_cuda(x, workspace, q, scale_out, amax_out)
    dev = x.device
    workspace = fused_workspace(dev) if workspace is None else workspace
    q = torch.empty(x.shape, dtype=torch.uint8, device=dev) if q is None else q
    scale_out = torch.empty(1, dtype=torch.float32, device=dev) if scale_out is None else scale_out
    amax_out = torch.empty(1, dtype=torch.float32, device=dev) if amax_out is None else amax_out
    st = load_library().fp8_quantize_per_tensor_fused(_ptr(x), _DTYPE_CODE[x.dtype], x.numel(), fmt, _ptr(q),
                                                      _ptr(scale_out), _ptr(amax_out), _ptr(workspace),
                                                      _stream(stream))
    _check("fp8_quantize_per_tensor_fused", st)
    return q, scale_out, amax_out


def fp8_amax(x: torch.Tensor, amax_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """max |x| into a 1-element fp32 CUDA tensor."""
    _need_cuda(x, amax_out)
    amax_out = torch.empty(1, dtype=torch.float32, device=x.device) if amax_out is None else amax_out
    _check("fp8_amax", load_library().fp8_amax(_ptr(x), _DTYPE_CODE[x.dtype], x.numel(), _ptr(amax_out),
                                               _stream(stream)))
    return amax_out


def fp8_scale_from_amax(amax: torch.Tensor, fmt: int = E4M3, scale_out: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """MAX / max(amax, 1e-12) into a 1-element fp32 CUDA tensor."""
    _need_cuda(amax, scale_out)
    scale_out = torch.empty(1, dtype=torch.float32, device=amax.device) if scale_out is None else scale_out
    _check("fp8_scale_from_amax", load_library().fp8_scale_from_amax(_ptr(amax), fmt, _ptr(scale_out),
                                                                     _stream(stream)))
    return scale_out


def fp8_quantize_blockwise(x: torch.Tensor, block=(1, 128), fmt: int = E4M3, q: torch.Tensor | None = None,
                           scales: torch.Tensor | None = None, stream=None):
    """Blockwise quantize of a 2-D tensor with (1, 128) or (128, 128) blocks.  Returns (q, scales)."""
    _need_cuda(x, q, scales)
    if x.dim() != 2:
        raise ValueError("blockwise quantize takes a 2-D tensor")
    R, C = x.shape
    br, bc = block
    q = torch.empty((R, C), dtype=torch.uint8, device=x.device) if q is None else q
    if scales is None:
        scales = torch.empty((math.ceil(R / br), math.ceil(C / bc)), dtype=torch.float32, device=x.device)
    st = load_library().fp8_quantize_blockwise(_ptr(x), _DTYPE_CODE[x.dtype], R, C, br, bc, fmt, _ptr(q),
                                               _ptr(scales), _stream(stream))
    _check("fp8_quantize_blockwise", st)
    return q, scales


def fp8_quantize_blockwise_grouped(xs, block=(1, 128), fmt: int = E4M3, qs=None, scales=None, stream=None):
    """Blockwise quantize of several 2-D tensors (same dtype, cols % 128 == 0) in as few launches as possible.

    Returns (list of q, list of scales)."""
    xs = list(xs)
    if not xs:
        return [], []
    dt = xs[0].dtype
    br, bc = block
    qs = [torch.empty(x.shape, dtype=torch.uint8, device=x.device) for x in xs] if qs is None else list(qs)
    if scales is None:
        scales = [torch.empty((math.ceil(x.shape[0] / br), math.ceil(x.shape[1] / bc)), dtype=torch.float32,
                              device=x.device) for x in xs]
    arr = (FP8BlockTensor * len(xs))()
    for i, (x, q, s_) in enumerate(zip(xs, qs, scales)):
        _need_cuda(x, q, s_)
        if x.dim() != 2 or x.dtype != dt:
            raise ValueError("grouped quantize takes 2-D tensors of one dtype")
        arr[i] = FP8BlockTensor(_ptr(x), _ptr(q), _ptr(s_), x.shape[0], x.shape[1])
    st = load_library().fp8_quantize_blockwise_grouped(arr, len(xs), _DTYPE_CODE[dt], br, bc, fmt, _stream(stream))
    _check("fp8_quantize_blockwise_grouped", st)
    return qs, scales


def fp8_quantize_blockwise_transpose(x: torch.Tensor, block=(1, 128), fmt: int = E4M3, q=None, scales=None,
                                     qt=None, scales_t=None, stream=None):
    """Blockwise quantize of x and of x^T in one pass (rows, cols multiples of 128).

    Returns (q, scales, qt, scales_t) = fp8_quantize_blockwise(x, block) + fp8_quantize_blockwise(x.T, block)."""
    _need_cuda(x, q, scales, qt, scales_t)
    if x.dim() != 2:
        raise ValueError("the transposing blockwise quantize takes a 2-D tensor")
    R, C = x.shape
    br, bc = block
    dev = x.device
    q = torch.empty((R, C), dtype=torch.uint8, device=dev) if q is None else q
    qt = torch.empty((C, R), dtype=torch.uint8, device=dev) if qt is None else qt
    if scales is None:
        scales = torch.empty((R // br, C // bc), dtype=torch.float32, device=dev)
    if scales_t is None:
        scales_t = torch.empty((C // br, R // bc), dtype=torch.float32, device=dev)
    st = load_library().fp8_quantize_blockwise_transpose(_ptr(x), _DTYPE_CODE[x.dtype], R, C, br, bc, fmt, _ptr(q),
                                                         _ptr(scales), _ptr(qt), _ptr(scales_t), _stream(stream))
    _check("fp8_quantize_blockwise_transpose", st)
    return q, scales, qt, scales_t


def fp8_quantize_mx(x: torch.Tensor, fmt: int = E4M3, rule: int = MX_FIT, q: torch.Tensor | None = None,
                    e8m0: torch.Tensor | None = None, stream=None):
    """MX quantize of a 2-D tensor: 1x32 blocks, power-of-two scales.  Returns (q, e8m0 uint8 [R, ceil(C/32)])."""
    _need_cuda(x, q, e8m0)
    if x.dim() != 2:
        raise ValueError("MX quantize takes a 2-D tensor")
    R, C = x.shape
    q = torch.empty((R, C), dtype=torch.uint8, device=x.device) if q is None else q
    if e8m0 is None:
        e8m0 = torch.empty((R, math.ceil(C / 32)), dtype=torch.uint8, device=x.device)
    st = load_library().fp8_quantize_mx(_ptr(x), _DTYPE_CODE[x.dtype], R, C, fmt, rule, _ptr(q), _ptr(e8m0),
                                        _stream(stream))
    _check("fp8_quantize_mx", st)
    return q, e8m0


def fp8_dequantize_mx(q: torch.Tensor, e8m0: torch.Tensor, fmt: int = E4M3, out_dtype=torch.float32,
                      y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """MX dequantize: y = decode(q) * 2^(e8m0 - 127) per 1x32 block."""
    _need_cuda(q, e8m0, y)
    if q.dim() != 2:
        raise ValueError("MX dequantize takes a 2-D tensor")
    R, C = q.shape
    y = torch.empty((R, C), dtype=out_dtype, device=q.device) if y is None else y
    st = load_library().fp8_dequantize_mx(_ptr(q), fmt, R, C, _ptr(e8m0), _ptr(y), _DTYPE_CODE[y.dtype],
                                          _stream(stream))
    _check("fp8_dequantize_mx", st)
    return y


def fp8_gemm_blockwise(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor, a_fmt: int = E4M3,
                       b_fmt: int = E4M3, out_dtype=torch.bfloat16, c: torch.Tensor | None = None,
                       stream=None, b_block: int = 128) -> torch.Tensor:
    """C [M, N] = A [M, K] (1x128 scales sa) x B [N, K]^T, FP8 tensor cores.

    b_block 128: B with 128x128 scales sb [N/128, K/128] (fp8_gemm_blockwise); b_block 1: B with 1x128
    scales sb [N, K/128], the weight-gradient form (fp8_gemm_blockwise_ex)."""
    _need_cuda(a, sa, b, sb, c)
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[1]:
        raise ValueError("fp8_gemm_blockwise takes a [M, K] and b [N, K]")
    M, K = a.shape
    N = b.shape[0]
    c = torch.empty((M, N), dtype=out_dtype, device=a.device) if c is None else c
    if b_block == 128:
        st = load_library().fp8_gemm_blockwise(_ptr(a), _ptr(sa), a_fmt, _ptr(b), _ptr(sb), b_fmt, M, N, K, _ptr(c),
                                               _DTYPE_CODE[c.dtype], _stream(stream))
        _check("fp8_gemm_blockwise", st)
    else:
        st = load_library().fp8_gemm_blockwise_ex(_ptr(a), _ptr(sa), a_fmt, _ptr(b), _ptr(sb), b_block, b_fmt, M, N,
                                                  K, _ptr(c), _DTYPE_CODE[c.dtype], _stream(stream))
        _check("fp8_gemm_blockwise_ex", st)
    return c


def fp8_dequantize(q: torch.Tensor, scales: torch.Tensor, block=(0, 0), fmt: int = E4M3,
                   out_dtype=torch.bfloat16, y: torch.Tensor | None = None, stream=None):
    """Dequantize codes; block (0, 0) = per-tensor (scales[0]).  Returns y."""
    _need_cuda(q, scales, y)
    if q.dim() == 1:
        R, C = 1, q.shape[0]
    elif q.dim() == 2:
        R, C = q.shape
    else:
        raise ValueError("dequantize takes a 1-D or 2-D tensor")
    y = torch.empty(q.shape, dtype=out_dtype, device=q.device) if y is None else y
    st = load_library().fp8_dequantize(_ptr(q), fmt, R, C, block[0], block[1], _ptr(scales), _ptr(y),
                                       _DTYPE_CODE[y.dtype], _stream(stream))
    _check("fp8_dequantize", st)
    return y


def fp8_fake_quantize(x: torch.Tensor, block=(1, 128), fmt: int = E4M3, scale_in: torch.Tensor | None = None,
                      y: torch.Tensor | None = None, scales_out: torch.Tensor | None = None, stream=None):
    """Quantize -> dequantize round trip in x's dtype (block (0, 0) = per tensor with scale_in).  Returns y."""
    _need_cuda(x, scale_in, y, scales_out)
    if x.dim() == 1:
        R, C = 1, x.shape[0]
    elif x.dim() == 2:
        R, C = x.shape
    else:
        raise ValueError("fake quantize takes a 1-D or 2-D tensor")
    y = torch.empty_like(x) if y is None else y
    st = load_library().fp8_fake_quantize(_ptr(x), _DTYPE_CODE[x.dtype], R, C, block[0], block[1], fmt,
                                          _ptr(scale_in), _ptr(y), _ptr(scales_out), _stream(stream))
    _check("fp8_fake_quantize", st)
    return y


def fp8_amax_history_update(history: torch.Tensor, state: torch.Tensor, amax: torch.Tensor, scale: torch.Tensor,
                            fmt: int = E4M3, stream=None):
    """Push amax into the history ring and refresh scale in place (all 4 are CUDA tensors)."""
    _need_cuda(history, state, amax, scale)
    st = load_library().fp8_amax_history_update(_ptr(history), _ptr(state), history.numel(), _ptr(amax), fmt,
                                                _ptr(scale), _stream(stream))
    _check("fp8_amax_history_update", st)
    return scale


def fp8_device_status(clear: bool = False, device=None, stream=None) -> int:
    """The device status word (FP8_DEVICE_STATUS_* bits); synchronizes the stream to read it."""
    out = torch.zeros(1, dtype=torch.int32, device=device or "cuda")
    _check("fp8_device_status", load_library().fp8_device_status(_ptr(out), 1 if clear else 0, _stream(stream)))
    return int(out.item())


def fp8_selftest_wait_timeout(timeout_us: int = 1000, stream=None):
    """Launch a wait that can only time out (sets DEVICE_STATUS_WAIT_TIMEOUT after timeout_us)."""
    _check("fp8_selftest_wait_timeout", load_library().fp8_selftest_wait_timeout(int(timeout_us), _stream(stream)))


def fp8_amax_history_update_ex(history: torch.Tensor, state: torch.Tensor, amax: torch.Tensor, scale: torch.Tensor,
                               fmt: int = E4M3, algo: int = AMAX_WINDOW_MAX, alpha: float = 1.0,
                               margin: float = 1.0, stream=None):
    """Delayed-scaling update with a margin and window-max or EMA smoothing (PyTorch-FP8 page s4.3)."""
    _need_cuda(history, state, amax, scale)
    st = load_library().fp8_amax_history_update_ex(_ptr(history), _ptr(state), history.numel(), _ptr(amax), fmt,
                                                   _ptr(scale), algo, float(alpha), float(margin), _stream(stream))
    _check("fp8_amax_history_update_ex", st)
    return scale


def fp8_quantize_delayed_step(x: torch.Tensor, scale: torch.Tensor, history: torch.Tensor, state: torch.Tensor,
                              fmt: int = E5M2, algo: int = AMAX_WINDOW_MAX, alpha: float = 1.0, margin: float = 1.0,
                              q: torch.Tensor | None = None, scale_used: torch.Tensor | None = None,
                              amax_out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                              stream=None) -> torch.Tensor:
    """Cast x with *scale, then (same launch) push amax(x) into the history and rewrite *scale."""
    _need_cuda(x, scale, history, state, q, scale_used, amax_out, workspace)
    dev = x.device
    q = torch.empty(x.shape, dtype=torch.uint8, device=dev) if q is None else q
    scale_used = torch.empty(1, dtype=torch.float32, device=dev) if scale_used is None else scale_used
    amax_out = torch.empty(1, dtype=torch.float32, device=dev) if amax_out is None else amax_out
    workspace = fused_workspace(dev) if workspace is None else workspace
    st = load_library().fp8_quantize_delayed_step(_ptr(x), _DTYPE_CODE[x.dtype], x.numel(), fmt, _ptr(scale),
                                                  _ptr(history), _ptr(state), history.numel(), algo, alpha, margin,
                                                  _ptr(q), _ptr(scale_used), _ptr(amax_out), _ptr(workspace),
                                                  _stream(stream))
    _check("fp8_quantize_delayed_step", st)
    return q


def fp8_quantize_delayed_step_grouped(xs, scalers, qs=None, workspace: torch.Tensor | None = None, stream=None):
    """One delayed-scaling step for several tensors in as few launches as possible.

    scalers: one DelayedScaler per tensor (same fmt, window, algo, alpha and margin); each is stepped as
    scaler.step(x) would step it.  Returns the list of codes."""
    xs, scalers = list(xs), list(scalers)
    if len(xs) != len(scalers):
        raise ValueError("one scaler per tensor")
    if not xs:
        return []
    s0 = scalers[0]
    if any((s.fmt, s.history.numel(), s.algo, s.alpha, s.margin) !=
           (s0.fmt, s0.history.numel(), s0.algo, s0.alpha, s0.margin) for s in scalers):
        raise ValueError("grouped scalers must share fmt, window, algo, alpha and margin")
    dt = xs[0].dtype
    qs = [torch.empty(x.shape, dtype=torch.uint8, device=x.device) for x in xs] if qs is None else list(qs)
    if workspace is None:
        workspace = torch.zeros(len(xs) * FUSED_WORKSPACE_BYTES // 4, dtype=torch.int32, device=xs[0].device)
    arr = (FP8DelayedTensor * len(xs))()
    for i, (x, q, sc) in enumerate(zip(xs, qs, scalers)):
        _need_cuda(x, q)
        if x.dtype != dt:
            raise ValueError("grouped tensors must share one dtype")
        arr[i] = FP8DelayedTensor(_ptr(x), _ptr(q), x.numel(), _ptr(sc.scale), _ptr(sc.history), _ptr(sc.state),
                                  _ptr(sc.scale_used), _ptr(sc.amax))
    st = load_library().fp8_quantize_delayed_step_grouped(arr, len(xs), _DTYPE_CODE[dt], s0.fmt, s0.history.numel(),
                                                          s0.algo, s0.alpha, s0.margin, _ptr(workspace),
                                                          _stream(stream))
    _check("fp8_quantize_delayed_step_grouped", st)
    return qs


def fp8_quantize_per_tensor_grouped(xs, fmt: int = E4M3, qs=None, scales=None, amaxes=None, stream=None):
    """Per-tensor current scaling of several tensors in three launches per 128 tensors: each tensor gets
    its own amax and scale, exactly as from fp8_quantize_per_tensor(x, fmt).  Returns (codes, scales, amaxes),
    lists of CUDA tensors (codes in each x's shape, scales and amaxes of one element)."""
    xs = list(xs)
    if not xs:
        return [], [], []
    dt = xs[0].dtype
    dev = xs[0].device
    qs = [torch.empty(x.shape, dtype=torch.uint8, device=x.device) for x in xs] if qs is None else list(qs)
    scales = [torch.empty(1, dtype=torch.float32, device=dev) for _ in xs] if scales is None else list(scales)
    amaxes = [torch.empty(1, dtype=torch.float32, device=dev) for _ in xs] if amaxes is None else list(amaxes)
    arr = (FP8CurrentTensor * len(xs))()
    for i, (x, q, s_, a_) in enumerate(zip(xs, qs, scales, amaxes)):
        _need_cuda(x, q, s_, a_)
        if x.dtype != dt:
            raise ValueError("grouped tensors must share one dtype")
        arr[i] = FP8CurrentTensor(_ptr(x), _ptr(q), x.numel(), _ptr(s_), _ptr(a_))
    st = load_library().fp8_quantize_per_tensor_grouped(arr, len(xs), _DTYPE_CODE[dt], fmt, _stream(stream))
    _check("fp8_quantize_per_tensor_grouped", st)
    return qs, scales, amaxes


# -- feed-forward operators ---------------------------------------------------------

# The small calls of a decode step are bound by this code: a launch costs 2.3 us, so the checks are written to
# cost about as much (torch._C._cuda_getCurrentRawStream, for one, instead of building a Stream object in 3.3 us).

_U8, _F32T, _BF16T = torch.uint8, torch.float32, torch.bfloat16
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else \
    lambda device: torch.cuda.current_stream(device).cuda_stream


def _ffn_context(x: torch.Tensor, stream):
    """Context in which a call on x runs and allocates: its device, and `stream` when one was given, so that
    memory allocated for the call belongs to the stream that uses it."""
    if stream is None:
        return torch.cuda.device(x.device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=x.device) if stream else \
            torch.cuda.default_stream(x.device)
    if stream.device != x.device:
        raise ValueError("the stream is on another device than the tensors")
    return torch.cuda.stream(stream)


def _here(x: torch.Tensor) -> int:
    """x's device if it is the current one, else -1."""
    device = x.get_device()
    if device < 0:
        raise ValueError("libfp8q works on CUDA tensors only")
    return device if device == _current_device() else -1


def _fits(t: torch.Tensor, name: str, device: int, shape, dtype) -> int:
    """The address of t, which has to be a contiguous tensor of this device, shape and dtype."""
    if t.shape == shape and t.dtype is dtype and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, not {dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name} is not on the device of the first tensor")
    raise ValueError(f"{name} is not contiguous")


def _float_code(t: torch.Tensor, name: str) -> int:
    dtype = t.dtype
    if dtype is _BF16T:
        return BF16
    if dtype is _F32T:
        return F32
    raise ValueError(f"{name} has dtype {dtype}, not float32 or bfloat16")


def fp8q_rmsnorm_quantize(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None, eps: float = 1e-6,
                          fmt: int = E4M3, q: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                          h: torch.Tensor | None = None, y: torch.Tensor | None = None,
                          rstd: torch.Tensor | None = None, want_y: bool = False, want_rstd: bool = False, stream=None):
    """h = x + residual; RMS norm of h times weight, as 1x128 codes.

    Returns (q [R, C], scales [R, ceil(C/128)], h (x itself without a residual), y [R, C] in x's dtype or None,
    rstd [R] or None).  y and rstd are made when asked for (want_*) or given; h may be x or residual (in place).  Without
    columns rstd is NaN: the mean of no elements."""
    dev = _here(x)
    if stream is not None or dev < 0:
        with _ffn_context(x, stream):
            return fp8q_rmsnorm_quantize(x, weight, residual, eps, fmt, q, scales, h, y, rstd, want_y, want_rstd)
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("the norm takes a 2-D tensor")
    R, C = shape
    dt, code = x.dtype, _float_code(x, "x")
    blocks = (R, (C + 127) // 128)
    if q is None:
        q = torch.empty(shape, dtype=_U8, device=x.device)
    if scales is None:
        scales = torch.empty(blocks, dtype=_F32T, device=x.device)
    if residual is None:
        if h is not None:
            raise ValueError("h is written only with a residual")
    elif h is None:
        h = torch.empty_like(x)
    if y is None and want_y:
        y = torch.empty(shape, dtype=dt, device=x.device)
    if rstd is None and want_rstd:
        rstd = torch.empty(R, dtype=_F32T, device=x.device)
    if C == 0 and rstd is not None:  # the C call writes nothing for rows without columns
        _fits(rstd, "rstd", dev, (R,), _F32T)
        rstd.fill_(math.nan)
    st = load_library().fp8q_rmsnorm_quantize(
        _fits(x, "x", dev, shape, dt), code, None if residual is None else _fits(residual, "residual", dev, shape, dt),
        _fits(weight, "weight", dev, (C,), weight.dtype), _float_code(weight, "weight"), R, C, eps, fmt,
        _fits(q, "q", dev, shape, _U8), _fits(scales, "scales", dev, blocks, _F32T),
        None if h is None else _fits(h, "h", dev, shape, dt), None if y is None else _fits(y, "y", dev, shape, dt),
        None if rstd is None else _fits(rstd, "rstd", dev, (R,), _F32T), _raw_stream(dev))
    if st:
        raise FP8Error("fp8q_rmsnorm_quantize", st)
    return q, scales, x if residual is None else h, y, rstd


@functools.lru_cache(maxsize=256)
def _norm_workspace_bytes(device: int, rows: int, cols: int) -> int:  # device: the current one
    return load_library().fp8q_rmsnorm_backward_workspace(rows, cols)


def fp8q_rmsnorm_backward(dy: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor, weight: torch.Tensor,
                          dh: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                          dweight: torch.Tensor | None = None, want_dweight: bool = True,
                          workspace: torch.Tensor | None = None, stream=None):
    """Gradients of the RMS norm y = h * rstd * weight for dy; dh is the gradient that reaches h by the residual.

    Returns (dx [R, C] in dy's dtype, dweight [C] fp32 or None).  dx may be dy or dh (in place).  The workspace (for
    dweight; fp8q_rmsnorm_backward_workspace(R, C) bytes) is allocated by the call unless it is given."""
    dev = _here(dy)
    if stream is not None or dev < 0:
        with _ffn_context(dy, stream):
            return fp8q_rmsnorm_backward(dy, h, rstd, weight, dh, dx, dweight, want_dweight, workspace)
    shape = dy.shape
    if len(shape) != 2:
        raise ValueError("the norm takes a 2-D tensor")
    R, C = shape
    dt, code = dy.dtype, _float_code(dy, "dy")
    if dx is None:
        dx = torch.empty_like(dy)
    if dweight is None and want_dweight:
        dweight = torch.empty(C, dtype=_F32T, device=dy.device)
    ws = ws_bytes = 0
    if dweight is not None:
        if workspace is None:
            ws_bytes = _norm_workspace_bytes(dev, R, C)
            if ws_bytes > 0:
                workspace = torch.empty(ws_bytes, dtype=_U8, device=dy.device)
                ws = workspace.data_ptr()
        else:
            ws = _fits(workspace, "workspace", dev, workspace.shape, workspace.dtype)
            ws_bytes = workspace.nbytes
    st = load_library().fp8q_rmsnorm_backward(
        _fits(dy, "dy", dev, shape, dt), _fits(h, "h", dev, shape, dt), code, _fits(rstd, "rstd", dev, (R,), _F32T),
        _fits(weight, "weight", dev, (C,), weight.dtype), _float_code(weight, "weight"),
        None if dh is None else _fits(dh, "dh", dev, shape, dt), R, C, _fits(dx, "dx", dev, shape, dt),
        None if dweight is None else _fits(dweight, "dweight", dev, (C,), _F32T), ws, ws_bytes, _raw_stream(dev))
    if st:
        raise FP8Error("fp8q_rmsnorm_backward", st)
    return dx, dweight


def fp8q_gemm_gated(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor, a_fmt: int = E4M3,
                    b_fmt: int = E4M3, act: int = ACT_SILU, fmt: int = E4M3, q: torch.Tensor | None = None,
                    scales: torch.Tensor | None = None, gu: torch.Tensor | None = None, want_q: bool = True,
                    want_gu: bool = False, gu_dtype=torch.bfloat16, stream=None):
    """act(A Wg^T) * (A Wu^T) as 1x128 codes, from codes a [M, K] (1x128 scales) and b = [Wg; Wu] [2F, K] (128x128).

    Returns (q [M, F], scales [M, F/128], gu [M, 2F] = the projections G | U, or None)."""
    dev = _here(a)
    if stream is not None or dev < 0:
        with _ffn_context(a, stream):
            return fp8q_gemm_gated(a, sa, b, sb, a_fmt, b_fmt, act, fmt, q, scales, gu, want_q, want_gu, gu_dtype)
    ashape, bshape = a.shape, b.shape
    if len(ashape) != 2 or len(bshape) != 2 or ashape[1] != bshape[1] or bshape[0] % 2:
        raise ValueError("fp8q_gemm_gated takes a [M, K] and b [2F, K]")
    M, K = ashape
    F2 = bshape[0]
    F = F2 // 2
    if (q is None) != (scales is None):
        raise ValueError("q and scales go together")
    if q is None and want_q:
        q = torch.empty((M, F), dtype=_U8, device=a.device)
        scales = torch.empty((M, F // 128), dtype=_F32T, device=a.device)
    if gu is None and want_gu:
        gu = torch.empty((M, F2), dtype=gu_dtype, device=a.device)
    st = load_library().fp8q_gemm_gated(
        _fits(a, "a", dev, ashape, _U8), _fits(sa, "sa", dev, (M, K // 128), _F32T), a_fmt, _fits(b, "b", dev, bshape, _U8),
        _fits(sb, "sb", dev, (F2 // 128, K // 128), _F32T), b_fmt, M, F, K, act, fmt,
        None if q is None else _fits(q, "q", dev, (M, F), _U8),
        None if q is None else _fits(scales, "scales", dev, (M, F // 128), _F32T),
        None if gu is None else _fits(gu, "gu", dev, (M, F2), gu.dtype), F32 if gu is None else _float_code(gu, "gu"),
        _raw_stream(dev))
    if st:
        raise FP8Error("fp8q_gemm_gated", st)
    return q, scales, gu


def fp8q_gated_backward(gu: torch.Tensor, dh: torch.Tensor, act: int = ACT_SILU, fmt: int = E4M3, transposed: bool = True,
                        q: torch.Tensor | None = None, scales: torch.Tensor | None = None, qt: torch.Tensor | None = None,
                        scales_t: torch.Tensor | None = None, ht: torch.Tensor | None = None,
                        ht_scales: torch.Tensor | None = None, stream=None):
    """Backward pass of H = act(G) * U from gu = G | U [M, 2F] and dh = dH [M, F], as 1x128 codes.

    Returns (q [M, 2F], scales) of [dG | dU] and, unless transposed is false, (qt [2F, Mt], scales_t) of its
    transpose and (ht [F, Mt], ht_scales) of H^T, Mt = M rounded up to 128 (zero codes from M on); else None."""
    dev = _here(gu)
    if stream is not None or dev < 0:
        with _ffn_context(gu, stream):
            return fp8q_gated_backward(gu, dh, act, fmt, transposed, q, scales, qt, scales_t, ht, ht_scales)
    shape = gu.shape
    if len(shape) != 2 or shape[1] % 2:
        raise ValueError("fp8q_gated_backward takes gu [M, 2F]")
    M, F2 = shape
    F, Mb = F2 // 2, (M + 127) // 128
    Mt = Mb * 128
    code = _float_code(gu, "gu")
    new = lambda t, shape, dtype: torch.empty(shape, dtype=dtype, device=gu.device) if t is None else t  # noqa: E731
    q, scales = new(q, shape, _U8), new(scales, (M, F2 // 128), _F32T)
    pqt = pst = pht = phs = None
    if transposed:
        qt, scales_t = new(qt, (F2, Mt), _U8), new(scales_t, (F2, Mb), _F32T)
        ht, ht_scales = new(ht, (F, Mt), _U8), new(ht_scales, (F, Mb), _F32T)
        pqt, pst = _fits(qt, "qt", dev, (F2, Mt), _U8), _fits(scales_t, "scales_t", dev, (F2, Mb), _F32T)
        pht, phs = _fits(ht, "ht", dev, (F, Mt), _U8), _fits(ht_scales, "ht_scales", dev, (F, Mb), _F32T)
    elif not (qt is scales_t is ht is ht_scales is None):
        raise ValueError("qt, scales_t, ht and ht_scales are written only with transposed")
    st = load_library().fp8q_gated_backward(
        _fits(gu, "gu", dev, shape, gu.dtype), _fits(dh, "dh", dev, (M, F), gu.dtype), code, M, F, act, fmt,
        _fits(q, "q", dev, shape, _U8), _fits(scales, "scales", dev, (M, F2 // 128), _F32T), pqt, pst, pht, phs,
        _raw_stream(dev))
    if st:
        raise FP8Error("fp8q_gated_backward", st)
    return q, scales, qt, scales_t, ht, ht_scales


# -- a block of experts ---------------------------------------------------------------

class MoeRoute(NamedTuple):
    """Where the (token, expert) pairs have their rows, as fp8q_moe_sort makes it (int32 CUDA tensors).

    Pairs may be dropped afterwards by setting their pos to -1; src stays as it is."""
    offsets: torch.Tensor         # [E + 1]: expert e has rows offsets[e] .. offsets[e + 1] - 1
    pos: torch.Tensor             # [T, top_k]: the row of a pair, or -1
    src: torch.Tensor             # [R]: the pair t * top_k + k of a row, or -1
    counts: torch.Tensor | None   # [E]: the pairs of an expert


_I32T = torch.int32


@functools.lru_cache(maxsize=256)
def _moe_sizes(tokens: int, top_k: int, num_experts: int, align: int):
    L = load_library()
    rows = L.fp8q_moe_rows(tokens, top_k, num_experts, align)
    if rows < 0:
        raise FP8Error("fp8q_moe_rows", rows)
    return rows, L.fp8q_moe_sort_workspace(tokens, top_k, num_experts)


def fp8q_moe_rows(tokens: int, top_k: int, num_experts: int, align: int = 1) -> int:
    """Rows that hold any routing of tokens * top_k pairs."""
    return _moe_sizes(tokens, top_k, num_experts, align)[0]


def fp8q_moe_sort(experts: torch.Tensor, num_experts: int, align: int = 1, offsets: torch.Tensor | None = None,
                  pos: torch.Tensor | None = None, src: torch.Tensor | None = None, counts: torch.Tensor | None = None,
                  want_counts: bool = True, workspace: torch.Tensor | None = None, stream=None) -> MoeRoute:
    """The pairs of experts [T, top_k] (int32; an id outside 0 .. num_experts - 1 gives no row) sorted by expert, stable.

    Returns a MoeRoute; src has fp8q_moe_rows(T, top_k, num_experts, align) rows unless it is given.  align 128 is what
    transposed codes and the weights' gradients need.  The workspace (more than 4096 pairs; fp8q_moe_sort_workspace bytes)
    is allocated by the call unless it is given."""
    dev = _here(experts)
    if stream is not None or dev < 0:
        with _ffn_context(experts, stream):
            return fp8q_moe_sort(experts, num_experts, align, offsets, pos, src, counts, want_counts, workspace)
    shape = experts.shape
    if len(shape) != 2:
        raise ValueError("fp8q_moe_sort takes experts [T, top_k]")
    T, top_k = shape
    rows, ws_bytes = _moe_sizes(T, top_k, num_experts, align)
    if offsets is None:
        offsets = torch.empty(num_experts + 1, dtype=_I32T, device=experts.device)
    if pos is None:
        pos = torch.empty(shape, dtype=_I32T, device=experts.device)
    if src is None:
        src = torch.empty(rows, dtype=_I32T, device=experts.device)
    if counts is None and want_counts:
        counts = torch.empty(num_experts, dtype=_I32T, device=experts.device)
    ws = 0
    if workspace is not None:
        ws, ws_bytes = _fits(workspace, "workspace", dev, workspace.shape, workspace.dtype), workspace.nbytes
    elif ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=_U8, device=experts.device)
        ws = workspace.data_ptr()
    R = src.numel()
    st = load_library().fp8q_moe_sort(
        _fits(experts, "experts", dev, shape, _I32T), T, top_k, num_experts, align, R,
        _fits(offsets, "offsets", dev, (num_experts + 1,), _I32T), _fits(pos, "pos", dev, shape, _I32T),
        _fits(src, "src", dev, (R,), _I32T), None if counts is None else _fits(counts, "counts", dev, (num_experts,), _I32T),
        ws, ws_bytes, _raw_stream(dev))
    if st:
        raise FP8Error("fp8q_moe_sort", st)
    return MoeRoute(offsets, pos, src, counts)


def _route_args(route: MoeRoute, dev: int, tokens: int):
    """The C arguments offsets, num_experts, pos, src, tokens, top_k, rows."""
    offsets, pos, src, _ = route
    oshape, pshape, sshape = offsets.shape, pos.shape, src.shape
    if len(oshape) != 1 or len(pshape) != 2 or len(sshape) != 1 or oshape[0] < 1:
        raise ValueError("a route has offsets [E + 1], pos [T, top_k] and src [R]")
    top_k = pshape[1]
    return (_fits(offsets, "offsets", dev, oshape, _I32T), oshape[0] - 1, _fits(pos, "pos", dev, (tokens, top_k), _I32T),
            _fits(src, "src", dev, sshape, _I32T), tokens, top_k, sshape[0])


def _row_codes(dev: int, device, R: int, C: int, transposed: bool, q, scales, qt, scales_t):
    """Outputs [R, C] as codes, with their transpose where it is wanted, and their addresses."""
    shape, blocks = (R, C), (R, C // 128)
    if q is None:
        q = torch.empty(shape, dtype=_U8, device=device)
    if scales is None:
        scales = torch.empty(blocks, dtype=_F32T, device=device)
    pq, ps = _fits(q, "q", dev, shape, _U8), _fits(scales, "scales", dev, blocks, _F32T)
    if not transposed:
        if not (qt is scales_t is None):
            raise ValueError("qt and scales_t are written only with transposed")
        return (q, scales, None, None), (pq, ps, None, None)
    shape, blocks = (C, R), (C, R // 128)
    if qt is None:
        qt = torch.empty(shape, dtype=_U8, device=device)
    if scales_t is None:
        scales_t = torch.empty(blocks, dtype=_F32T, device=device)
    return (q, scales, qt, scales_t), (pq, ps, _fits(qt, "qt", dev, shape, _U8), _fits(scales_t, "scales_t", dev, blocks, _F32T))


def fp8q_moe_dispatch(x: torch.Tensor, route: MoeRoute, fmt: int = E4M3, transposed: bool = False,
                      q: torch.Tensor | None = None, scales: torch.Tensor | None = None, qt: torch.Tensor | None = None,
                      scales_t: torch.Tensor | None = None, stream=None):
    """The tokens x [T, C] at the rows of their experts, as 1x128 codes; zeros on rows without a pair.

    Returns (q [R, C], scales [R, C/128], qt [C, R], scales_t [C, R/128]); the transposed two are None unless transposed.
    Rows from offsets[E] on are not written.  The gradient is fp8q_moe_combine(drows, route) without weights."""
    dev = _here(x)
    if stream is not None or dev < 0:
        with _ffn_context(x, stream):
            return fp8q_moe_dispatch(x, route, fmt, transposed, q, scales, qt, scales_t)
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("fp8q_moe_dispatch takes x [T, C]")
    T, C = shape
    rargs = _route_args(route, dev, T)
    out, ptrs = _row_codes(dev, x.device, rargs[-1], C, transposed, q, scales, qt, scales_t)
    st = load_library().fp8q_moe_dispatch(_fits(x, "x", dev, shape, x.dtype), _float_code(x, "x"), C, *rargs, fmt, *ptrs,
                                          _raw_stream(dev))
    if st:
        raise FP8Error("fp8q_moe_dispatch", st)
    return out


def fp8q_moe_dispatch_codes(xq: torch.Tensor, xs: torch.Tensor, route: MoeRoute, fmt: int = E4M3,
                            q: torch.Tensor | None = None, scales: torch.Tensor | None = None, stream=None):
    """The tokens' codes xq [T, C] and scales xs [T, C/128] at the rows of their experts.  Returns (q [R, C], scales)."""
    dev = _here(xq)
    if stream is not None or dev < 0:
        with _ffn_context(xq, stream):
            return fp8q_moe_dispatch_codes(xq, xs, route, fmt, q, scales)
    shape = xq.shape
    if len(shape) != 2:
        raise ValueError("fp8q_moe_dispatch_codes takes xq [T, C]")
    T, C = shape
    rargs = _route_args(route, dev, T)
    out, ptrs = _row_codes(dev, xq.device, rargs[-1], C, False, q, scales, None, None)
    st = load_library().fp8q_moe_dispatch_codes(_fits(xq, "xq", dev, shape, _U8), _fits(xs, "xs", dev, (T, C // 128), _F32T),
                                                fmt, C, *rargs, ptrs[0], ptrs[1], _raw_stream(dev))
    if st:
        raise FP8Error("fp8q_moe_dispatch_codes", st)
    return out[:2]


def fp8q_moe_combine(rows: torch.Tensor, route: MoeRoute, weights: torch.Tensor | None = None,
                     residual: torch.Tensor | None = None, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[t] = residual[t] + sum over k of weights[t, k] * rows[pos[t, k]] (ones without weights), [T, C] in rows' dtype."""
    dev = _here(rows)
    if stream is not None or dev < 0:
        with _ffn_context(rows, stream):
            return fp8q_moe_combine(rows, route, weights, residual, y)
    shape = rows.shape
    pos = route.pos
    if len(shape) != 2 or pos.dim() != 2:
        raise ValueError("fp8q_moe_combine takes rows [R, C] and a route with pos [T, top_k]")
    R, C = shape
    T, top_k = pos.shape
    dt, code = rows.dtype, _float_code(rows, "rows")
    if y is None:
        y = torch.empty((T, C), dtype=dt, device=rows.device)
    st = load_library().fp8q_moe_combine(
        _fits(rows, "rows", dev, shape, dt), code, R, C, _fits(pos, "pos", dev, (T, top_k), _I32T),
        None if weights is None else _fits(weights, "weights", dev, (T, top_k), _F32T),
        None if residual is None else _fits(residual, "residual", dev, (T, C), dt), T, top_k, _fits(y, "y", dev, (T, C), dt),
        _raw_stream(dev))
    if st:
        raise FP8Error("fp8q_moe_combine", st)
    return y


def fp8q_moe_combine_backward(dy: torch.Tensor, rows: torch.Tensor | None, route: MoeRoute, weights: torch.Tensor,
                              fmt: int = E4M3, transposed: bool = True, q: torch.Tensor | None = None,
                              scales: torch.Tensor | None = None, qt: torch.Tensor | None = None,
                              scales_t: torch.Tensor | None = None, dweights: torch.Tensor | None = None,
                              want_dweights: bool = True, stream=None):
    """Gradients of fp8q_moe_combine for dy [T, C]: of the rows, weights[t, k] * dy[t] as 1x128 codes, and of the weights.

    Returns (q [R, C], scales, qt [C, R], scales_t, dweights [T, top_k] fp32); qt and scales_t are None unless
    transposed, dweights unless wanted (rows, the forward call's, may then be None).  Rows from offsets[E] on are not
    written."""
    dev = _here(dy)
    if stream is not None or dev < 0:
        with _ffn_context(dy, stream):
            return fp8q_moe_combine_backward(dy, rows, route, weights, fmt, transposed, q, scales, qt, scales_t, dweights,
                                             want_dweights)
    shape = dy.shape
    if len(shape) != 2:
        raise ValueError("fp8q_moe_combine_backward takes dy [T, C]")
    T, C = shape
    dt, code = dy.dtype, _float_code(dy, "dy")
    rargs = _route_args(route, dev, T)
    top_k, R = rargs[-2:]
    if dweights is None and want_dweights:
        dweights = torch.empty((T, top_k), dtype=_F32T, device=dy.device)
    if dweights is not None and rows is None:
        raise ValueError("the weights' gradient needs the rows")
    out, ptrs = _row_codes(dev, dy.device, R, C, transposed, q, scales, qt, scales_t)
    st = load_library().fp8q_moe_combine_backward(
        _fits(dy, "dy", dev, shape, dt), None if rows is None else _fits(rows, "rows", dev, (R, C), dt), code, C, *rargs,
        _fits(weights, "weights", dev, (T, top_k), _F32T), fmt, *ptrs,
        None if dweights is None else _fits(dweights, "dweights", dev, (T, top_k), _F32T), _raw_stream(dev))
    if st:
        raise FP8Error("fp8q_moe_combine_backward", st)
    return (*out, dweights)


def _grouped_args(a, sa, b, sb, offsets, dev: int, name: str):
    """The C arguments a, sa, a_fmt .. of both grouped products, checked: (pointers, offsets, E, R, N, K)."""
    ashape, bshape = a.shape, b.shape
    if len(ashape) != 2 or len(bshape) != 3 or ashape[1] != bshape[2] or offsets.dim() != 1:
        raise ValueError(f"{name} takes a [R, K], b [E, N, K] and offsets [E + 1]")
    R, K = ashape
    E, N = bshape[:2]
    return (_fits(a, "a", dev, ashape, _U8), _fits(sa, "sa", dev, (R, K // 128), _F32T), _fits(b, "b", dev, bshape, _U8),
            _fits(sb, "sb", dev, (E, N // 128, K // 128), _F32T), _fits(offsets, "offsets", dev, (E + 1,), _I32T), E, R, N, K)


def fp8q_gemm_grouped(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor, offsets: torch.Tensor,
                      a_fmt: int = E4M3, b_fmt: int = E4M3, out_dtype=torch.bfloat16, c: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """c [R, N]: rows offsets[e] .. offsets[e + 1] - 1 of a [R, K] (1x128 scales) times b[e]^T, b [E, N, K] (128x128).

    Rows from offsets[E] on are not written."""
    dev = _here(a)
    if stream is not None or dev < 0:
        with _ffn_context(a, stream):
            return fp8q_gemm_grouped(a, sa, b, sb, offsets, a_fmt, b_fmt, out_dtype, c)
    pa, psa, pb, psb, poff, E, R, N, K = _grouped_args(a, sa, b, sb, offsets, dev, "fp8q_gemm_grouped")
    if c is None:
        c = torch.empty((R, N), dtype=out_dtype, device=a.device)
    st = load_library().fp8q_gemm_grouped(pa, psa, a_fmt, pb, psb, b_fmt, poff, E, R, N, K, _fits(c, "c", dev, (R, N), c.dtype),
                                          _float_code(c, "c"), _raw_stream(dev))
    if st:
        raise FP8Error("fp8q_gemm_grouped", st)
    return c


def fp8q_gemm_gated_grouped(a: torch.Tensor, sa: torch.Tensor, b: torch.Tensor, sb: torch.Tensor, offsets: torch.Tensor,
                            a_fmt: int = E4M3, b_fmt: int = E4M3, act: int = ACT_SILU, fmt: int = E4M3,
                            q: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                            gu: torch.Tensor | None = None, want_q: bool = True, want_gu: bool = False,
                            gu_dtype=torch.bfloat16, stream=None):
    """fp8q_gemm_gated with rows offsets[e] .. offsets[e + 1] - 1 of a [R, K] against b[e] = [Wg; Wu], b [E, 2F, K].

    Returns (q [R, F], scales [R, F/128], gu [R, 2F] = the projections G | U, or None).  Rows from offsets[E] on are not
    written."""
    dev = _here(a)
    if stream is not None or dev < 0:
        with _ffn_context(a, stream):
            return fp8q_gemm_gated_grouped(a, sa, b, sb, offsets, a_fmt, b_fmt, act, fmt, q, scales, gu, want_q, want_gu,
                                           gu_dtype)
    pa, psa, pb, psb, poff, E, R, F2, K = _grouped_args(a, sa, b, sb, offsets, dev, "fp8q_gemm_gated_grouped")
    if F2 % 2:
        raise ValueError("fp8q_gemm_gated_grouped takes b [E, 2F, K]")
    F = F2 // 2
    if (q is None) != (scales is None):
        raise ValueError("q and scales go together")
    if q is None and want_q:
        q = torch.empty((R, F), dtype=_U8, device=a.device)
        scales = torch.empty((R, F // 128), dtype=_F32T, device=a.device)
    if gu is None and want_gu:
        gu = torch.empty((R, F2), dtype=gu_dtype, device=a.device)
    st = load_library().fp8q_gemm_gated_grouped(
        pa, psa, a_fmt, pb, psb, b_fmt, poff, E, R, F, K, act, fmt, None if q is None else _fits(q, "q", dev, (R, F), _U8),
        None if q is None else _fits(scales, "scales", dev, (R, F // 128), _F32T),
        None if gu is None else _fits(gu, "gu", dev, (R, F2), gu.dtype), F32 if gu is None else _float_code(gu, "gu"),
        _raw_stream(dev))
    if st:
        raise FP8Error("fp8q_gemm_gated_grouped", st)
    return q, scales, gu


def fp8q_gemm_grouped_wgrad(at: torch.Tensor, sat: torch.Tensor, bt: torch.Tensor, sbt: torch.Tensor, offsets: torch.Tensor,
                            a_fmt: int = E4M3, b_fmt: int = E4M3, out_dtype=torch.float32, dw: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """dw [E, N, K]: the products of at [N, R] and bt [K, R] (1x128 scales) over each expert's rows; offsets [E + 1] are
    multiples of 128 (a sort with align 128)."""
    dev = _here(at)
    if stream is not None or dev < 0:
        with _ffn_context(at, stream):
            return fp8q_gemm_grouped_wgrad(at, sat, bt, sbt, offsets, a_fmt, b_fmt, out_dtype, dw)
    ashape, bshape = at.shape, bt.shape
    if len(ashape) != 2 or len(bshape) != 2 or ashape[1] != bshape[1] or offsets.dim() != 1 or offsets.numel() < 1:
        raise ValueError("fp8q_gemm_grouped_wgrad takes at [N, R], bt [K, R] and offsets [E + 1]")
    N, R = ashape
    K, E = bshape[0], offsets.numel() - 1
    if dw is None:
        dw = torch.empty((E, N, K), dtype=out_dtype, device=at.device)
    st = load_library().fp8q_gemm_grouped_wgrad(
        _fits(at, "at", dev, ashape, _U8), _fits(sat, "sat", dev, (N, R // 128), _F32T), a_fmt,
        _fits(bt, "bt", dev, bshape, _U8), _fits(sbt, "sbt", dev, (K, R // 128), _F32T), b_fmt,
        _fits(offsets, "offsets", dev, (E + 1,), _I32T), E, R, N, K, _fits(dw, "dw", dev, (E, N, K), dw.dtype),
        _float_code(dw, "dw"), _raw_stream(dev))
    if st:
        raise FP8Error("fp8q_gemm_grouped_wgrad", st)
    return dw


class DelayedScaler:
    """Device-resident delayed-scaling state (history ring, {pos, count}, scale), after the
    PyTorch-FP8 page's DelayedScaler (s4.2).  step(x) quantizes x with the current scale, then
    pushes amax(x) into the history -- all on the device, no host round trip.  fused=True (the
    default) does both in one launch (fp8_quantize_delayed_step); fused=False uses the two calls."""

    def __init__(self, window: int = 16, fmt: int = E5M2, device="cuda", algo: int = AMAX_WINDOW_MAX,
                 alpha: float = 1.0, margin: float = 1.0, fused: bool = True):
        self.fmt = fmt
        self.fused = fused
        self.workspace = fused_workspace(device) if fused else None
        self.algo, self.alpha, self.margin = algo, alpha, margin
        self.history = torch.zeros(window, dtype=torch.float32, device=device)
        self.state = torch.zeros(2, dtype=torch.int32, device=device)
        self.scale = torch.ones(1, dtype=torch.float32, device=device)
        self.amax = torch.zeros(1, dtype=torch.float32, device=device)
        self.scale_used = torch.ones(1, dtype=torch.float32, device=device)

    def step(self, x: torch.Tensor, q: torch.Tensor | None = None, stream=None):
        if self.fused:
            q = fp8_quantize_delayed_step(x, self.scale, self.history, self.state, self.fmt, self.algo, self.alpha,
                                          self.margin, q=q, scale_used=self.scale_used, amax_out=self.amax,
                                          workspace=self.workspace, stream=stream)
            return q, self.scale_used
        q, s, _ = fp8_quantize_per_tensor(x, self.fmt, scale_in=self.scale, q=q, scale_out=self.scale_used,
                                          amax_out=self.amax, stream=stream)
        if self.algo == AMAX_WINDOW_MAX and self.margin == 1.0:
            fp8_amax_history_update(self.history, self.state, self.amax, self.scale, self.fmt, stream=stream)
        else:
            fp8_amax_history_update_ex(self.history, self.state, self.amax, self.scale, self.fmt, self.algo,
                                       self.alpha, self.margin, stream=stream)
        return q, self.scale_used
