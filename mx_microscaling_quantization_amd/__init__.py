"""MX (microscaling) quantize on AMD MI355X -- Python binding of ``libmxq.so``.

A thin ctypes layer over the C ABI declared in ``include/mxq.h``: it maps
torch dtypes to the ABI's codes, allocates outputs with torch when the caller
gives none, and passes raw device pointers and the current HIP stream. Every
step of the quantize runs in the library's HIP kernels; there is no fallback.
If ``libmxq.so`` is missing or cannot be loaded, importing the functions below
raises.
"""
from __future__ import annotations

import array
import ctypes
import functools
import os
import threading
from typing import NamedTuple

import torch  # loaded first so that the library binds to torch's HIP runtime

__all__ = [
    "IN_DTYPES", "OUT_DTYPES", "RES_DTYPES", "ELEM_DTYPES", "MXQError", "quantize", "dequantize", "quantize_axis",
    "scaled_matmul", "scaled_matmul_quantize", "MoEPlan", "moe_rows", "moe_sort", "moe_gather_quantize", "moe_combine",
    "moe_combine_backward", "grouped_scaled_matmul", "grouped_scaled_matmul_wgrad", "clip_grad_norm", "grad_norm",
    "data_bytes", "scale_image_bytes", "result_bytes", "data_shape", "scale_image_shape",
    "axis_view_shape", "logical_scale_view", "status_string", "library_path", "load",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libmxq.so"

IN_DTYPES = {torch.bfloat16: 0, torch.float16: 1}
OUT_DTYPES = {"e4m3fn": 0, "e5m2": 1, "e2m1": 2}
RES_DTYPES = {torch.float32: 0, torch.bfloat16: 1}
ELEM_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
FLAG_ALT_EMAX = 1
FLAG_DENSE_SCALE = 2
ABI_VERSION = 1

_lock = threading.Lock()
_lib = None


class MXQError(RuntimeError):
    """A non-zero status from the library (``status`` holds the code)."""

    def __init__(self, status: int, message: str):
        super().__init__("mxq status %d: %s" % (status, message))
        self.status = status


def library_path() -> str:
    return os.path.join(_HERE, _LIB_NAME)


def load():
    """Load ``libmxq.so`` (once) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            raise ImportError("%s is not built; run `python -m mx_microscaling_quantization_amd._build` (hipcc, gfx950) first" % path)
        lib = ctypes.CDLL(path)
        c = ctypes
        lib.mxq_quantize.argtypes = [c.c_void_p, c.c_int64, c.c_int64, c.c_int, c.c_int, c.c_void_p,
                                     c.c_void_p, c.c_void_p]
        lib.mxq_quantize.restype = c.c_int
        lib.mxq_quantize_ex.argtypes = [c.c_void_p, c.c_int64, c.c_int64, c.c_int, c.c_int, c.c_uint,
                                        c.c_void_p, c.c_void_p, c.c_void_p]
        lib.mxq_quantize_ex.restype = c.c_int
        lib.mxq_dequantize_ex.argtypes = [c.c_void_p, c.c_void_p, c.c_int64, c.c_int64, c.c_int, c.c_int,
                                          c.c_uint, c.c_void_p, c.c_void_p]
        lib.mxq_dequantize_ex.restype = c.c_int
        lib.mxq_scaled_matmul.argtypes = [c.c_void_p, c.c_void_p, c.c_void_p, c.c_void_p, c.c_int64, c.c_int64,
                                          c.c_int64, c.c_int, c.c_int, c.c_uint, c.c_void_p, c.c_void_p]
        lib.mxq_scaled_matmul.restype = c.c_int
        lib.mxq_scaled_matmul_quantize.argtypes = [c.c_void_p, c.c_void_p, c.c_void_p, c.c_void_p, c.c_int64,
                                                   c.c_int64, c.c_int64, c.c_int, c.c_int, c.c_uint, c.c_void_p,
                                                   c.c_void_p, c.c_void_p]
        lib.mxq_scaled_matmul_quantize.restype = c.c_int
        lib.mxq_quantize_axis.argtypes = [c.c_void_p, c.c_int64, c.c_int64, c.c_int, c.c_int, c.c_int, c.c_uint,
                                          c.c_void_p, c.c_void_p, c.c_void_p]
        lib.mxq_quantize_axis.restype = c.c_int
        lib.mxq_scale_bytes.argtypes = [c.c_int64, c.c_int64, c.c_uint]
        lib.mxq_scale_bytes.restype = c.c_size_t
        lib.mxq_data_bytes.argtypes = [c.c_int64, c.c_int64, c.c_int]
        lib.mxq_data_bytes.restype = c.c_size_t
        lib.mxq_scale_image_bytes.argtypes = [c.c_int64, c.c_int64]
        lib.mxq_scale_image_bytes.restype = c.c_size_t
        lib.mxq_dequantize.argtypes = [c.c_void_p, c.c_void_p, c.c_int64, c.c_int64, c.c_int, c.c_int,
                                       c.c_void_p, c.c_void_p]
        lib.mxq_dequantize.restype = c.c_int
        lib.mxq_result_bytes.argtypes = [c.c_int64, c.c_int64, c.c_int]
        lib.mxq_result_bytes.restype = c.c_size_t
        p, i64 = c.c_void_p, c.c_int64
        lib.mxq_moe_rows.argtypes = [i64, i64, i64, i64]
        lib.mxq_moe_rows.restype = i64
        lib.mxq_moe_sort_workspace_bytes.argtypes = [i64, i64, i64]
        lib.mxq_moe_sort_workspace_bytes.restype = c.c_size_t
        lib.mxq_moe_sort.argtypes = [p, c.c_int, i64, i64, i64, i64, p, p, p, p, p]
        lib.mxq_moe_sort.restype = c.c_int
        lib.mxq_moe_gather_quantize.argtypes = [p, i64, i64, i64, c.c_int, c.c_int, c.c_int, c.c_uint, p, i64, p, p, p]
        lib.mxq_moe_gather_quantize.restype = c.c_int
        lib.mxq_moe_combine.argtypes = [p, i64, i64, c.c_int, p, p, i64, i64, p, p]
        lib.mxq_moe_combine.restype = c.c_int
        lib.mxq_moe_combine_backward.argtypes = [p, p, i64, i64, c.c_int, p, p, p, i64, i64, p, p, p]
        lib.mxq_moe_combine_backward.restype = c.c_int
        for name in ("mxq_grouped_matmul", "mxq_grouped_matmul_wgrad"):
            fn = getattr(lib, name)
            fn.argtypes = [p, p, p, p, p, i64, i64, i64, i64, c.c_int, c.c_int, p, p]
            fn.restype = c.c_int
        lib.mxq_clip_grad_norm_workspace_bytes.argtypes = [p, p, i64]
        lib.mxq_clip_grad_norm_workspace_bytes.restype = c.c_size_t
        lib.mxq_clip_grad_norm.argtypes = [p, p, p, p, i64, c.c_double, p, p, p]
        lib.mxq_clip_grad_norm.restype = c.c_int
        lib.mxq_status_string.argtypes = [c.c_int]
        lib.mxq_status_string.restype = c.c_char_p
        lib.mxq_abi_version.argtypes = []
        lib.mxq_abi_version.restype = c.c_int
        if lib.mxq_abi_version() != ABI_VERSION:
            raise ImportError("libmxq.so ABI %d, binding expects %d" % (lib.mxq_abi_version(), ABI_VERSION))
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().mxq_status_string(int(status)).decode()


def _check(status: int) -> None:
    if status != 0:
        raise MXQError(status, status_string(status))


def _out_code(out_dtype: str) -> int:
    try:
        return OUT_DTYPES[out_dtype]
    except KeyError:
        raise MXQError(2, "output element type must be one of %s" % sorted(OUT_DTYPES)) from None


# torch's accessor for the raw handle of a device's current stream (what its
# own kernels launch on), when it has one; the public route costs more per
# call
_raw_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream, device: torch.device) -> int:
    """The raw HIP stream handle to enqueue on: ``stream``'s, else the current
    stream of ``device``."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_current_stream is not None:
        return _raw_current_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


# the current device's index; its tensors are there, so nothing is left to
# initialize
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call_on(device: torch.device, fn, *args) -> int:
    """Call ``fn(*args)`` with ``device`` current (the library launches on
    the current device), entering a device context only when it is not."""
    if _current_device() == device.index:
        return fn(*args)
    with torch.cuda.device(device):
        return fn(*args)


@functools.lru_cache(maxsize=256)
def _data_nbytes(P: int, F: int, code: int) -> int:
    return int(load().mxq_data_bytes(P, F, code))


@functools.lru_cache(maxsize=256)
def _scale_nbytes(P: int, F: int, flags: int) -> int:
    return int(load().mxq_scale_bytes(P, F, flags))


def _check_out_buffer(name: str, t: torch.Tensor, nbytes: int, device: torch.device) -> None:
    """An output the library writes through a raw pointer: contiguous, on
    ``device``, and at least ``nbytes`` long (its element type is not read)."""
    if t.device != device or not t.is_contiguous() or t.numel() * t.element_size() < nbytes:
        raise ValueError("%s must be a contiguous buffer of >= %d bytes on %s" % (name, nbytes, device))


def data_bytes(P: int, F: int, out_dtype: str) -> int:
    return int(load().mxq_data_bytes(P, F, _out_code(out_dtype)))


def scale_image_bytes(P: int, F: int) -> int:
    return int(load().mxq_scale_image_bytes(P, F))


def result_bytes(P: int, F: int, res_dtype: torch.dtype) -> int:
    return int(load().mxq_result_bytes(P, F, RES_DTYPES[res_dtype]))


def data_shape(P: int, F: int, out_dtype: str):
    """uint8 shape of the data output: [P, F] (FP8) or [P, F/2] (FP4)."""
    return (P, F // 2) if out_dtype == "e2m1" else (P, F)


def scale_image_shape(P: int, F: int, dense_scale: bool = False):
    """uint8 shape of the scale output: the [P, F/4] image, or [P/8, F/4]
    with ``dense_scale``."""
    return (P // 8, F // 4) if dense_scale else (P, F // 4)


def logical_scale_view(image: torch.Tensor) -> torch.Tensor:
    """View [P/32, 4, F/4] of the written rows of a scale image (P % 32 == 0):
    element [q, j, c] is the E8M0 of row group 4q + j, column block c."""
    P, C = image.shape
    if P % 32:
        raise ValueError("logical_scale_view needs P % 32 == 0")
    return image.view(P // 32, 32, C)[:, :4, :]


def quantize(x: torch.Tensor, out_dtype: str = "e4m3fn", data_out: torch.Tensor | None = None,
             scale_out: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None,
             alt_emax: bool = False, dense_scale: bool = False):
    """MX-quantize a contiguous [P, F] bf16/f16 CUDA (HIP) tensor.

    Returns ``(data, scale)`` as uint8 tensors: data [P, F] (FP8) or
    [P, F/2] (FP4); the scale image [P, F/4], of which rows
    (i mod 4) + 32 * floor(i / 4) hold row group i's E8M0 bytes and the other
    rows keep whatever ``scale_out`` held -- or, with ``dense_scale``, the
    dense [P/8, F/4] scale array. ``alt_emax`` selects the EMAX - 1 bias.
    The kernel is enqueued on ``stream`` (default: the current stream of x's
    device).
    """
    lib = load()
    if x.dtype not in IN_DTYPES:
        raise MXQError(1, "input element type must be bfloat16 or float16, got %s" % x.dtype)
    code = _out_code(out_dtype)
    if x.dim() != 2:
        raise ValueError("x must be 2-D [P, F]")
    if not x.is_cuda:
        raise ValueError("x must be a device tensor")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous (row pitch F)")
    P, F = x.shape
    if data_out is None:
        data_out = torch.empty(data_shape(P, F, out_dtype), dtype=torch.uint8, device=x.device)
    flags = (FLAG_ALT_EMAX if alt_emax else 0) | (FLAG_DENSE_SCALE if dense_scale else 0)
    if scale_out is None:
        scale_out = torch.empty(scale_image_shape(P, F, dense_scale), dtype=torch.uint8, device=x.device)
    _check_out_buffer("data_out", data_out, _data_nbytes(P, F, code), x.device)
    _check_out_buffer("scale_out", scale_out, _scale_nbytes(P, F, flags), x.device)
    sh = _stream_handle(stream, x.device)
    if flags == 0:    # the contract's own entry point
        _check(_call_on(x.device, lib.mxq_quantize, x.data_ptr(), P, F, IN_DTYPES[x.dtype], code,
                        data_out.data_ptr(), scale_out.data_ptr(), sh))
    else:
        _check(_call_on(x.device, lib.mxq_quantize_ex, x.data_ptr(), P, F, IN_DTYPES[x.dtype], code, flags,
                        data_out.data_ptr(), scale_out.data_ptr(), sh))
    return data_out, scale_out


def dequantize(data: torch.Tensor, scale_image: torch.Tensor, out_dtype: str = "e4m3fn",
               res_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
               stream: torch.cuda.Stream | None = None, dense_scale: bool = False) -> torch.Tensor:
    """Decode MX data back to [P, F] float32 or bfloat16.

    ``data`` is the uint8 data output of :func:`quantize` for format
    ``out_dtype`` ([P, F] FP8 or [P, F/2] FP4) and ``scale_image`` its
    [P, F/4] scale image (or, with ``dense_scale``, its [P/8, F/4] scale
    array). Each result is decode(code) * 2^(E8M0 - 127), rounded once to
    float32 (then nearest-even to bfloat16).
    """
    lib = load()
    code = _out_code(out_dtype)
    if res_dtype not in RES_DTYPES:
        raise MXQError(10, "result type must be float32 or bfloat16, got %s" % res_dtype)
    if data.dim() != 2 or scale_image.dim() != 2:
        raise ValueError("data and scale_image must be 2-D")
    if not data.is_cuda or scale_image.device != data.device:
        raise ValueError("data and scale_image must be device tensors on one device")
    if not (data.is_contiguous() and scale_image.is_contiguous()):
        raise ValueError("data and scale_image must be contiguous")
    if data.dtype != torch.uint8 or scale_image.dtype != torch.uint8:
        raise ValueError("data and scale_image must be uint8 (the bytes quantize wrote)")
    P = data.shape[0]
    F = scale_image.shape[1] * 4
    if tuple(data.shape) != data_shape(P, F, out_dtype) or \
            tuple(scale_image.shape) != scale_image_shape(P, F, dense_scale):
        raise ValueError("data %s / scale_image %s do not describe one [P, F] tensor in format %s"
                         % (tuple(data.shape), tuple(scale_image.shape), out_dtype))
    if out is None:
        out = torch.empty((P, F), dtype=res_dtype, device=data.device)
    elif out.dtype != res_dtype or tuple(out.shape) != (P, F) or not out.is_contiguous() or out.device != data.device:
        raise ValueError("out must be a contiguous [%d, %d] %s tensor on %s" % (P, F, res_dtype, data.device))
    sh = _stream_handle(stream, data.device)
    _check(_call_on(data.device, lib.mxq_dequantize_ex, data.data_ptr(), scale_image.data_ptr(), P, F, code,
                    RES_DTYPES[res_dtype], FLAG_DENSE_SCALE if dense_scale else 0, out.data_ptr(), sh))
    return out


def _check_operands(lhs, lhs_scale, rhs, rhs_scale, dense_scale):
    for t in (lhs, lhs_scale, rhs, rhs_scale):
        if t.dim() != 2 or t.dtype != torch.uint8 or not t.is_contiguous() or t.device != lhs.device or not t.is_cuda:
            raise ValueError("operands must be contiguous 2-D uint8 device tensors on one device")
    P = lhs.shape[0]
    M, N = lhs.shape[1] // 4, rhs.shape[1] // 4
    if rhs.shape[0] != P or lhs.shape[1] % 4 or rhs.shape[1] % 4:
        raise ValueError("lhs [P, 4M] and rhs [P, 4N] must share P")
    if tuple(lhs_scale.shape) != scale_image_shape(P, 4 * M, dense_scale) or \
            tuple(rhs_scale.shape) != scale_image_shape(P, 4 * N, dense_scale):
        raise ValueError("scale shapes do not match the operands")
    return P, M, N


def scaled_matmul(lhs: torch.Tensor, lhs_scale: torch.Tensor, rhs: torch.Tensor, rhs_scale: torch.Tensor,
                  fmt: str = "e4m3fn", res_dtype: torch.dtype = torch.float32, out: torch.Tensor | None = None,
                  stream: torch.cuda.Stream | None = None, dense_scale: bool = False) -> torch.Tensor:
    """Block-scaled matmul of two quantized operands.

    ``lhs`` [P, 4M] and ``rhs`` [P, 4N] are FP8 data outputs of
    :func:`quantize` (format ``fmt``) with their scale images ``lhs_scale``
    [P, M] and ``rhs_scale`` [P, N] (or dense [P/8, M], [P/8, N] with
    ``dense_scale``). Each operand is read as the [K = 4P, C] matrix whose
    row k = 4p + j holds element (p, 4c + j). Returns
    out[m][n] = sum_k L[k][m] * R[k][n] as [M, N] float32 or bfloat16.
    """
    lib = load()
    code = _out_code(fmt)
    if res_dtype not in RES_DTYPES:
        raise MXQError(10, "result type must be float32 or bfloat16, got %s" % res_dtype)
    P, M, N = _check_operands(lhs, lhs_scale, rhs, rhs_scale, dense_scale)
    if out is None:
        out = torch.empty((M, N), dtype=res_dtype, device=lhs.device)
    elif out.dtype != res_dtype or tuple(out.shape) != (M, N) or not out.is_contiguous() or out.device != lhs.device:
        raise ValueError("out must be a contiguous [%d, %d] %s tensor on %s" % (M, N, res_dtype, lhs.device))
    sh = _stream_handle(stream, lhs.device)
    _check(_call_on(lhs.device, lib.mxq_scaled_matmul, lhs.data_ptr(), lhs_scale.data_ptr(), rhs.data_ptr(),
                    rhs_scale.data_ptr(), P, M, N, code, RES_DTYPES[res_dtype],
                    FLAG_DENSE_SCALE if dense_scale else 0, out.data_ptr(), sh))
    return out


def scaled_matmul_quantize(lhs: torch.Tensor, lhs_scale: torch.Tensor, rhs: torch.Tensor, rhs_scale: torch.Tensor,
                           fmt: str = "e4m3fn", out_dtype: str = "e4m3fn", data_out: torch.Tensor | None = None,
                           scale_out: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None,
                           alt_emax: bool = False, dense_scale: bool = False):
    """The scaled matmul with its [M, N] result quantized in the same kernel.

    Operands as for :func:`scaled_matmul`. Returns ``(data, scale)`` -- the
    bytes :func:`quantize` would write for the bfloat16 result of
    :func:`scaled_matmul` (P = M rows, F = N columns, format ``out_dtype``),
    without that result ever being stored. ``dense_scale`` applies to the
    operand scales and the result scale; ``alt_emax`` to the result.
    """
    lib = load()
    code = _out_code(fmt)
    out_code = _out_code(out_dtype)
    P, M, N = _check_operands(lhs, lhs_scale, rhs, rhs_scale, dense_scale)
    flags = (FLAG_ALT_EMAX if alt_emax else 0) | (FLAG_DENSE_SCALE if dense_scale else 0)
    if M % 8:
        raise MXQError(3, "the result's rows M = %d must be a multiple of 8" % M)
    if data_out is None:
        data_out = torch.empty(data_shape(M, N, out_dtype), dtype=torch.uint8, device=lhs.device)
    if scale_out is None:
        scale_out = torch.empty(scale_image_shape(M, N, dense_scale), dtype=torch.uint8, device=lhs.device)
    _check_out_buffer("data_out", data_out, _data_nbytes(M, N, out_code), lhs.device)
    _check_out_buffer("scale_out", scale_out, _scale_nbytes(M, N, flags), lhs.device)
    sh = _stream_handle(stream, lhs.device)
    _check(_call_on(lhs.device, lib.mxq_scaled_matmul_quantize, lhs.data_ptr(), lhs_scale.data_ptr(),
                    rhs.data_ptr(), rhs_scale.data_ptr(), P, M, N, code, out_code, flags,
                    data_out.data_ptr(), scale_out.data_ptr(), sh))
    return data_out, scale_out


def axis_view_shape(R: int, C: int, dim: int):
    """(P, F) of the partition-major view that :func:`quantize_axis` writes
    for an R x C tensor: (K/4, 4*O) with K the block axis' extent."""
    d = dim + 2 if dim < 0 else dim
    if d not in (0, 1):
        raise MXQError(11, "quantize axis must be -1 or -2 (or 1, 0), got %r" % dim)
    K, O = (C, R) if d == 1 else (R, C)
    return K // 4, 4 * O


def quantize_axis(x: torch.Tensor, out_dtype: str = "e4m3fn", dim: int = -1, data_out: torch.Tensor | None = None,
                  scale_out: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None,
                  alt_emax: bool = False, dense_scale: bool = False):
    """Quantize a row-major [R, C] bf16/f16 device tensor with its 32-element
    blocks along ``dim`` (-1: along each row, -2: down each column).

    Returns ``(data, scale)`` in the layout :func:`quantize` produces for the
    partition-major [K/4, 4*O] view (K the block axis' extent, O the other):
    the operand layout of :func:`scaled_matmul`. Activations X [M, K] with
    ``dim=-1`` and weights W [K, N] with ``dim=-2`` make it compute X @ W.
    """
    lib = load()
    code = _out_code(out_dtype)
    if x.dtype not in IN_DTYPES:
        raise MXQError(1, "input must be bfloat16 or float16, got %s" % x.dtype)
    if x.dim() != 2 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous 2-D device tensor [R, C]")
    R, C = x.shape
    P, F = axis_view_shape(R, C, dim)
    flags = (FLAG_ALT_EMAX if alt_emax else 0) | (FLAG_DENSE_SCALE if dense_scale else 0)
    if data_out is None:
        data_out = torch.empty(data_shape(P, F, out_dtype), dtype=torch.uint8, device=x.device)
    if scale_out is None:
        scale_out = torch.empty(scale_image_shape(P, F, dense_scale), dtype=torch.uint8, device=x.device)
    _check_out_buffer("data_out", data_out, _data_nbytes(P, F, code), x.device)
    _check_out_buffer("scale_out", scale_out, _scale_nbytes(P, F, flags), x.device)
    sh = _stream_handle(stream, x.device)
    _check(_call_on(x.device, lib.mxq_quantize_axis, x.data_ptr(), R, C, IN_DTYPES[x.dtype], code, dim, flags,
                    data_out.data_ptr(), scale_out.data_ptr(), sh))
    return data_out, scale_out


# ---------------------------------------------------------------------------
# Mixture of experts
# ---------------------------------------------------------------------------
#
# The calls take no part in autograd: a result never requires a gradient, also
# where an argument does. Gradients are calls of their own (moe_combine_backward,
# the grouped product with the weights' dim -1 form, the _wgrad product and, for
# the gather, moe_combine without weights), for a torch.autograd.Function or by
# hand.

class MoEPlan(NamedTuple):
    """Where each (token, slot) pair goes when a batch is sorted by expert
    (int32 device tensors, see :func:`moe_sort`)."""

    offsets: torch.Tensor   # [experts + 1]: group e is sorted rows offsets[e] .. offsets[e + 1] - 1
    src: torch.Tensor       # [rows]: the pair t * slots + j of a sorted row, -1 without one
    dest: torch.Tensor      # [tokens, slots]: the sorted row of a pair, -1 without one


def _new(shape, dtype: torch.dtype, device: torch.device, stream) -> torch.Tensor:
    """An output or workspace for a kernel on ``stream``: allocated on that
    stream, so that neither its memory's earlier use nor its next one can
    overlap the kernel."""
    if stream is None:    # (extents as arguments of their own: 0.4 us less than as a tuple)
        return torch.empty(*shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=dtype, device=device)


# Tells autograd that a kernel has written to the caller's tensors (one, or a
# list), so that a backward pass that kept one of them from before raises, as
# after torch's own in-place operations.
_written = torch.autograd.graph.increment_version


def _check_tensor(name: str, t: torch.Tensor, shape, dtypes, device: torch.device | None = None) -> None:
    """A contiguous device tensor of this shape (an int: of that many
    dimensions) and one of these types, on ``device`` if given."""
    if t.is_cuda and (device is None or t.device == device) and t.dtype in dtypes and t.is_contiguous() and \
            (t.dim() == shape if type(shape) is int else t.shape == shape):
        return
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError("%s must be a device tensor%s" % (name, "" if device is None else " on %s" % device))
    if t.dtype not in dtypes:
        raise ValueError("%s must be %s, got %s" % (name, " or ".join(str(d) for d in dtypes), t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    raise ValueError("%s must %s, got shape %s" % (
        name, "have %d dimensions" % shape if type(shape) is int else "have shape %s" % (tuple(shape),),
        tuple(t.shape)))


_INT32 = (torch.int32,)
_IDS = (torch.int32, torch.int64)
_FLOAT32 = (torch.float32,)
_UINT8 = (torch.uint8,)
_IN = tuple(IN_DTYPES)
_ELEMS = tuple(ELEM_DTYPES)


def _elem_code(dtype: torch.dtype) -> int:
    try:
        return ELEM_DTYPES[dtype]
    except KeyError:
        raise MXQError(14, "element type must be bfloat16, float16 or float32, got %s" % dtype) from None


@functools.lru_cache(maxsize=256)
def _sort_sizes(tokens: int, slots: int, experts: int, align: int):
    """(rows, workspace bytes) of a sort."""
    return moe_rows(tokens, slots, experts, align), int(load().mxq_moe_sort_workspace_bytes(tokens, slots, experts))


@functools.lru_cache(maxsize=256)
def _gather_sizes(rows: int, K: int, out_dtype: str, dim: int, dense: bool):
    """(data shape, scale shape, data bytes, scale bytes) of a gathered quantize."""
    P, F = axis_view_shape(rows, K, dim)
    return (data_shape(P, F, out_dtype), scale_image_shape(P, F, dense), _data_nbytes(P, F, _out_code(out_dtype)),
            _scale_nbytes(P, F, FLAG_DENSE_SCALE if dense else 0))


def moe_rows(tokens: int, slots: int, experts: int, align: int = 32) -> int:
    """Sorted rows that hold any assignment of ``tokens * slots`` pairs to
    ``experts`` experts with groups aligned to ``align`` rows."""
    rows = int(load().mxq_moe_rows(tokens, slots, experts, align))
    if rows < 0:
        raise MXQError(12, "tokens %d, slots %d, experts %d, align %d" % (tokens, slots, experts, align))
    return rows


def moe_sort(experts: torch.Tensor, num_experts: int, align: int = 32,
             stream: torch.cuda.Stream | None = None) -> MoEPlan:
    """Sort the (token, slot) pairs of a batch by expert.

    ``experts`` [tokens, slots] int32 or int64 holds each pair's expert; a
    number outside 0 .. ``num_experts`` - 1 is a pair without a row here.
    Pairs keep their order within an expert, and every expert's group of rows
    starts at a multiple of ``align`` (a multiple of 4 up to 256; 32 where the
    weight gradients are to be computed). Nothing is copied to the host: the
    plan has :func:`moe_rows` rows, whatever the assignment.
    """
    lib = load()
    _check_tensor("experts", experts, 2, _IDS)
    T, k = experts.shape
    dev = experts.device
    rows, nws = _sort_sizes(T, k, num_experts, align)
    offsets = _new((num_experts + 1,), torch.int32, dev, stream)
    src = _new((rows,), torch.int32, dev, stream)
    dest = _new((T, k), torch.int32, dev, stream)
    ws = _new((nws,), torch.uint8, dev, stream) if nws else None
    _check(_call_on(dev, lib.mxq_moe_sort, experts.data_ptr(), experts.element_size(), T, k, num_experts, align,
                    offsets.data_ptr(), src.data_ptr(), dest.data_ptr(), ws.data_ptr() if nws else None,
                    _stream_handle(stream, dev)))
    return MoEPlan(offsets, src, dest)


def _check_plan(plan: MoEPlan, device: torch.device):
    """(rows, tokens, slots) of a plan on ``device``."""
    src, dest = plan.src, plan.dest
    _check_tensor("plan.src", src, 1, _INT32, device)
    _check_tensor("plan.dest", dest, 2, _INT32, device)
    return (*src.shape, *dest.shape)


def moe_gather_quantize(x: torch.Tensor, plan: MoEPlan, out_dtype: str = "e4m3fn", dim: int = -1,
                        data_out: torch.Tensor | None = None, scale_out: torch.Tensor | None = None,
                        stream: torch.cuda.Stream | None = None, alt_emax: bool = False, dense_scale: bool = True):
    """Gather the rows of ``x`` [tokens, K] (bf16/f16) into sorted order and
    quantize them.

    Returns the ``(data, scale)`` that :func:`quantize_axis` with ``dim`` gives
    for the [rows, K] tensor whose row r is the row of ``x`` that
    ``plan.src[r]`` names, or zeros: with ``dim=-1`` the left operand of
    :func:`grouped_scaled_matmul`, with ``dim=-2`` an operand of
    :func:`grouped_scaled_matmul_wgrad`. Scales are dense by default, as the
    grouped products read them.
    """
    lib = load()
    code = _out_code(out_dtype)
    if x.dtype not in IN_DTYPES:
        raise MXQError(1, "input must be bfloat16 or float16, got %s" % x.dtype)
    _check_tensor("x", x, 2, _IN)
    dev = x.device
    rows, T, k = _check_plan(plan, dev)
    n, K = x.shape
    if n != T:
        raise ValueError("x has %d rows, the plan %d tokens" % (n, T))
    dshape, sshape, dbytes, sbytes = _gather_sizes(rows, K, out_dtype, dim, dense_scale)
    flags = (FLAG_ALT_EMAX if alt_emax else 0) | (FLAG_DENSE_SCALE if dense_scale else 0)
    if data_out is None:
        data_out = _new(dshape, torch.uint8, dev, stream)
    else:
        _check_out_buffer("data_out", data_out, dbytes, dev)
    if scale_out is None:
        scale_out = _new(sshape, torch.uint8, dev, stream)
    else:
        _check_out_buffer("scale_out", scale_out, sbytes, dev)
    _check(_call_on(dev, lib.mxq_moe_gather_quantize, x.data_ptr(), T, k, K, IN_DTYPES[x.dtype], code, dim, flags,
                    plan.src.data_ptr(), rows, data_out.data_ptr(), scale_out.data_ptr(), _stream_handle(stream, dev)))
    return data_out, scale_out


def moe_combine(y: torch.Tensor, plan: MoEPlan, weights: torch.Tensor | None = None,
                out: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Bring sorted rows back to token order: out[t] = sum over j of
    weights[t, j] * y[dest[t, j]], added in float32 in slot order.

    ``y`` [rows, N] is bf16, f16 or f32, ``weights`` [tokens, slots] float32
    (None: all 1, the gradient of the gather). A pair without a row adds
    nothing. Returns [tokens, N] of y's type.
    """
    lib = load()
    code = _elem_code(y.dtype)
    _check_tensor("y", y, 2, _ELEMS)
    dev = y.device
    rows, T, k = _check_plan(plan, dev)
    n, N = y.shape
    if n != rows:
        raise ValueError("y has %d rows, the plan %d" % (n, rows))
    if weights is not None:
        _check_tensor("weights", weights, (T, k), _FLOAT32, dev)
    given = out is not None
    if not given:
        out = _new((T, N), y.dtype, dev, stream)
    else:
        _check_tensor("out", out, (T, N), (y.dtype,), dev)
    _check(_call_on(dev, lib.mxq_moe_combine, y.data_ptr(), rows, N, code, plan.dest.data_ptr(),
                    None if weights is None else weights.data_ptr(), T, k, out.data_ptr(),
                    _stream_handle(stream, dev)))
    if given:
        _written(out)
    return out


def moe_combine_backward(grad: torch.Tensor, y: torch.Tensor, plan: MoEPlan, weights: torch.Tensor,
                         grad_y: torch.Tensor | None = None, grad_weights: torch.Tensor | None = None,
                         stream: torch.cuda.Stream | None = None):
    """The gradients ``(grad_y, grad_weights)`` of :func:`moe_combine` with
    weights, given the gradient ``grad`` [tokens, N] of its result.

    grad_y [rows, N] (y's type) is zero in the rows without a pair,
    grad_weights [tokens, slots] (float32) for the pairs without a row. (The
    gradient of the unweighted combine is the gather of its rows;
    :func:`moe_gather_quantize` gives it quantized, as the products before it
    read it. There is no call that gathers without quantizing.)
    """
    lib = load()
    code = _elem_code(y.dtype)
    _check_tensor("y", y, 2, _ELEMS)
    dev = y.device
    rows, T, k = _check_plan(plan, dev)
    n, N = y.shape
    if n != rows:
        raise ValueError("y has %d rows, the plan %d" % (n, rows))
    _check_tensor("grad", grad, (T, N), (y.dtype,), dev)
    _check_tensor("weights", weights, (T, k), _FLOAT32, dev)
    given = [t for t in (grad_y, grad_weights) if t is not None]
    if grad_y is None:
        grad_y = _new((rows, N), y.dtype, dev, stream)
    else:
        _check_tensor("grad_y", grad_y, (rows, N), (y.dtype,), dev)
    if grad_weights is None:
        grad_weights = _new((T, k), torch.float32, dev, stream)
    else:
        _check_tensor("grad_weights", grad_weights, (T, k), _FLOAT32, dev)
    _check(_call_on(dev, lib.mxq_moe_combine_backward, grad.data_ptr(), y.data_ptr(), rows, N, code,
                    plan.src.data_ptr(), plan.dest.data_ptr(), weights.data_ptr(), T, k, grad_y.data_ptr(),
                    grad_weights.data_ptr(), _stream_handle(stream, dev)))
    if given:
        _written(given)
    return grad_y, grad_weights


def grouped_scaled_matmul(lhs: torch.Tensor, lhs_scale: torch.Tensor, rhs: torch.Tensor, rhs_scale: torch.Tensor,
                          offsets: torch.Tensor, fmt: str = "e4m3fn", res_dtype: torch.dtype = torch.bfloat16,
                          out: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The experts' products: out[r] = X[r] @ W_g for the sorted rows r of
    group g, zeros for the rows of no group (past the last one; before the first
    where ``offsets[0]`` is above 0).

    ``lhs`` [P, 4 rows] with dense scales [P/8, rows] are the sorted rows
    quantized along K = 4P (:func:`moe_gather_quantize`, or
    :func:`quantize_axis` with ``dim=-1, dense_scale=True``); ``rhs``
    [groups, P, 4N] with [groups, P/8, N] the experts' weights [K, N], each
    quantized with ``dim=-2`` (for the gradient of the input: the weights with
    ``dim=-1``); ``offsets`` [groups + 1] from :func:`moe_sort`. Returns
    [rows, N] float32 or bfloat16. Groups and arithmetic as in
    :func:`scaled_matmul`.
    """
    lib = load()
    code = _out_code(fmt)
    if res_dtype not in RES_DTYPES:
        raise MXQError(10, "result type must be float32 or bfloat16, got %s" % res_dtype)
    _check_tensor("lhs", lhs, 2, _UINT8)
    dev = lhs.device
    _check_tensor("rhs", rhs, 3, _UINT8, dev)
    P, M4 = lhs.shape
    G, P2, N4 = rhs.shape
    if P2 != P or M4 % 4 or N4 % 4 or P % 8:
        raise ValueError("lhs [P, 4 rows] and rhs [groups, P, 4 N] must share P, a multiple of 8")
    M, N = M4 // 4, N4 // 4
    _check_tensor("lhs_scale", lhs_scale, (P // 8, M), _UINT8, dev)
    _check_tensor("rhs_scale", rhs_scale, (G, P // 8, N), _UINT8, dev)
    _check_tensor("offsets", offsets, (G + 1,), _INT32, dev)
    given = out is not None
    if not given:
        out = _new((M, N), res_dtype, dev, stream)
    else:
        _check_tensor("out", out, (M, N), (res_dtype,), dev)
    _check(_call_on(dev, lib.mxq_grouped_matmul, lhs.data_ptr(), lhs_scale.data_ptr(), rhs.data_ptr(),
                    rhs_scale.data_ptr(), offsets.data_ptr(), G, P, M, N, code, RES_DTYPES[res_dtype], out.data_ptr(),
                    _stream_handle(stream, dev)))
    if given:
        _written(out)
    return out


def grouped_scaled_matmul_wgrad(lhs: torch.Tensor, lhs_scale: torch.Tensor, rhs: torch.Tensor,
                                rhs_scale: torch.Tensor, offsets: torch.Tensor, fmt: str = "e4m3fn",
                                res_dtype: torch.dtype = torch.bfloat16, out: torch.Tensor | None = None,
                                stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The gradient of the experts' weights: out[g] = X_g^T @ dY_g over the
    sorted rows of group g, zeros for an empty group.

    ``lhs`` [P, 4M] and ``rhs`` [P, 4N] with dense scales [P/8, M] and
    [P/8, N] are the 4P sorted rows of the forward input [rows, M] and of the
    result's gradient [rows, N], quantized with ``dim=-2``; the groups in
    ``offsets`` [groups + 1] start at multiples of 32. Returns [groups, M, N].
    """
    lib = load()
    code = _out_code(fmt)
    if res_dtype not in RES_DTYPES:
        raise MXQError(10, "result type must be float32 or bfloat16, got %s" % res_dtype)
    P, M, N = _check_operands(lhs, lhs_scale, rhs, rhs_scale, True)
    dev = lhs.device
    _check_tensor("offsets", offsets, 1, _INT32, dev)
    G = offsets.shape[0] - 1
    given = out is not None
    if not given:
        out = _new((max(G, 0), M, N), res_dtype, dev, stream)
    else:
        _check_tensor("out", out, (G, M, N), (res_dtype,), dev)
    _check(_call_on(dev, lib.mxq_grouped_matmul_wgrad, lhs.data_ptr(), lhs_scale.data_ptr(), rhs.data_ptr(),
                    rhs_scale.data_ptr(), offsets.data_ptr(), G, P, M, N, code, RES_DTYPES[res_dtype], out.data_ptr(),
                    _stream_handle(stream, dev)))
    if given:
        _written(out)
    return out


# ---------------------------------------------------------------------------
# Gradient norm and clipping
# ---------------------------------------------------------------------------

def _check_tensors(name, tensors, device):
    """Contiguous device tensors of element types, as (addresses, elements,
    type codes). A list may hold hundreds: one pass per property, each at the
    interpreter's C speed."""
    T = torch.Tensor
    codes = list(map(ELEM_DTYPES.get, [t.dtype for t in tensors]))
    if None in codes or not all(map(T.is_contiguous, tensors)) or set(map(T.get_device, tensors)) != {device.index}:
        for t in tensors:
            _check_tensor(name, t, t.dim(), _ELEMS, device)
    return list(map(T.data_ptr, tensors)), list(map(T.numel, tensors)), codes


def _c_array(typecode: str, values):
    a = array.array(typecode, values)
    return a, a.buffer_info()[0]    # (the array keeps the memory)


def _norm_call(grads, max_norm, outs, stream):
    lib = load()
    if not grads:
        raise ValueError("no tensors")
    dev = grads[0].device
    if dev.type != "cuda":
        raise ValueError("grads must be device tensors")
    ptrs, numels, codes = _check_tensors("grads", grads, dev)
    if outs is None:
        optrs = None
    elif outs is grads:
        optrs = ptrs
    else:
        optrs, onumels, ocodes = _check_tensors("out", outs, dev)
        if ocodes != codes or onumels != numels:
            raise ValueError("out must hold a tensor of each gradient's size and type")
    n = len(grads)
    # the workgroups of a tensor listed twice would each scale what the others have
    # scaled or not (a tensor without elements has no address of its own)
    if optrs is not None and len(set(optrs)) != n:
        some = [p for p, e in zip(optrs, numels) if e]
        if len(set(some)) != len(some):
            raise ValueError("the tensors that are scaled must not share memory")
    pa, pp = _c_array("Q", ptrs)
    oa, op = (None, None) if optrs is None else (pa, pp) if optrs is ptrs else _c_array("Q", optrs)
    na, np_ = _c_array("q", numels)
    ca, cp = _c_array("i", codes)
    norm = _new(((),), torch.float32, dev, stream)
    ws = _new((lib.mxq_clip_grad_norm_workspace_bytes(np_, cp, n),), torch.uint8, dev, stream)
    _check(_call_on(dev, lib.mxq_clip_grad_norm, pp, op, np_, cp, n, max_norm, norm.data_ptr(), ws.data_ptr(),
                    _stream_handle(stream, dev)))
    if outs is not None:
        _written(outs)
    return norm


def grad_norm(grads, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """The norm of all elements of all tensors (bf16, f16 or f32, mixed), as a
    float32 device scalar; the squares are added in 64 bits."""
    return _norm_call(list(grads), 0.0, None, stream)


def clip_grad_norm(grads, max_norm: float, out=None, stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Scale contiguous device tensors by max_norm / norm where their global
    norm is finite and above ``max_norm``; return the norm (before scaling, a
    float32 device scalar).

    The tensors (bf16, f16 or f32, mixed) are scaled in place, or into the
    tensors of ``out``; those must not share memory with each other (one
    gradient of several layers is listed once). A norm that is not finite leaves the values as they
    are. Nothing is copied to the host.
    """
    if not max_norm >= 0.0:
        raise MXQError(15, "max_norm must not be negative or NaN, got %r" % (max_norm,))
    grads = list(grads)
    return _norm_call(grads, float(max_norm), grads if out is None else list(out), stream)
