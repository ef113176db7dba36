"""The 8-bit floating-point operators on torch tensors (C ABI: include/gemm_fp8.h).

An 8-bit matrix is two tensors: ``data`` (rows x cols, ``torch.float8_e4m3fn``
or ``torch.float8_e5m2``, rows a multiple of 16 bytes apart) and ``scales``
(float32, one for each 128 columns of each row, or of each 128 rows:
``[rows or ceil(rows / 128), ceil(cols / 128)]``, in any strides).  Which of the
two it is follows from the scales' shape.  The value of element (r, c) is
``data[r, c] * scales[r or r // 128, c // 128]``.

Everything runs on the current stream of the tensors' device (or ``stream``);
this module allocates outputs and passes pointers, and a failing call raises
``GemmError``.
"""
import ctypes
import functools
import struct

import torch

from . import _binding
from ._binding import GP_OK, FP8_FORMATS, GemmError, GpFp8Options, GpPlan, fp8_calls, lib

GROUP = 128

_FORMAT_OF = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}
_FP8_DTYPE = (torch.float8_e4m3fn, torch.float8_e5m2)
_REAL_OF = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}
_F32 = torch.float32

# The calls below are short (a few microseconds on the GPU at the smallest
# sizes), so this module counts its own steps: one allocation per output,
# descriptors packed as bytes, no views.
_pack = struct.Struct("PPqqqii").pack       # gp_fp8_matrix
_empty = torch.empty_strided
_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _check(rc, where):
    if rc != GP_OK:
        raise GemmError(rc, where)


class _On:
    """The tensors' device and the call's stream made current, so that outputs are allocated for that stream."""
    __slots__ = ("device", "stream", "before", "other")

    def __init__(self, device, stream):
        self.device, self.stream, self.before, self.other = device, stream, None, None

    def __enter__(self):
        now = torch.cuda.current_device()
        if now != self.device:
            self.before = now
            torch.cuda.set_device(self.device)
        s = self.stream
        if s is not None:
            if not isinstance(s, torch.cuda.Stream):
                s = torch.cuda.ExternalStream(s, self.device) if s else torch.cuda.default_stream(self.device)
            self.other = torch.cuda.stream(s)
            self.other.__enter__()

    def __exit__(self, *exc):
        if self.other is not None:
            self.other.__exit__(*exc)
        if self.before is not None:
            torch.cuda.set_device(self.before)
        return False


def _elsewhere(x, name, stream):
    """Whether the call has to change the current device or stream first."""
    device = x.get_device()
    if device < 0:
        raise ValueError("%s must be on a CUDA device" % name)
    return stream is not None or device != _device()


def _matrix(x, name):
    """Shape of a 2-D CUDA tensor whose rows are contiguous, and its row stride."""
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("%s must have two dimensions, got %d" % (name, len(shape)))
    if not x.is_cuda:
        raise ValueError("%s must be on a CUDA device" % name)
    rows, cols = shape
    ld, inner = x.stride()
    if inner != 1 and cols > 1:
        raise ValueError("%s must have contiguous rows (stride 1 along the last dimension)" % name)
    return rows, cols, (ld if rows > 1 or ld > cols else cols)


def _real(x, name):
    t = _REAL_OF.get(x.dtype)
    if t is None:
        raise ValueError("%s must be float16, bfloat16 or float32, got %s" % (name, x.dtype))
    return t


def _same(x, like, name):
    if x.shape != like.shape or x.dtype != like.dtype or x.get_device() != like.get_device():
        raise ValueError("%s must have the shape, type and device of the other operand: got %s %s %s, want %s %s %s" % (
            name, tuple(x.shape), x.dtype, x.device, tuple(like.shape), like.dtype, like.device))


def _fp8(data, scales, name):
    """(rows, cols, descriptor) of an 8-bit matrix."""
    fmt = _FORMAT_OF.get(data.dtype)
    if fmt is None:
        raise ValueError("%s must be float8_e4m3fn or float8_e5m2, got %s" % (name, data.dtype))
    rows, cols, ld = _matrix(data, name)
    if rows <= 1:
        ld = (ld + 15) // 16 * 16      # the stride of a single row is never used
    if scales.dtype is not _F32 or len(scales.shape) != 2 or scales.get_device() != data.get_device():
        raise ValueError("the scales of %s must be a float32 matrix on its device" % name)
    groups, blocks = scales.shape
    if blocks != (cols + 127) // 128 or (groups != rows and groups != (rows + 127) // 128):
        raise ValueError("the scales of %s have shape %s: want (%d or %d, %d)" % (
            name, (groups, blocks), rows, (rows + 127) // 128, (cols + 127) // 128))
    sr, sc = scales.stride()
    return rows, cols, _pack(data.data_ptr(), scales.data_ptr(), ld, sr, sc, fmt, 1 if groups == rows else GROUP)


def _new_fp8(rows, cols, fmt, group, device):
    """An 8-bit matrix to be written: rows 16 bytes aligned, the scales of one group of columns side by side."""
    ld = (cols + 15) // 16 * 16
    data = _empty((rows, cols), (ld, 1), dtype=_FP8_DTYPE[fmt], device=device)
    groups = rows if group == 1 else (rows + 127) // 128
    scales = _empty((groups, (cols + 127) // 128), (1, groups or 1), dtype=_F32, device=device)
    return data, scales, _pack(data.data_ptr(), scales.data_ptr(), ld, 1, groups, fmt, group)


def _group(scales):
    """Rows that share a scale."""
    if scales == "rows":
        return 1
    if scales == "blocks":
        return GROUP
    raise ValueError("unknown scales %r" % (scales,))


def quantize_fp8(x, scales="rows", *, format="e4m3", transpose=False, stream=None):
    """x (rows x cols; float16, bfloat16 or float32) to 8 bits.

    ``scales``: "rows" (one scale for each row's 128 values: activations,
    gradients) or "blocks" (one for each 128 x 128 block: weights).
    ``transpose``: True also returns the 8-bit matrix of the transpose,
    quantised along x's columns, from the same pass over x; "only" returns that
    alone.  ``format``: "e4m3" or "e5m2".

    Returns (data, scales), or (data, scales, data_t, scales_t).
    """
    if _elsewhere(x, "x", stream):
        with _On(x.get_device(), stream):
            return quantize_fp8(x, scales, format=format, transpose=transpose)
    rows, cols, ld = _matrix(x, "x")
    real = _real(x, "x")
    group = _group(scales)
    if transpose not in (False, True, "only"):
        raise ValueError("unknown transpose %r" % (transpose,))
    fmt = _binding._enum(format, FP8_FORMATS, "format")
    device = x.device
    out, q, qt = (), None, None
    if transpose != "only":
        data, s, q = _new_fp8(rows, cols, fmt, group, device)
        out = (data, s)
    if transpose:
        data, s, qt = _new_fp8(cols, rows, fmt, group, device)
        out += (data, s)
    _check(fp8_calls().quantize(x.data_ptr(), ld, rows, cols, real, q, qt, _raw_stream(x.get_device())), "fp8_quantize")
    return out


def dequantize_fp8(data, scales, dtype=torch.float32):
    """The values of an 8-bit matrix (elementary torch operations, on any device: for checks and inspection)."""
    rows, cols = data.shape
    group = 1 if scales.shape[0] == rows else GROUP
    wide = scales.to(dtype).repeat_interleave(group, 0)[:rows].repeat_interleave(GROUP, 1)[:, :cols]
    return data.to(dtype) * wide


def gemm_fp8(A, A_scales, B, B_scales, *, out_dtype=None, addend=None, out=None, stream=None, bn=0,
             no_split=False, timeout_ns=0, inject_lost_load=False):
    """C = A x B^T (+ addend) of two 8-bit matrices, A: M x K, B: N x K.

    The three products of a linear layer y = x W^T are
    ``gemm_fp8(x, W)``, ``gemm_fp8(dy, W^T)`` and ``gemm_fp8(dy^T, x^T, addend=dW)``
    on what ``quantize_fp8`` gives.  ``out``: where to write (M x N, rows
    contiguous); ``out_dtype``: the type of a new output (bfloat16 where neither
    is given), or out's own.  ``addend``: an M x N tensor of the output's type
    added in FP32 before the rounding; it may be ``out`` itself.  ``bn``, ``no_split``, ``timeout_ns``,
    ``inject_lost_load``: see gp_fp8_options.
    """
    if _elsewhere(A, "A", stream):
        with _On(A.get_device(), stream):
            return gemm_fp8(A, A_scales, B, B_scales, out_dtype=out_dtype, addend=addend, out=out, bn=bn,
                            no_split=no_split, timeout_ns=timeout_ns, inject_lost_load=inject_lost_load)
    M, K, a = _fp8(A, A_scales, "A")
    N, kb, b = _fp8(B, B_scales, "B")
    if kb != K:
        raise ValueError("A has %d columns and B %d" % (K, kb))
    if B.get_device() != A.get_device():
        raise ValueError("A is on %s and B on %s" % (A.device, B.device))
    if out is None:
        out = _empty((M, N), (N, 1), dtype=torch.bfloat16 if out_dtype is None else out_dtype, device=A.device)
        ldc = N
    else:
        if out_dtype is not None and out.dtype is not out_dtype:
            raise ValueError("out is %s: out_dtype %s asks for another type" % (out.dtype, out_dtype))
        rows, cols, ldc = _matrix(out, "out")
        if (rows, cols) != (M, N) or out.get_device() != A.get_device():
            raise ValueError("out has shape %s on %s: want %s on %s" % ((rows, cols), out.device, (M, N), A.device))
    real = _real(out, "out")
    add_ptr, ld_add = None, 0
    if addend is not None:
        _same(addend, out, "addend")
        ld_add = _matrix(addend, "addend")[2]
        add_ptr = addend.data_ptr()
    opts = None
    if bn or no_split or timeout_ns or inject_lost_load:
        opts = GpFp8Options(int(timeout_ns), int(bn), int(no_split), int(inject_lost_load))
    _check(fp8_calls().gemm(a, b, out.data_ptr(), ldc, add_ptr, ld_add, M, N, K, real, _raw_stream(A.get_device()), opts),
           "gemm_fp8")
    return out


def gemm_fp8_plan(M, N, K, A_scales="rows", B_scales="blocks", *, sms=0, bn=0, no_split=False) -> dict:
    """The tile, ring and split that gemm_fp8 would choose (see gemm_fp8_plan in the C header)."""
    p = GpPlan()
    opts = GpFp8Options(0, int(bn), int(no_split), 0)
    _check(lib().gemm_fp8_plan(M, N, K, _group(A_scales), _group(B_scales), sms, opts, p), "gemm_fp8_plan")
    return p.as_dict()


def rmsnorm_fp8(x, weight, residual=None, *, eps=1e-6, format="e4m3", normed=False, stream=None):
    """Residual addition, RMS norm and quantisation in one pass.

    h = x + residual (rounded to x's type), rstd = 1 / sqrt(mean(h^2) + eps),
    y = h * rstd * weight, and y in 8 bits with a scale for each row's 128 values.
    Returns (data, scales, h, rstd), and y rounded to x's type as a fifth with
    ``normed``.  Without a residual h is x itself.  Without columns rstd is NaN.
    """
    if _elsewhere(x, "x", stream):
        with _On(x.get_device(), stream):
            return rmsnorm_fp8(x, weight, residual, eps=eps, format=format, normed=normed)
    rows, cols, ld = _matrix(x, "x")
    real = _real(x, "x")
    wtype = _weight(weight, cols, x)
    fmt = _binding._enum(format, FP8_FORMATS, "format")
    device = x.device
    h, res_ptr, ld_res, h_ptr, y_ptr = x, None, 0, None, None
    if residual is not None:
        _same(residual, x, "residual")
        ld_res = _matrix(residual, "residual")[2]
        res_ptr = residual.data_ptr()
        h = _empty((rows, cols), (cols, 1), dtype=x.dtype, device=device)
        h_ptr = h.data_ptr()
    data, scales, q = _new_fp8(rows, cols, fmt, 1, device)
    rstd = _empty((rows,), (1,), dtype=_F32, device=device)
    out = (data, scales, h, rstd)
    if normed:
        y = _empty((rows, cols), (cols, 1), dtype=x.dtype, device=device)
        y_ptr = y.data_ptr()
        out += (y,)
    _check(fp8_calls().rmsnorm(x.data_ptr(), ld, res_ptr, ld_res, weight.data_ptr(), wtype, eps, rows, cols, real, h_ptr,
                               cols, rstd.data_ptr(), y_ptr, cols, q, _raw_stream(x.get_device())), "fp8_rmsnorm")
    return out


def rmsnorm_backward(dy, h, weight, rstd, dresidual=None, *, weight_grad=True, stream=None):
    """Gradient of the norm: (dx, dweight) from the gradient of y and the stored h and rstd.

    dx, of h's type, is the gradient of both x and the residual; ``dresidual``
    (the gradient that reaches h past the norm) is added to it.  dweight is
    float32, or None with ``weight_grad=False``.
    """
    if _elsewhere(dy, "dy", stream):
        with _On(dy.get_device(), stream):
            return rmsnorm_backward(dy, h, weight, rstd, dresidual, weight_grad=weight_grad)
    rows, cols, ld_dy = _matrix(dy, "dy")
    real = _real(dy, "dy")
    _same(h, dy, "h")
    ld_h = _matrix(h, "h")[2]
    wtype = _weight(weight, cols, dy)
    if rstd.dtype is not _F32 or rstd.shape != (rows,) or rstd.get_device() != dy.get_device() or (
            rows > 1 and rstd.stride(0) != 1):
        raise ValueError("rstd must be %d contiguous float32 values on %s" % (rows, dy.device))
    res_ptr, ld_res = None, 0
    if dresidual is not None:
        _same(dresidual, dy, "dresidual")
        ld_res = _matrix(dresidual, "dresidual")[2]
        res_ptr = dresidual.data_ptr()
    device = dy.device
    dx = _empty((rows, cols), (cols, 1), dtype=dy.dtype, device=device)
    dw, dw_ptr, work_ptr, work_bytes = None, None, None, 0
    if weight_grad:
        dw = _empty((cols,), (1,), dtype=_F32, device=device)
        dw_ptr = dw.data_ptr()
        work_bytes = _backward_workspace(rows, cols, dy.get_device())
        if work_bytes:
            work = _empty((work_bytes // 4,), (1,), dtype=_F32, device=device)   # (freed in the call's stream order)
            work_ptr = work.data_ptr()
    _check(fp8_calls().backward(dy.data_ptr(), ld_dy, h.data_ptr(), ld_h, res_ptr, ld_res, weight.data_ptr(), wtype,
                                rstd.data_ptr(), rows, cols, real, dx.data_ptr(), cols,
                                dw_ptr, work_ptr, work_bytes, _raw_stream(dy.get_device())),
           "fp8_rmsnorm_backward")
    return dx, dw


@functools.lru_cache(maxsize=256)
def _backward_workspace(rows, cols, device):
    """Bytes that rmsnorm_backward needs for the weight's gradient on `device`, the current one."""
    size = ctypes.c_int64()
    _check(lib().fp8_rmsnorm_backward_workspace(rows, cols, 0, size), "fp8_rmsnorm_backward_workspace")
    return size.value


def _weight(weight, cols, like):
    if weight.shape != (cols,) or weight.get_device() != like.get_device() or (cols > 1 and weight.stride(0) != 1):
        raise ValueError("weight must be %d contiguous values on %s" % (cols, like.device))
    return _real(weight, "weight")
