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

import torch

from . import _binding
from ._binding import GP_OK, FP8_FORMATS, GemmError, GpFp8Matrix, GpFp8Options, GpPlan, lib

GROUP = 128

_FORMAT_OF = {torch.float8_e4m3fn: 0, torch.float8_e5m2: 1}
_FP8_DTYPE = (torch.float8_e4m3fn, torch.float8_e5m2)
_REAL_OF = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


def _check(rc, where):
    if rc != GP_OK:
        raise GemmError(rc, where)


class _On:
    """The tensors' device and the call's stream made current, so that outputs are allocated for that stream."""
    __slots__ = ("device", "stream", "before", "other")

    def __init__(self, device, stream):
        self.device, self.stream, self.before, self.other = device.index, stream, None, None

    def __enter__(self):
        now = torch.cuda.current_device()
        if now != self.device:
            self.before = now
            torch.cuda.set_device(self.device)
        if self.stream is None:
            return torch._C._cuda_getCurrentRawStream(self.device)
        s = self.stream
        if not isinstance(s, torch.cuda.Stream):
            s = torch.cuda.ExternalStream(s, self.device) if s else torch.cuda.default_stream(self.device)
        self.other = torch.cuda.stream(s)
        self.other.__enter__()
        return s.cuda_stream

    def __exit__(self, *exc):
        if self.other is not None:
            self.other.__exit__(*exc)
        if self.before is not None:
            torch.cuda.set_device(self.before)
        return False


def _matrix(x, name):
    """Shape of a 2-D CUDA tensor whose rows are contiguous, and its row stride."""
    if x.dim() != 2:
        raise ValueError("%s must have two dimensions, got %d" % (name, x.dim()))
    if not x.is_cuda:
        raise ValueError("%s must be on a CUDA device" % name)
    rows, cols = x.shape
    ld, inner = x.stride()
    if inner != 1 and cols > 1:
        raise ValueError("%s must have contiguous rows (stride 1 along the last dimension)" % name)
    return rows, cols, (ld if rows > 1 else max(ld, cols))


def _real(x, name):
    t = _REAL_OF.get(x.dtype)
    if t is None:
        raise ValueError("%s must be float16, bfloat16 or float32, got %s" % (name, x.dtype))
    return t


def _same(x, like, name):
    if x.shape != like.shape or x.dtype != like.dtype or x.device != like.device:
        raise ValueError("%s must have the shape, type and device of the other operand: got %s %s %s, want %s %s %s" % (
            name, tuple(x.shape), x.dtype, x.device, tuple(like.shape), like.dtype, like.device))


def _fp8(data, scales, name):
    """(rows, cols, descriptor) of an 8-bit matrix."""
    fmt = _FORMAT_OF.get(data.dtype)
    if fmt is None:
        raise ValueError("%s must be float8_e4m3fn or float8_e5m2, got %s" % (name, data.dtype))
    rows, cols, ld = _matrix(data, name)
    if rows <= 1:
        ld = -(-ld // 16) * 16         # the stride of a single row is never used
    if scales.dtype != torch.float32 or scales.dim() != 2 or scales.device != data.device:
        raise ValueError("the scales of %s must be a float32 matrix on its device" % name)
    groups, blocks = scales.shape
    if blocks != -(-cols // GROUP) or groups not in (rows, -(-rows // GROUP)):
        raise ValueError("the scales of %s have shape %s: want (%d or %d, %d)" % (
            name, (groups, blocks), rows, -(-rows // GROUP), -(-cols // GROUP)))
    sr, sc = scales.stride()
    return rows, cols, GpFp8Matrix(data.data_ptr(), scales.data_ptr(), ld, sr, sc, fmt, 1 if groups == rows else GROUP)


def _new_fp8(rows, cols, fmt, group, device):
    """An 8-bit matrix to be written: rows 16 bytes aligned, the scales of one group of columns side by side."""
    ld = -(-cols // 16) * 16
    data = torch.empty((rows, ld), dtype=_FP8_DTYPE[fmt], device=device)
    if ld != cols:
        data = data[:, :cols]
    groups = rows if group == 1 else -(-rows // GROUP)
    blocks = -(-cols // GROUP)
    scales = torch.empty((blocks, groups), dtype=torch.float32, device=device).t()
    return data, scales, GpFp8Matrix(data.data_ptr(), scales.data_ptr(), ld, 1, groups, fmt, group)


def quantize_fp8(x, scales="rows", *, format="e4m3", transpose=False, stream=None):
    """x (rows x cols; float16, bfloat16 or float32) to 8 bits.

    ``scales``: "rows" (one scale for each row's 128 values: activations,
    gradients) or "blocks" (one for each 128 x 128 block: weights).
    ``transpose``: True also returns the 8-bit matrix of the transpose,
    quantised along x's columns, from the same pass over x; "only" returns that
    alone.  ``format``: "e4m3" or "e5m2".

    Returns (data, scales), or (data, scales, data_t, scales_t).
    """
    rows, cols, ld = _matrix(x, "x")
    real = _real(x, "x")
    if scales not in ("rows", "blocks"):
        raise ValueError("unknown scales %r" % (scales,))
    if transpose not in (False, True, "only"):
        raise ValueError("unknown transpose %r" % (transpose,))
    fmt = _binding._enum(format, FP8_FORMATS, "format")
    group = 1 if scales == "rows" else GROUP
    out, q, qt = (), None, None
    with _On(x.device, stream) as st:
        if transpose != "only":
            data, s, q = _new_fp8(rows, cols, fmt, group, x.device)
            out = (data, s)
        if transpose:
            data, s, qt = _new_fp8(cols, rows, fmt, group, x.device)
            out += (data, s)
        _check(lib().fp8_quantize(x.data_ptr(), ld, rows, cols, real, q, qt, st), "fp8_quantize")
    return out


def dequantize_fp8(data, scales, dtype=torch.float32):
    """The values of an 8-bit matrix (elementary torch operations, on any device: for checks and inspection)."""
    rows, cols = data.shape
    group = 1 if scales.shape[0] == rows else GROUP
    wide = scales.to(dtype).repeat_interleave(group, 0)[:rows].repeat_interleave(GROUP, 1)[:, :cols]
    return data.to(dtype) * wide


def gemm_fp8(A, A_scales, B, B_scales, *, out_dtype=torch.bfloat16, addend=None, out=None, stream=None, bn=0,
             no_split=False, timeout_ns=0, inject_lost_load=False):
    """C = A x B^T (+ addend) of two 8-bit matrices, A: M x K, B: N x K.

    The three products of a linear layer y = x W^T are
    ``gemm_fp8(x, W)``, ``gemm_fp8(dy, W^T)`` and ``gemm_fp8(dy^T, x^T, addend=dW)``
    on what ``quantize_fp8`` gives.  ``addend``: an M x N tensor of ``out_dtype``
    added in FP32 before the rounding; it may be ``out`` itself.  ``out``: where
    to write (M x N, rows contiguous).  ``bn``, ``no_split``, ``timeout_ns``,
    ``inject_lost_load``: see gp_fp8_options.
    """
    M, K, a = _fp8(A, A_scales, "A")
    N, kb, b = _fp8(B, B_scales, "B")
    if kb != K:
        raise ValueError("A has %d columns and B %d" % (K, kb))
    if B.device != A.device:
        raise ValueError("A is on %s and B on %s" % (A.device, B.device))
    opts = None
    if bn or no_split or timeout_ns or inject_lost_load:
        opts = GpFp8Options(int(timeout_ns), int(bn), int(no_split), int(inject_lost_load))
    with _On(A.device, stream) as st:
        if out is None:
            out = torch.empty((M, N), dtype=out_dtype, device=A.device)
            ldc = N
        else:
            rows, cols, ldc = _matrix(out, "out")
            if (rows, cols) != (M, N) or out.device != A.device:
                raise ValueError("out has shape %s on %s: want %s on %s" % ((rows, cols), out.device, (M, N), A.device))
        real = _real(out, "out")
        add_ptr, ld_add = None, 0
        if addend is not None:
            _same(addend, out, "addend")
            ld_add = _matrix(addend, "addend")[2]
            add_ptr = addend.data_ptr()
        _check(lib().gemm_fp8(a, b, out.data_ptr(), ldc, add_ptr, ld_add, M, N, K, real, st, opts), "gemm_fp8")
    return out


def gemm_fp8_plan(M, N, K, A_scales="rows", B_scales="blocks", *, sms=0, bn=0, no_split=False) -> dict:
    """The tile, ring and split that gemm_fp8 would choose (see gemm_fp8_plan in the C header)."""
    group = {"rows": 1, "blocks": GROUP}
    p = GpPlan()
    opts = GpFp8Options(0, int(bn), int(no_split), 0)
    _check(lib().gemm_fp8_plan(M, N, K, group[A_scales], group[B_scales], sms, opts, p), "gemm_fp8_plan")
    return p.as_dict()


def rmsnorm_fp8(x, weight, residual=None, *, eps=1e-6, format="e4m3", normed=False, stream=None):
    """Residual addition, RMS norm and quantisation in one pass.

    h = x + residual (rounded to x's type), rstd = 1 / sqrt(mean(h^2) + eps),
    y = h * rstd * weight, and y in 8 bits with a scale for each row's 128 values.
    Returns (data, scales, h, rstd), and y rounded to x's type as a fifth with
    ``normed``.  Without a residual h is x itself.
    """
    rows, cols, ld = _matrix(x, "x")
    real = _real(x, "x")
    wtype = _weight(weight, cols, x.device)
    fmt = _binding._enum(format, FP8_FORMATS, "format")
    h, res_ptr, ld_res, h_ptr, y_ptr = x, None, 0, None, None
    if residual is not None:
        _same(residual, x, "residual")
        ld_res = _matrix(residual, "residual")[2]
        res_ptr = residual.data_ptr()
    with _On(x.device, stream) as st:
        if residual is not None:
            h = torch.empty((rows, cols), dtype=x.dtype, device=x.device)
            h_ptr = h.data_ptr()
        data, scales, q = _new_fp8(rows, cols, fmt, 1, x.device)
        rstd = torch.empty((rows,), dtype=torch.float32, device=x.device)
        out = (data, scales, h, rstd)
        if normed:
            y = torch.empty((rows, cols), dtype=x.dtype, device=x.device)
            y_ptr = y.data_ptr()
            out += (y,)
        _check(lib().fp8_rmsnorm(x.data_ptr(), ld, res_ptr, ld_res, weight.data_ptr(), wtype, eps, rows, cols, real,
                                 h_ptr, cols, rstd.data_ptr(), y_ptr, cols, q, st), "fp8_rmsnorm")
    return out


def rmsnorm_backward(dy, h, weight, rstd, dresidual=None, *, weight_grad=True, stream=None):
    """Gradient of the norm: (dx, dweight) from the gradient of y and the stored h and rstd.

    dx, of h's type, is the gradient of both x and the residual; ``dresidual``
    (the gradient that reaches h past the norm) is added to it.  dweight is
    float32, or None with ``weight_grad=False``.
    """
    rows, cols, ld_dy = _matrix(dy, "dy")
    real = _real(dy, "dy")
    _same(h, dy, "h")
    ld_h = _matrix(h, "h")[2]
    wtype = _weight(weight, cols, dy.device)
    if rstd.dtype != torch.float32 or rstd.shape != (rows,) or rstd.device != dy.device or not rstd.is_contiguous():
        raise ValueError("rstd must be %d contiguous float32 values on %s" % (rows, dy.device))
    res_ptr, ld_res = None, 0
    if dresidual is not None:
        _same(dresidual, dy, "dresidual")
        ld_res = _matrix(dresidual, "dresidual")[2]
        res_ptr = dresidual.data_ptr()
    with _On(dy.device, stream) as st:
        dx = torch.empty((rows, cols), dtype=dy.dtype, device=dy.device)
        dw = torch.empty((cols,), dtype=torch.float32, device=dy.device) if weight_grad else None
        _check(lib().fp8_rmsnorm_backward(dy.data_ptr(), ld_dy, h.data_ptr(), ld_h, res_ptr, ld_res,
                                          weight.data_ptr(), wtype, rstd.data_ptr(), rows, cols, real, dx.data_ptr(),
                                          cols, dw.data_ptr() if weight_grad else None, st), "fp8_rmsnorm_backward")
    return dx, dw


def _weight(weight, cols, device):
    if weight.shape != (cols,) or weight.device != device or (cols > 1 and weight.stride(0) != 1):
        raise ValueError("weight must be %d contiguous values on %s" % (cols, device))
    return _real(weight, "weight")
