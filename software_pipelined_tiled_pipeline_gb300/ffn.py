"""The feed-forward operators in 16 bits on torch tensors (C ABI: include/gemm_ffn.h).

A block of a network, forward and backward, around its two products:

    y = linear(x, W, b, activation=..., residual=...)       one kernel
    h = gated(x, Wg, Wu, activation="silu")                 act(x Wg^T) * (x Wu^T), one kernel

with what the backward pass needs of them (the values before the activation)
kept in the inputs' type or in 8 bits (E4M3 codes with a scale for each row's
128 values, as ``quantize_fp8`` makes them), and ``linear_backward`` and
``gated_backward`` that read either.

Matrices are float16 or bfloat16 with contiguous rows; an output may be float32
where it says so.  The tensor cores want rows that begin on 16-byte boundaries:
new outputs are laid out that way (their rows may be a few elements apart), and
an operand that is not is copied first.  Everything runs on the current stream
of the tensors' device (or ``stream``); this module allocates outputs and passes
pointers, and a failing call raises ``GemmError``.
"""
import ctypes
import functools
import struct

import torch

from . import _binding
from ._binding import ACTIVATIONS, GpFfnOptions, GpPlan, ffn_calls, lib
from .fp8 import _FORMAT_OF, _REAL_OF, _check, _device, _elsewhere, _empty, _matrix, _new_fp8, _On, _raw_stream

_F32 = torch.float32
_TYPE_OF = {torch.float16: 0, torch.bfloat16: 1}
_NO_CODES = struct.pack("PPqqqii", 0, 0, 0, 0, 0, 0, 0)
_linear = struct.Struct("6P48s8q4i").pack
_gated = struct.Struct("6P48s48s9q2i").pack
_input_grad = struct.Struct("5P8q4i").pack
_weight_grad = struct.Struct("7P10q4i").pack
_act_backward = struct.Struct("2P48s3P6q2i").pack
_gated_backward = struct.Struct("3P48s48s3P8q2i").pack
_codes = struct.Struct("PPqqqii").pack


def _options(tile, k_splits, timeout_ns, inject_lost_load):
    if tile or k_splits or timeout_ns or inject_lost_load:
        return GpFfnOptions(int(timeout_ns), int(tile), int(k_splits), int(inject_lost_load))
    return None


def _activation(name):
    if name is None:
        return 0
    act = ACTIVATIONS.get(name)
    if act is None:
        raise ValueError("unknown activation %r" % (name,))
    return act


def _type(x, name):
    t = _TYPE_OF.get(x.dtype)
    if t is None:
        raise ValueError("%s must be float16 or bfloat16, got %s" % (name, x.dtype))
    return t


def _operand(x, name, like=None):
    """(rows, cols, row stride, tensor) of a product's operand: x itself, or a copy whose rows begin on 16-byte boundaries."""
    rows, cols, ld = _matrix(x, name)
    if like is not None and (x.dtype is not like.dtype or x.get_device() != like.get_device()):
        raise ValueError("%s is %s on %s: want %s on %s" % (name, x.dtype, x.device, like.dtype, like.device))
    if rows <= 1:
        ld = (cols + 7) // 8 * 8       # the stride of a single row is never used
    if (x.data_ptr() | (ld << 1)) & 15:
        if ld < cols:
            raise ValueError("the rows of %s overlap" % name)
        wide = (cols + 7) // 8 * 8
        packed = _empty((rows, cols), (wide, 1), dtype=x.dtype, device=x.device)
        _check(ffn_calls().pack(x.data_ptr(), ld, packed.data_ptr(), wide, rows, cols, _raw_stream(x.get_device())),
               "ffn_pack_rows")
        return rows, cols, wide, packed
    return rows, cols, ld, x


def _new(rows, cols, dtype, device):
    """An output whose rows begin on 16-byte boundaries, and its row stride."""
    ld = (cols + 3) // 4 * 4 if dtype is _F32 else (cols + 7) // 8 * 8
    return _empty((rows, cols), (ld, 1), dtype=dtype, device=device), ld


def _shaped(x, rows, cols, dtype, device, name):
    """The row stride of a rows x cols matrix of that type on that device."""
    r, c, ld = _matrix(x, name)
    if (r, c) != (rows, cols) or x.dtype is not dtype or x.get_device() != device:
        raise ValueError("%s must be %s %s on cuda:%d: got %s %s on %s" % (
            name, (rows, cols), dtype, device, tuple(x.shape), x.dtype, x.device))
    return ld


def _out_type(x, out_dtype):
    if out_dtype is None or out_dtype is x.dtype:
        return x.dtype
    if out_dtype is not _F32:
        raise ValueError("out_dtype must be %s or float32, got %s" % (x.dtype, out_dtype))
    return out_dtype


def _kept_codes(data, scales, rows, cols, device, name):
    """The descriptor of values kept in 8 bits."""
    fmt = _FORMAT_OF.get(data.dtype)
    r, c, ld = _matrix(data, name)
    if fmt is None or (r, c) != (rows, cols) or data.get_device() != device:
        raise ValueError("%s must be an 8-bit %s matrix on cuda:%d: got %s %s on %s" % (
            name, (rows, cols), device, tuple(data.shape), data.dtype, data.device))
    if rows <= 1:
        ld = (cols + 15) // 16 * 16
    if scales.dtype is not _F32 or scales.shape != (rows, (cols + 127) // 128) or scales.get_device() != device:
        raise ValueError("the scales of %s must be float32 %s on its device" % (name, (rows, (cols + 127) // 128)))
    sr, sc = scales.stride()
    return _codes(data.data_ptr(), scales.data_ptr(), ld, sr, sc, fmt, 1)


def _kept(kept, weights, rows, cols, dtype, device):
    """((pointer, row stride) of each matrix kept as it is, descriptors of those kept in 8 bits)."""
    if isinstance(kept, torch.Tensor):
        kept = (kept,)
    names = ("kept[0]",) if weights == 1 else ("the gate's kept values", "the other kept values")
    if kept is not None and len(kept) == weights:
        return [(z.data_ptr(), _shaped(z, rows, cols, dtype, device, n)) for z, n in zip(kept, names)], [_NO_CODES] * weights
    if kept is not None and len(kept) == 2 * weights:
        return [(None, 0)] * weights, [_kept_codes(kept[2 * i], kept[2 * i + 1], rows, cols, device, names[i])
                                       for i in range(weights)]
    raise ValueError("kept must be what the forward call returned: %d matrices, or %d with their scales" % (weights, 2 * weights))


def linear(x, weight, bias=None, *, activation=None, residual=None, keep=None, out=None, out_dtype=None, stream=None,
           tile=0, k_splits=0, timeout_ns=0, inject_lost_load=False):
    """y = act(x W^T + bias) + residual, rounded once.  x: M x K, weight: N x K, float16 or bfloat16.

    ``activation``: None, "relu", "gelu", "gelu_tanh", "silu" or "sigmoid".
    ``bias``: N values of x's type or float32.  ``residual``: M x N of the
    output's type; it may be ``out`` itself.  ``out``: where to write;
    ``out_dtype``: x's type or float32.  ``keep``: "real" or "fp8" also returns
    the values before the activation, as ``kept`` of ``linear_backward``: (z,)
    in x's type, or (codes, scales).  ``tile``, ``k_splits``, ``timeout_ns``,
    ``inject_lost_load``: see gp_ffn_options.

    Returns y, or (y, kept) with ``keep``.
    """
    if _elsewhere(x, "x", stream):
        with _On(x.get_device(), stream):
            return linear(x, weight, bias, activation=activation, residual=residual, keep=keep, out=out, out_dtype=out_dtype,
                          tile=tile, k_splits=k_splits, timeout_ns=timeout_ns, inject_lost_load=inject_lost_load)
    real = _type(x, "x")
    act = _activation(activation)
    M, K, ldx, x = _operand(x, "x")
    N, kw, ldw, weight = _operand(weight, "weight", x)
    if kw != K:
        raise ValueError("x has %d columns and weight %d" % (K, kw))
    device = x.get_device()
    b_ptr, b_type = None, real
    if bias is not None:
        if bias.shape != (N,) or bias.get_device() != device or (N > 1 and bias.stride(0) != 1) or (
                bias.dtype is not _F32 and bias.dtype is not x.dtype):
            raise ValueError("bias must be %d contiguous values of %s or float32 on %s" % (N, x.dtype, x.device))
        b_ptr, b_type = bias.data_ptr(), _REAL_OF[bias.dtype]
    if out is None:
        out, ldy = _new(M, N, _out_type(x, out_dtype), x.device)
    else:
        if out_dtype is not None and out.dtype is not out_dtype:
            raise ValueError("out is %s: out_dtype %s asks for another type" % (out.dtype, out_dtype))
        ldy = _shaped(out, M, N, _out_type(x, out.dtype), device, "out")
    r_ptr, ld_res = None, 0
    if residual is not None:
        ld_res = _shaped(residual, M, N, out.dtype, device, "residual")
        r_ptr = residual.data_ptr()
    z_ptr, ldz, q, kept = None, 0, _NO_CODES, None
    if keep is not None:
        if keep == "real":
            z, ldz = _new(M, N, x.dtype, x.device)
            z_ptr, kept = z.data_ptr(), (z,)
        elif keep == "fp8":
            data, scales, q = _new_fp8(M, N, 0, 1, x.device)
            kept = (data, scales)
        else:
            raise ValueError("unknown keep %r" % (keep,))
    args = _linear(x.data_ptr(), weight.data_ptr(), b_ptr or 0, r_ptr or 0, out.data_ptr(), z_ptr or 0, q, M, N, K, ldx, ldw,
                   ld_res, ldy, ldz, real, _REAL_OF[out.dtype], b_type, act)
    _check(ffn_calls().linear(args, _raw_stream(device), _options(tile, k_splits, timeout_ns, inject_lost_load)),
           "gemm_linear")
    return out if kept is None else (out, kept)


def gated(x, w_gate, w_up, *, activation="silu", keep=None, out=None, stream=None, tile=0, k_splits=0, timeout_ns=0,
          inject_lost_load=False):
    """h = act(x Wg^T) * (x Wu^T), both products in one kernel, rounded once.  x: M x K, weights: N x K.

    ``keep``: "real" or "fp8" also returns both products, as ``kept`` of
    ``gated_backward``: (g, u) in x's type, or (codes of g, scales, codes of u,
    scales).  Other arguments as in ``linear``.

    Returns h, or (h, kept) with ``keep``.
    """
    if _elsewhere(x, "x", stream):
        with _On(x.get_device(), stream):
            return gated(x, w_gate, w_up, activation=activation, keep=keep, out=out, tile=tile, k_splits=k_splits,
                         timeout_ns=timeout_ns, inject_lost_load=inject_lost_load)
    real = _type(x, "x")
    act = _activation(activation)
    M, K, ldx, x = _operand(x, "x")
    N, kg, ld_gate, w_gate = _operand(w_gate, "w_gate", x)
    nu, ku, ld_up, w_up = _operand(w_up, "w_up", x)
    if kg != K or (nu, ku) != (N, K):
        raise ValueError("x has %d columns: the weights are %s and %s" % (K, tuple(w_gate.shape), tuple(w_up.shape)))
    device = x.get_device()
    if out is None:
        out, ldh = _new(M, N, x.dtype, x.device)
    else:
        ldh = _shaped(out, M, N, x.dtype, device, "out")
    zg, zu, ldz, qg, qu, kept = 0, 0, 0, _NO_CODES, _NO_CODES, None
    if keep is not None:
        if keep == "real":
            g, ldz = _new(M, N, x.dtype, x.device)
            u, ldz = _new(M, N, x.dtype, x.device)
            zg, zu, kept = g.data_ptr(), u.data_ptr(), (g, u)
        elif keep == "fp8":
            g, gs, qg = _new_fp8(M, N, 0, 1, x.device)
            u, us, qu = _new_fp8(M, N, 0, 1, x.device)
            kept = (g, gs, u, us)
        else:
            raise ValueError("unknown keep %r" % (keep,))
    args = _gated(x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), out.data_ptr(), zg, zu, qg, qu, M, N, K, ldx, ld_gate,
                  ld_up, ldh, ldz, ldz, real, act)
    _check(ffn_calls().gated(args, _raw_stream(device), _options(tile, k_splits, timeout_ns, inject_lost_load)), "gemm_gated")
    return out if kept is None else (out, kept)


def _input_gradient(dz, weights, M, N, K, real, x, opts):
    """dx of one product or of a pair: dz and weights are (pointer, row stride) of each."""
    dx, ld = _new(M, K, x.dtype, x.device)
    n = len(dz)
    (a, lda), (b, ldb), (w, ldw), (v, ldv) = dz[0], dz[-1], weights[0], weights[-1]
    args = _input_grad(a, b, w, v, dx.data_ptr(), M, N, K, lda, ldb, ldw, ldv, ld, real, real, n, 0)
    _check(ffn_calls().input_grad(args, _raw_stream(x.get_device()), opts), "gemm_input_grad")
    return dx


def _weight_gradients(dz, x, ldx, M, N, K, real, out_dtype, addend, out, opts):
    """The gradients of the weights that share x: lists of one or two."""
    n = len(dz)
    device = x.get_device()
    out = list(out) if out is not None else [None] * n
    addend = list(addend) if addend is not None else [None] * n
    if len(out) != n or len(addend) != n or (n == 2 and (addend[0] is None) != (addend[1] is None)):
        raise ValueError("addend and out take %d matrices" % n)
    dtype = _out_type(x, out_dtype if out_dtype is not None else next((t.dtype for t in out + addend if t is not None), None))
    at, adds = [], []
    for i in range(n):
        if out[i] is None:
            out[i], ld = _new(N, K, dtype, x.device)
        else:
            ld = _shaped(out[i], N, K, dtype, device, "out")
        at.append((out[i].data_ptr(), ld))
        adds.append((0, 0) if addend[i] is None else (addend[i].data_ptr(), _shaped(addend[i], N, K, dtype, device, "addend")))
    args = _weight_grad(dz[0][0], dz[-1][0], x.data_ptr(), adds[0][0], adds[-1][0], at[0][0], at[-1][0], M, N, K, dz[0][1],
                        dz[-1][1], ldx, adds[0][1], adds[-1][1], at[0][1], at[-1][1], real, _REAL_OF[dtype], n, 0)
    _check(ffn_calls().weight_grad(args, _raw_stream(device), opts), "gemm_weight_grad")
    return out


@functools.lru_cache(maxsize=256)
def _bias_workspace(M, N, device):
    """Bytes that the bias gradient needs on `device`, the current one."""
    size = ctypes.c_int64()
    _check(lib().ffn_act_backward_workspace(M, N, 0, size), "ffn_act_backward_workspace")
    return size.value


def linear_backward(dy, x, weight, *, activation=None, kept=None, bias_grad=False, input_grad=True, weight_grad=True,
                    out_dtype=None, addend=None, out=None, stream=None, tile=0, timeout_ns=0):
    """Gradients of y = act(x W^T + bias) + residual: (dx, dweight, dbias); the residual's is dy itself.

    ``kept``: what ``linear`` returned with ``keep``, where there is an
    activation.  dz = dy * act'(z) is rounded to x's type for the two products.
    dx has x's type, dweight x's type or ``out_dtype`` (float32), and is written
    to ``out`` if given; ``addend`` (of dweight's type, may be ``out`` itself) is
    added to it in FP32.  dbias (float32) is summed from dz before its rounding.
    What is not asked for (``input_grad``, ``weight_grad``, ``bias_grad``) is None.
    """
    if _elsewhere(dy, "dy", stream):
        with _On(dy.get_device(), stream):
            return linear_backward(dy, x, weight, activation=activation, kept=kept, bias_grad=bias_grad,
                                   input_grad=input_grad, weight_grad=weight_grad, out_dtype=out_dtype, addend=addend, out=out,
                                   tile=tile, timeout_ns=timeout_ns)
    real = _type(dy, "dy")
    act = _activation(activation)
    if not act and kept is not None:
        raise ValueError("without an activation nothing is kept")
    if not weight_grad and (addend is not None or out is not None):
        raise ValueError("addend and out are for dweight")
    opts = _options(tile, 0, timeout_ns, False)
    M, N, ldd = _matrix(dy, "dy")
    device = dy.get_device()
    if act or bias_grad:
        (z, ldz), code = (0, 0), _NO_CODES
        dz, dz_ptr = dy, 0
        if act:
            zs, codes = _kept(kept, 1, M, N, dy.dtype, device)
            (z, ldz), code = zs[0], codes[0]
            if input_grad or weight_grad:
                dz, ldz_out = _new(M, N, dy.dtype, dy.device)
                dz_ptr = dz.data_ptr()
        dbias, db_ptr, work, work_bytes = None, 0, None, 0
        if bias_grad:
            dbias = _empty((N,), (1,), dtype=_F32, device=dy.device)
            db_ptr = dbias.data_ptr()
            work_bytes = _bias_workspace(M, N, device)
            if work_bytes:
                work = _empty((work_bytes // 4,), (1,), dtype=_F32, device=dy.device)   # (freed in the call's stream order)
        args = _act_backward(dy.data_ptr(), z or 0, code, dz_ptr, db_ptr, work.data_ptr() if work is not None else 0, work_bytes,
                             M, N, ldd, ldz, ldz_out if dz_ptr else 0, real, act)
        _check(ffn_calls().act_backward(args, _raw_stream(device)), "ffn_act_backward")
    else:
        dz, dbias = dy, None
    dx = dw = None
    if input_grad or weight_grad:
        _, _, ldd, dz = _operand(dz, "dy")
        mx, K, ldx, x = _operand(x, "x", dy)
        if mx != M or weight.shape != (N, K):
            raise ValueError("dy is %s and x %s: the weight is %s" % ((M, N), (mx, K), tuple(weight.shape)))
        at = [(dz.data_ptr(), ldd)]
        if input_grad:
            _, _, ldw, weight = _operand(weight, "weight", dy)
            dx = _input_gradient(at, [(weight.data_ptr(), ldw)], M, N, K, real, x, opts)
        if weight_grad:
            dw = _weight_gradients(at, x, ldx, M, N, K, real, out_dtype, None if addend is None else [addend],
                                   None if out is None else [out], opts)[0]
    return dx, dw, dbias


def gated_backward(dh, x, w_gate, w_up, kept, *, activation="silu", product=False, input_grad=True, weight_grad=True,
                   out_dtype=None, addend=None, out=None, stream=None, tile=0, timeout_ns=0):
    """Gradients of h = act(x Wg^T) * (x Wu^T): (dx, dw_gate, dw_up), and h once more with ``product``.

    ``kept``: what ``gated`` returned with ``keep``.  The gradients of both
    products are rounded to x's type for the products behind them.  ``out_dtype``,
    ``addend``, ``out`` as in ``linear_backward``, the last two a pair each.
    h, for the gradient of the weight that reads it, need not have been kept.
    """
    if _elsewhere(dh, "dh", stream):
        with _On(dh.get_device(), stream):
            return gated_backward(dh, x, w_gate, w_up, kept, activation=activation, product=product, input_grad=input_grad,
                                  weight_grad=weight_grad, out_dtype=out_dtype, addend=addend, out=out, tile=tile,
                                  timeout_ns=timeout_ns)
    real = _type(dh, "dh")
    act = _activation(activation)
    if not weight_grad and (addend is not None or out is not None):
        raise ValueError("addend and out are for the weights' gradients")
    opts = _options(tile, 0, timeout_ns, False)
    M, N, ldd = _matrix(dh, "dh")
    device = dh.get_device()
    mx, K, ldx, x = _operand(x, "x", dh)
    if mx != M or w_gate.shape != (N, K) or w_up.shape != (N, K):
        raise ValueError("dh is %s and x %s: the weights are %s and %s" % (
            (M, N), (mx, K), tuple(w_gate.shape), tuple(w_up.shape)))
    ((zg, ldg), (zu, ldu)), (qg, qu) = _kept(kept, 2, M, N, dh.dtype, device)
    ld = (N + 7) // 8 * 8
    both = _empty((2 * M, N), (ld, 1), dtype=dh.dtype, device=dh.device)      # the products' gradients, one after the other
    dgate = both.data_ptr()
    dup = dgate + 2 * M * ld
    h, ldh, h_ptr = None, 0, 0
    if product:
        h, ldh = _new(M, N, dh.dtype, dh.device)
        h_ptr = h.data_ptr()
    args = _gated_backward(dh.data_ptr(), zg or 0, zu or 0, qg, qu, dgate, dup, h_ptr, M, N, ldd, ldg, ldu, ld, ld, ldh, real,
                           act)
    _check(ffn_calls().gated_backward(args, _raw_stream(device)), "ffn_gated_backward")
    dz = [(dgate, ld), (dup, ld)]
    dx, dws = None, (None, None)
    if input_grad:
        _, _, ldg, w_gate = _operand(w_gate, "w_gate", dh)
        _, _, ldu, w_up = _operand(w_up, "w_up", dh)
        dx = _input_gradient(dz, [(w_gate.data_ptr(), ldg), (w_up.data_ptr(), ldu)], M, N, K, real, x, opts)
    if weight_grad:
        dws = _weight_gradients(dz, x, ldx, M, N, K, real, out_dtype, addend, out, opts)
    return (dx, dws[0], dws[1], h) if product else (dx, dws[0], dws[1])


OPERATORS = {"linear": 0, "gated": 1, "input_grad": 2, "weight_grad": 3}


def ffn_plan(op, M, N, K, *, count=1, kept=False, sms=0, tile=0, k_splits=0) -> dict:
    """The kernel and tile that a product of ``linear``, ``gated`` or a backward pass would take (see gemm_ffn_plan)."""
    p = GpPlan()
    opts = GpFfnOptions(0, int(tile), int(k_splits), 0)
    _check(lib().gemm_ffn_plan(_binding._enum(op, OPERATORS, "op"), M, N, K, count, int(kept), sms, opts, p), "gemm_ffn_plan")
    return p.as_dict()
