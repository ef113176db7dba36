"""The feed-forward operators in 16 bits on torch tensors (C ABI: include/gemm_ffn.h).

A block of a network, forward and backward, around its two products:

    y = linear(x, W, b, activation=..., residual=...)       one kernel
    h = gated(x, Wg, Wu, activation="silu")                 act(x Wg^T) * (x Wu^T), one kernel

with what the backward pass needs of them (the values before the activation)
kept in the inputs' type or in 8 bits (E4M3 codes with a scale for each row's
128 values, as ``quantize_fp8`` makes them), and ``linear_backward`` and
``gated_backward`` that read either.

The calls are below autograd, as those of ``fp8``: results carry no graph, also
where operands require gradients, and a ``torch.autograd.Function`` around a
forward and its backward call is the program's to write.  What is written to
``out`` counts as a change of that tensor in place.

Matrices are float16 or bfloat16 with contiguous rows; an output may be float32
where it says so.  The tensor cores want rows that begin on 16-byte boundaries:
new outputs are laid out that way (their rows may be a few elements apart), and
an operand that is not is copied first.  Everything runs on the current stream
of the tensors' device (or ``stream``).  The checks of arguments and the
allocations are compiled (``csrc/torch_ffn.cpp``): a refused argument raises
``ValueError``, a failing call ``GemmError``.
"""
import importlib
import struct

import torch

from . import _binding
from ._binding import ACTIVATIONS, GemmError, GpFfnOptions, GpPlan, lib
from .fp8 import _check, _On

_KEEP = {None: 0, "real": 1, "fp8": 2}
_packed = struct.Struct("Qiii4x").pack        # gp_ffn_options


def _pack(timeout_ns, tile, k_splits, inject_lost_load):
    try:
        return _packed(timeout_ns, tile, k_splits, inject_lost_load)
    except struct.error as e:
        raise ValueError("timeout_ns, tile, k_splits and inject_lost_load: %s" % e) from None


def _load():
    """The compiled half of this module; raises if it has not been built."""
    lib()
    try:
        module = importlib.import_module("._torch_ffn", __package__)
    except ImportError as e:
        raise RuntimeError("_torch_ffn.so is not built (run software_pipelined_tiled_pipeline_gb300.build.build())") from e
    module.load(_binding.LIB_PATH, GemmError)
    return module


_calls = _load()


def _activation(name):
    """The number of an activation's name."""
    act = ACTIVATIONS.get(name, 0 if name is None else -1)
    if act < 0:
        raise ValueError("unknown activation %r" % (name,))
    return act


def _keep(name):
    keep = _KEEP.get(name, -1)
    if keep < 0:
        raise ValueError("unknown keep %r" % (name,))
    return keep


def _device_of(x, name):
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError("%s must be on a CUDA device" % name)
    return x.get_device()


def linear(x, weight, bias=None, *, activation=None, residual=None, keep=None, out=None, out_dtype=None, stream=None, tile=0,
           k_splits=0, timeout_ns=0, inject_lost_load=False):
    """y = act(x W^T + bias) + residual, rounded once.  x: M x K, weight: N x K, float16 or bfloat16.

    ``activation``: None, "relu", "gelu", "gelu_tanh", "silu" or "sigmoid".
    ``bias``: N values of x's type or float32.  ``residual``: M x N of the
    output's type; it may be ``out`` itself.  ``out``: where to write, apart
    from what is read; ``out_dtype``: x's type or float32.  ``keep``: "real" or
    "fp8" also returns the values before the activation, as ``kept`` of
    ``linear_backward``: (z,) in x's type, or (codes, scales).  (Without an
    activation the backward pass needs, and takes, none of them.)  Activations
    are off by up to 1e-6 relative where they are not small, and up to 1e-5 in
    the tails that fall towards 0, which shows in float32 outputs alone.  ``tile``,
    ``k_splits``, ``timeout_ns``, ``inject_lost_load``: see gp_ffn_options.

    Returns y, or (y, kept) with ``keep``.
    """
    if stream is not None:
        with _On(_device_of(x, "x"), stream):
            return linear(x, weight, bias, activation=activation, residual=residual, keep=keep, out=out, out_dtype=out_dtype,
                          tile=tile, k_splits=k_splits, timeout_ns=timeout_ns, inject_lost_load=inject_lost_load)
    opts = _pack(timeout_ns, tile, k_splits, inject_lost_load) if tile or k_splits or timeout_ns or inject_lost_load else None
    return _calls.linear(x, weight, bias, _activation(activation), residual, _keep(keep), out, out_dtype, opts)


def gated(x, w_gate, w_up, *, activation="silu", keep=None, out=None, stream=None, tile=0, k_splits=0, timeout_ns=0,
          inject_lost_load=False):
    """h = act(x Wg^T) * (x Wu^T), both products in one kernel, rounded once.  x: M x K, weights: N x K.

    ``keep``: "real" or "fp8" also returns both products, as ``kept`` of
    ``gated_backward``: (g, u) in x's type, or (codes of g, scales, codes of u,
    scales).  Other arguments as in ``linear``.

    Returns h, or (h, kept) with ``keep``.
    """
    if stream is not None:
        with _On(_device_of(x, "x"), stream):
            return gated(x, w_gate, w_up, activation=activation, keep=keep, out=out, tile=tile, k_splits=k_splits,
                         timeout_ns=timeout_ns, inject_lost_load=inject_lost_load)
    opts = _pack(timeout_ns, tile, k_splits, inject_lost_load) if tile or k_splits or timeout_ns or inject_lost_load else None
    return _calls.gated(x, w_gate, w_up, _activation(activation), _keep(keep), out, opts)


def linear_backward(dy, x, weight, *, activation=None, kept=None, bias_grad=False, input_grad=True, weight_grad=True,
                    out_dtype=None, addend=None, out=None, stream=None, tile=0, k_splits=0, timeout_ns=0, inject_lost_load=0):
    """Gradients of y = act(x W^T + bias) + residual: (dx, dweight, dbias); the residual's is dy itself.

    ``kept``: what ``linear`` returned with ``keep``, where there is an
    activation.  dz = dy * act'(z) is rounded to x's type for the two products.
    dx has x's type, dweight x's type or ``out_dtype`` (float32), and is written
    to ``out`` if given (apart from x and dy); ``addend`` (of dweight's type, may
    be ``out`` itself) is added to it in FP32.  dbias (float32) is summed from dz
    before its rounding.  What is not asked for (``input_grad``, ``weight_grad``,
    ``bias_grad``) is None; without ``weight_grad`` x may be None too.
    ``gemm_stats(sync=True)`` speaks of both products: a wait that gave up in
    either is its status.  ``inject_lost_load``: 1 in dx's product, 2 in
    dweight's, 3 in both.
    """
    if stream is not None:
        with _On(_device_of(dy, "dy"), stream):
            return linear_backward(dy, x, weight, activation=activation, kept=kept, bias_grad=bias_grad,
                                   input_grad=input_grad, weight_grad=weight_grad, out_dtype=out_dtype, addend=addend, out=out,
                                   tile=tile, k_splits=k_splits, timeout_ns=timeout_ns, inject_lost_load=inject_lost_load)
    opts = _pack(timeout_ns, tile, k_splits, inject_lost_load) if tile or k_splits or timeout_ns or inject_lost_load else None
    return _calls.linear_backward(dy, x, weight, _activation(activation), kept, bool(bias_grad), bool(input_grad),
                                  bool(weight_grad), out_dtype, addend, out, opts)


def gated_backward(dh, x, w_gate, w_up, kept, *, activation="silu", product=False, input_grad=True, weight_grad=True,
                   out_dtype=None, addend=None, out=None, stream=None, tile=0, k_splits=0, timeout_ns=0, inject_lost_load=0):
    """Gradients of h = act(x Wg^T) * (x Wu^T): (dx, dw_gate, dw_up), and h once more with ``product``.

    ``kept``: what ``gated`` returned with ``keep``.  The gradients of both
    products are rounded to x's type for the products behind them.  ``out_dtype``,
    ``addend``, ``out`` as in ``linear_backward``, the last two a pair each.
    h, for the gradient of the weight that reads it, need not have been kept.
    Without ``weight_grad`` x may be None.  ``inject_lost_load`` and what
    ``gemm_stats`` says as in ``linear_backward``.
    """
    if stream is not None:
        with _On(_device_of(dh, "dh"), stream):
            return gated_backward(dh, x, w_gate, w_up, kept, activation=activation, product=product, input_grad=input_grad,
                                  weight_grad=weight_grad, out_dtype=out_dtype, addend=addend, out=out, tile=tile,
                                  k_splits=k_splits, timeout_ns=timeout_ns, inject_lost_load=inject_lost_load)
    opts = _pack(timeout_ns, tile, k_splits, inject_lost_load) if tile or k_splits or timeout_ns or inject_lost_load else None
    return _calls.gated_backward(dh, x, w_gate, w_up, kept, _activation(activation), bool(product), bool(input_grad),
                                 bool(weight_grad), out_dtype, addend, out, opts)


OPERATORS = {"linear": 0, "gated": 1, "input_grad": 2, "weight_grad": 3}


def ffn_plan(op, M, N, K, *, count=1, kept=False, dtype=torch.bfloat16, out_dtype=None, sms=0, tile=0, k_splits=0) -> dict:
    """The kernel and tile that a product of ``linear``, ``gated`` or a backward pass would take (see gemm_ffn_plan).

    ``kept``: True where values are kept in 8 bits.  ``dtype``, ``out_dtype``: of the operands, and of what is written.
    """
    p = GpPlan()
    opts = GpFfnOptions(0, int(tile), int(k_splits), 0)
    if dtype not in (torch.float16, torch.bfloat16) or out_dtype not in (None, dtype, torch.float32):
        raise ValueError("no product of %s into %s" % (dtype, out_dtype))
    flags = int(kept) + 2 * (out_dtype is torch.float32) + 4 * (dtype is torch.float16)
    _check(lib().gemm_ffn_plan(_binding._enum(op, OPERATORS, "op"), M, N, K, count, flags, sms, opts, p), "gemm_ffn_plan")
    return p.as_dict()
