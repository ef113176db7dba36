"""Plain implementations of the feed-forward operators for the tests, in
float64, and how far the library may be from them."""
import math

import numpy as np
import torch
from scipy.special import erfc, expit

import fp8_ref

REAL = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half the spacing at 1
LEAST = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}
LARGEST = {torch.float16: 65520.0, torch.bfloat16: math.inf, torch.float32: math.inf}
ACTS = [None, "relu", "gelu", "gelu_tanh", "silu", "sigmoid"]
RESTART = 768          # of the summed axis per accumulator where FP32 leaves


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def inner(z):
    return 2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)


def value(z, act):
    if act is None:
        return z
    if act == "relu":
        return np.where(z > 0, z, 0.0)
    if act == "gelu":
        return z * 0.5 * erfc(-z / math.sqrt(2.0))
    if act == "gelu_tanh":
        return z * expit(inner(z))
    return expit(z) if act == "sigmoid" else z * expit(z)


def slope(z, act):
    if act is None:
        return np.ones_like(z)
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "gelu":
        return 0.5 * erfc(-z / math.sqrt(2.0)) + z * np.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        s, c = expit(inner(z)), expit(-inner(z))
        return s + z * s * c * 2.0 * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * z ** 2)
    s, c = expit(z), expit(-z)
    return s * c if act == "sigmoid" else s + z * s * c


def steps(z):
    """Relative error of an activation's FP32 evaluation, in units of 2^-24.  exp(t) is off by two spacings and by half a
    spacing of t, |t| of which there are (t = z, or inner(z), formed with four roundings); erfc is off by four spacings and
    its argument by one and a half, of which its relative derivative makes 2 t^2 = z^2 each; sums, products and a quotient
    add less than eight."""
    return 2.0 * z * z + 6.0 * np.abs(inner(z)) + 2.0 * np.abs(z) + 16.0


def sum_error(mag, summed, wide):
    """Largest error of a sum of `summed` products whose magnitudes add up to `mag`: the tensor cores cut each product's
    addition by 2^-23 of the sum of magnitudes so far at most; where FP32 leaves, they do so over RESTART products at a
    time, and those parts, and an addend that the sum may begin with, are added with 2^-24 each."""
    if wide:
        return (min(summed, RESTART) * 2.0 ** -23 + (summed // RESTART + 2) * 2.0 ** -24) * mag
    return (summed * 2.0 ** -23 + 2.0 ** -24) * mag


def rounded(x, err, dtype):
    """Error after rounding a value near x, already off by err, to dtype."""
    return err + UNIT[dtype] * (np.abs(x) + err) + LEAST[dtype]


def worst(got, want, bound, dtype=torch.float32):
    """Largest error in units of the bound; values past the type's range have to be infinite."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    if not got.size:
        return 0.0
    past = np.abs(want) + bound >= LARGEST[dtype]
    ok = np.isinf(got) & past & (np.sign(got) == np.sign(want))
    d = np.where(ok, 0.0, np.abs(got - want))
    return float(np.max(np.where(np.isnan(d), np.inf, d) / bound))


def kept_real(z, err, got):
    return worst(f64(got), z, rounded(z, err, got.dtype), got.dtype)


def kept_codes(z, err, data, scales):
    """Codes and scales against z, each value of which the kernel had off by at most err."""
    rows, cols = z.shape
    s = f64(scales)
    most = fp8_ref.group_max(np.abs(z), 1)
    off = fp8_ref.group_max(err, 1)
    floor = 2.0 ** -64
    want = np.maximum(most / 448.0, floor)
    a = worst(s, want, off / 448.0 + 2.0 ** -23 * want)          # (a correctly rounded quotient)
    wide = fp8_ref.spread(s, rows, cols, 1)
    code = fp8_ref.TABLE["e4m3"][fp8_ref.codes(data)]
    # a code is off by half a spacing: 2^-4 of the value, or of 2^-9, the least spacing; 1 / s and the product by 2^-23
    near = np.abs(z) / wide
    b = worst(code, z / wide, 2.0 ** -4 * near + 2.0 ** -10 + (err / wide + near * 2.0 ** -22) * 1.0625)
    return max(a, b)


def held(kept, dtype):
    """The values that were kept, in float64: of one product."""
    if len(kept) == 1:
        return f64(kept[0])
    data, scales = kept
    return fp8_ref.TABLE["e4m3" if data.dtype is torch.float8_e4m3fn else "e5m2"][fp8_ref.codes(data)] * fp8_ref.spread(
        f64(scales), *data.shape, 1)


GUARD = 512


def guarded(rows, cols, dtype, ld=None):
    """A NaN-filled output inside a NaN-filled buffer, and the buffer."""
    ld = ld or cols
    buf = torch.full((rows * ld + 2 * GUARD,), float("nan"), dtype=dtype, device="cuda")
    return buf[GUARD:GUARD + rows * ld].view(rows, ld)[:, :cols], buf


def outside_untouched(buf, rows, cols, ld):
    body = buf[GUARD:GUARD + rows * ld].view(rows, ld)
    return bool(torch.isnan(buf[:GUARD]).all() and torch.isnan(buf[GUARD + rows * ld:]).all()
                and torch.isnan(body[:, cols:]).all())


def matrix(rng, rows, cols, dtype, spread=1.0, pad=0, whole=None):
    """A random matrix on the GPU; `pad`: NaN elements between its rows."""
    x = rng.integers(-whole, whole + 1, (rows, cols)).astype(np.float64) if whole else rng.standard_normal((rows, cols)) * spread
    wide = torch.full((rows, cols + pad), float("nan"), dtype=dtype)
    wide[:, :cols] = torch.from_numpy(x).to(dtype)
    return wide.cuda()[:, :cols]


def magnitudes(a, b):
    return np.abs(a) @ np.abs(b).T
