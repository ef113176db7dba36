"""Plain implementations of the 8-bit operators for the tests, in NumPy: the
formats from their bit layouts, quantisation step by step in float32 (its
definition is float32 arithmetic, so codes and scales are compared for
equality), and the product, the norm and its gradient in float64."""
import numpy as np
import torch

GROUP = 128
FLOOR = np.float32(2.0 ** -64)
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}
TORCH = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
REAL = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
UNIT = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}   # half the spacing at 1


def decode_table(fmt):
    """The values of the 256 codes."""
    ebits, mbits, bias = (4, 3, 7) if fmt == "e4m3" else (5, 2, 15)
    out = np.zeros(256)
    for code in range(256):
        e, m = (code >> mbits) & ((1 << ebits) - 1), code & ((1 << mbits) - 1)
        v = m * 2.0 ** (1 - bias - mbits) if e == 0 else (1 + m / 2.0 ** mbits) * 2.0 ** (e - bias)
        if fmt == "e4m3":
            if e == 15 and m == 7:
                v = np.nan
        elif e == 31:
            v = np.nan if m else np.inf
        out[code] = -v if code & 0x80 else v
    return out


TABLE = {f: decode_table(f) for f in FMAX}


def encode(x, fmt):
    """Nearest code (ties to the even one), saturated at the largest finite value; NaN to 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    pos = TABLE[fmt][:128]
    pos = pos[np.isfinite(pos)]
    a = np.minimum(np.abs(x), FMAX[fmt])
    hi = np.clip(np.searchsorted(pos, a), 1, len(pos) - 1)
    lo = hi - 1
    up = a - pos[lo] > pos[hi] - a
    tie = a - pos[lo] == pos[hi] - a
    code = np.where(up | (tie & (hi % 2 == 0)), hi, lo)
    code = np.where(a == 0, 0, code)
    code = np.where(np.isnan(x), 0x7F, np.where(np.signbit(x), code + 128, code))
    return code.astype(np.uint8)


def group_max(x, high):
    """Largest magnitude of each group of `high` rows x 128 columns (a NaN stays)."""
    rows, cols = x.shape
    a = np.pad(np.abs(x), ((0, -rows % high), (0, -cols % GROUP)))
    return a.reshape(a.shape[0] // high, high, a.shape[1] // GROUP, GROUP).max(axis=(1, 3))


def spread(s, rows, cols, high):
    return np.repeat(np.repeat(s, high, 0)[:rows], GROUP, 1)[:, :cols]


def quantize(x, scales, fmt):
    """(codes, scales) of a float32 matrix, in float32 as the definition says."""
    x = np.asarray(x, dtype=np.float32)
    high = 1 if scales == "rows" else GROUP
    with np.errstate(all="ignore"):
        s = group_max(x, high) / np.float32(FMAX[fmt])
        s = np.where(s < FLOOR, FLOOR, s).astype(np.float32)
        inv = (np.float32(1.0) / s).astype(np.float32)
        y = (x * spread(inv, *x.shape, high)).astype(np.float32)
    return encode(y, fmt), s


def codes(t):
    """The codes of an 8-bit torch tensor."""
    return t.contiguous().view(torch.uint8).cpu().numpy()


def same_codes(got, want, fmt):
    """Equal codes; any NaN code stands for any other."""
    a, b = TABLE[fmt][got], TABLE[fmt][want]
    return np.array_equal(np.isnan(a), np.isnan(b)) and np.array_equal(got[~np.isnan(a)], want[~np.isnan(b)])


def values(code, s, fmt):
    """What codes and scales stand for, in float64."""
    rows, cols = code.shape
    high = 1 if s.shape[0] == rows else GROUP
    return TABLE[fmt][code] * spread(s.astype(np.float64), rows, cols, high)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


class Fp8:
    """A random 8-bit matrix on the host (codes, scales) and on the GPU (data, scales as passed)."""

    def __init__(self, rows, cols, scales, fmt, rng, order="groups", spread_log2=3.0, data=None):
        x = rng.standard_normal((rows, cols)) * np.exp2(spread_log2 * rng.standard_normal((rows, 1))) if data is None else data
        self.fmt = fmt
        self.code, self.s = quantize(x.astype(np.float32), scales, fmt)
        self.put(order)

    def put(self, order="groups", pad=None):
        rows, cols = self.code.shape
        ld = -(-cols // 16) * 16 if pad is None else pad
        wide = np.full((rows, ld), 0x7F, dtype=np.uint8)      # what lies between the rows reads as NaN
        wide[:, :cols] = self.code
        self.data = torch.from_numpy(wide).cuda().view(TORCH[self.fmt])[:, :cols]
        s = torch.from_numpy(self.s).cuda()
        if order == "groups":
            s = s.t().contiguous().t()
        elif order == "strided":
            s = s.repeat_interleave(3, 0).repeat_interleave(2, 1)[::3, ::2]
        self.scales = s
        return self

    @property
    def values(self):
        return values(self.code, self.s, self.fmt)


def gemm_bound(a, b, exact, out, addend=None):
    """Largest error of each output.  Within a K block the tensor cores add 128 exact products in FP32, each
    addition off by at most 2^-23 of the sum of magnitudes so far (they may cut instead of round); the product
    of the two scales and each FP32 addition of a block are off by 2^-24 relative to the sum of magnitudes, and the
    addend and the output's rounding by their unit of the result.  Half of the output's least spacing for
    numbers below its normal range."""
    mag = np.abs(a) @ np.abs(b).T
    blocks = -(-a.shape[1] // GROUP)
    fp32 = (GROUP * 2.0 ** -23 + (blocks + 2) * 2.0 ** -24) * mag
    if addend is not None:
        fp32 = fp32 + 2.0 ** -24 * (np.abs(exact) + np.abs(addend))
    least = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}[out]
    return fp32 + UNIT[out] * (np.abs(exact) + fp32) + least


def past_the_range(got, want, bound, out):
    """(got, want) with the right infinities taken out: an output past its type's largest number rounds to infinity."""
    if out != "f16":
        return got, want
    over = 65520.0                                    # the largest number, and half a spacing
    right = np.isinf(got) & (np.sign(got) == np.sign(want)) & (np.abs(want) + bound >= over)
    wrong = np.isfinite(got) & (np.abs(want) - bound >= over)
    assert not wrong.any(), "a finite output where the exact one is past the range"
    return np.where(right, 0.0, got), np.where(right, 0.0, want)
