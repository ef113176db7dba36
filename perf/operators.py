"""The FP8 operators as a user's program calls them, and their plain forms.

Four operators that belong together, all on 8-bit floating point with one FP32 scale for each 128 values along the
summed axis:

* ``quantize_fp8``: a matrix to 8 bits, with a scale for each row's 128 values or each 128 x 128 block, and the same
  transposed (the operands of a linear layer's three products);
* ``rmsnorm_fp8``: the residual's addition, the root-mean-square norm and the 8-bit output in one;
* ``rmsnorm_backward``: its gradient (the input's, the residual's and the weight's);
* ``gemm_fp8``: the matrix product of two such matrices, from one token to a training batch.

Each case is measured as a user's call makes it (``own`` true) and as elementary torch operations in 32 bits
(``own`` false).
"""
import math

import torch

own = False

GROUP = 128                      # values along the summed axis that share a scale
SCALE_FLOOR = 2.0 ** -64         # the least scale
MAX_OF = {"e4m3": 448.0, "e5m2": 57344.0}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
REAL = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-6


def listed():
    return [
        # one token through a square projection: the latency of single-token decoding
        gemm("token_4096", 1, 4096, 4096, "bf16"),
        # a batch of sequences decoded together: the weights' bytes bound it
        gemm("decode_batch_48", 48, 8192, 8192, "bf16"),
        # a short prompt through a projection with ragged sizes
        gemm("prompt_1000_ragged", 1000, 776, 2056, "f16"),
        # a weight's gradient over 8192 tokens, added to the one that is there; 8-bit gradients of the wider range,
        # both operands with a scale for each row's 128 tokens
        gemm("weight_gradient", 4096, 4096, 8192, "f32", a="e5m2", b_scales="rows", add=True),
        # the forward product of a training step (the repository's 8192 x 8192 x 4096 workload)
        gemm("forward_8192", 8192, 8192, 4096, "bf16"),
        # the norm in front of a projection, for one token
        norm("norm_token", 1, 4096, "bf16"),
        # the same for a prompt of 4096 tokens
        norm("norm_prompt", 4096, 8192, "bf16"),
        # the norm's gradient for a short ragged batch
        back("norm_gradient_ragged", 200, 2056, "f16"),
        # and for a training batch, with the gradient that comes along the residual
        back("norm_gradient_8192", 8192, 8192, "bf16"),
        # activations of a short ragged batch, for the forward product only
        quant("activations_ragged", 333, 1000, "f16", "rows", False),
        # activations or gradients of a training batch, for the forward product and the weight's gradient
        quant("activations_both", 8192, 8192, "bf16", "rows", True),
        # a weight kept in 32 bits, after each step of the optimiser: for the forward product and the input's gradient
        quant("weight_blocks", 8192, 4096, "f32", "blocks", True),
    ]


def gemm(name, m, n, k, out, a="e4m3", b="e4m3", a_scales="rows", b_scales="blocks", add=False):
    return dict(name=name, op="gemm", m=m, n=n, k=k, out=out, a=a, b=b, a_scales=a_scales, b_scales=b_scales, add=add)


def norm(name, rows, cols, type, residual=True, format="e4m3"):
    return dict(name=name, op="norm", rows=rows, cols=cols, type=type, residual=residual, format=format)


def back(name, rows, cols, type, residual=True):
    return dict(name=name, op="back", rows=rows, cols=cols, type=type, residual=residual)


def quant(name, rows, cols, type, scales, transpose, format="e4m3"):
    return dict(name=name, op="quant", rows=rows, cols=cols, type=type, scales=scales, transpose=transpose, format=format)


def draw(rng):
    """One more case: sizes spread over the logarithm, as odd as they come."""
    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return max(lo, min(hi, v))

    def no_name(case):
        del case["name"]
        return case

    op = rng.choice(["gemm", "gemm", "gemm", "norm", "back", "quant"])
    type = rng.choice(["f16", "bf16", "bf16", "f32"])
    if op == "gemm":
        m, n, k = size(1, 8192), size(64, 8192), size(64, 8192)
        k = min(k, 8192 * 8192 * 4096 // (m * n))
        return no_name(gemm("", m, n, k, type, a=rng.choice(["e4m3", "e4m3", "e5m2"]), b=rng.choice(["e4m3", "e4m3", "e5m2"]),
                            a_scales=rng.choice(["rows", "rows", "rows", "blocks"]), b_scales=rng.choice(["blocks", "blocks", "rows"]),
                            add=rng.random() < 0.3))
    rows, cols = size(1, 8192), size(64, 8192)
    if op == "norm":
        rows = min(rows, 4096)
        return no_name(norm("", rows, cols, type, rng.random() < 0.8, rng.choice(["e4m3", "e4m3", "e5m2"])))
    if op == "back":
        return no_name(back("", rows, cols, type, rng.random() < 0.8))
    return no_name(quant("", rows, cols, type, rng.choice(["rows", "rows", "blocks"]), rng.random() < 0.6, rng.choice(["e4m3", "e4m3", "e5m2"])))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _values(rows, cols, g, spread=1.0):
    """Normal values, with a few columns far larger than the others and each row at its own level, as activations and
    gradients have them."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    level = torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    loud = torch.where(torch.rand(1, cols, generator=g, device="cuda") < 0.004, 20.0, 1.0)
    return x.mul_(level).mul_(loud).mul_(spread)


def _padded(q):
    """`q` with rows that begin on 16-byte boundaries, as quantize_fp8 and rmsnorm_fp8 lay them out (their scales are
    stored with those of one group of 128 next to one another, whichever row they belong to)."""
    rows, cols = q.shape
    ld = -(-cols // 16) * 16
    if ld == cols:
        return q
    wide = torch.zeros(rows, ld, dtype=torch.uint8, device=q.device).view(q.dtype)
    wide[:, :cols].copy_(q)
    return wide[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    state = {"case": case}
    op = case["op"]
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        for side, rows, spread in (("a", m, 1.0), ("b", n, 0.02)):
            x = _values(rows, k, g, spread)
            if side == "a" and rows > 8:
                x[rows // 3] = 0.0                     # a token that only pads the batch
            q, s = quantize_plain(x, case[side + "_scales"], case[side])
            state[side], state[side + "_scales"] = _padded(q), s.t().contiguous().t()
        if case["add"]:
            state["add"] = torch.randn(m, n, generator=g, device="cuda").to(REAL[case["out"]])
        return state
    rows, cols, type = case["rows"], case["cols"], REAL[case["type"]]
    if op == "quant":
        spread = 0.02 if case["scales"] == "blocks" else 1.0
        state["x"] = _values(rows, cols, g, spread).to(type)
        return state
    state["weight"] = (1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(type)
    if op == "norm":
        state["x"] = _values(rows, cols, g).to(type)
        state["residual"] = _values(rows, cols, g, 3.0).to(type) if case["residual"] else None
        return state
    state["h"] = _values(rows, cols, g).to(type)
    state["rstd"] = torch.rsqrt(state["h"].float().square().mean(1) + EPS)
    state["dy"] = _values(rows, cols, g, 0.05).to(type)
    state["dresidual"] = _values(rows, cols, g, 0.05).to(type) if case["residual"] else None
    return state


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(state):
    import software_pipelined_tiled_pipeline_gb300 as gp

    case = state["case"]
    op = case["op"]
    if op == "gemm":
        return gp.gemm_fp8(state["a"], state["a_scales"], state["b"], state["b_scales"], out_dtype=REAL[case["out"]],
                           addend=state.get("add"))
    if op == "quant":
        return gp.quantize_fp8(state["x"], case["scales"], format=case["format"], transpose=case["transpose"])
    if op == "norm":
        return gp.rmsnorm_fp8(state["x"], state["weight"], state["residual"], eps=EPS, format=case["format"])
    return gp.rmsnorm_backward(state["dy"], state["h"], state["weight"], state["rstd"], state["dresidual"])


def _run_plain(state):
    case = state["case"]
    op = case["op"]
    if op == "gemm":
        a = dequantize_plain(state["a"], state["a_scales"])
        b = dequantize_plain(state["b"], state["b_scales"])
        c = a @ b.t()
        if case["add"]:
            c += state["add"].float()
        return c.to(REAL[case["out"]])
    if op == "quant":
        x = state["x"].float()
        got = quantize_plain(x, case["scales"], case["format"])
        return got + quantize_plain(x.t().contiguous(), case["scales"], case["format"]) if case["transpose"] else got
    if op == "norm":
        h = state["x"]
        if state["residual"] is not None:
            h = (h.float() + state["residual"].float()).to(h.dtype)
        wide = h.float()
        rstd = torch.rsqrt(wide.square().mean(1) + EPS)
        q, s = quantize_plain(wide * rstd[:, None] * state["weight"].float(), "rows", case["format"])
        return q, s, h, rstd
    dy, h, rstd = state["dy"].float(), state["h"].float(), state["rstd"][:, None]
    unit = h * rstd
    scaled = dy * state["weight"].float()
    dx = rstd * (scaled - unit * (scaled * unit).mean(1, keepdim=True))
    if state["dresidual"] is not None:
        dx += state["dresidual"].float()
    return dx.to(state["h"].dtype), (dy * unit).sum(0)


def _blocks(x, scales):
    """`x` padded with zeros and seen as [row groups, rows of one, groups along the row, 128]."""
    rows, cols = x.shape
    high = GROUP if scales == "blocks" else 1
    x = torch.nn.functional.pad(x, (0, -cols % GROUP, 0, -rows % high))
    return x.view(x.shape[0] // high, high, x.shape[1] // GROUP, GROUP)


def quantize_plain(x, scales, format):
    """(8-bit values, scales) of a 32-bit matrix: scale = max|x| / the format's largest value over each group."""
    rows, cols = x.shape
    wide = _blocks(x, scales)
    s = (wide.abs().amax((1, 3)) / MAX_OF[format]).clamp(min=SCALE_FLOOR)
    q = (wide * (1.0 / s)[:, None, :, None]).to(FP8[format])
    return q.view(wide.shape[0] * wide.shape[1], -1)[:rows, :cols], s


def dequantize_plain(q, s, to=torch.float32):
    """The values that 8-bit data and scales stand for."""
    rows, cols = q.shape
    high = GROUP if s.shape[0] < rows else 1
    wide = s.to(to).repeat_interleave(high, 0)[:rows].repeat_interleave(GROUP, 1)[:, :cols]
    return q.to(to) * wide


# ---------------------------------------------------------------------------
# what a pass cannot do without, and what it has to give
# ---------------------------------------------------------------------------
def _scale_bytes(rows, cols, scales):
    return 4 * (-(-rows // GROUP) if scales == "blocks" else rows) * -(-cols // GROUP)


def work(case):
    op = case["op"]
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        read = (m + n) * k + _scale_bytes(m, k, case["a_scales"]) + _scale_bytes(n, k, case["b_scales"])
        return {"bytes": read + m * n * SIZE[case["out"]] * (2 if case["add"] else 1), "flops": 2 * m * n * k}
    rows, cols = case["rows"], case["cols"]
    cells, wide = rows * cols, SIZE[case["type"]]
    if op == "quant":
        out = cells + _scale_bytes(rows, cols, case["scales"])
        if case["transpose"]:
            out += cells + _scale_bytes(cols, rows, case["scales"])
        return {"bytes": cells * wide + out, "flops": (4 if case["transpose"] else 2) * cells}
    more = 1 if case["residual"] else 0
    if op == "norm":
        # x and the residual in; the sum, the 8-bit values, their scales and the row's factor out
        bytes = cells * (wide * (2 + more) + 1) + _scale_bytes(rows, cols, "rows") + 4 * rows + cols * wide
        return {"bytes": bytes if more else bytes - cells * wide, "flops": 6 * cells}
    # dy, h and the residual's gradient in; dx and dweight out
    return {"bytes": cells * wide * (3 + more) + 4 * rows + cols * (wide + 4), "flops": 10 * cells}


def exact(case, seed):
    """The outputs in 64 bits: 8-bit ones before their rounding."""
    state = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        a = dequantize_exact(state["a"], state["a_scales"])
        b = dequantize_exact(state["b"], state["b_scales"])
        c = torch.mm(a, b.t())
        return c + state["add"].double() if case["add"] else c
    if op == "quant":
        x = state["x"].double()
        got = quantize_exact(x, case["scales"], case["format"])
        return got + quantize_exact(x.t(), case["scales"], case["format"]) if case["transpose"] else got
    if op == "norm":
        h = state["x"]
        if state["residual"] is not None:
            h = (h.double() + state["residual"].double()).to(h.dtype)
        wide = h.double()
        rstd = 1.0 / torch.sqrt((wide * wide).sum(1) / wide.shape[1] + EPS)
        return quantize_exact(wide * rstd[:, None] * state["weight"].double(), "rows", case["format"]) + (wide, rstd)
    dy, h, rstd, w = state["dy"].double(), state["h"].double(), state["rstd"].double(), state["weight"].double()
    along = (dy * w * h).sum(1) * rstd ** 3 / h.shape[1]
    dx = rstd[:, None] * (dy * w) - along[:, None] * h
    if state["dresidual"] is not None:
        dx = dx + state["dresidual"].double()
    return dx, torch.mv((dy * h).t(), rstd)


def _spread_scales(s, rows, cols, high):
    r = torch.arange(rows, device=s.device) // high
    c = torch.arange(cols, device=s.device) // GROUP
    return s[r][:, c]


def quantize_exact(x, scales, format):
    rows, cols = x.shape
    high = GROUP if scales == "blocks" else 1
    s = torch.zeros(-(-rows // high), -(-cols // GROUP), dtype=torch.float64, device=x.device)
    for j in range(s.shape[1]):
        most = x[:, j * GROUP:(j + 1) * GROUP].abs().amax(1)
        most = torch.cat([most, most.new_zeros(-rows % high)]).view(-1, high).amax(1)
        s[:, j] = torch.clamp(most / MAX_OF[format], min=SCALE_FLOOR)
    return x / _spread_scales(s, rows, cols, high), s


def dequantize_exact(q, s):
    high = GROUP if s.shape[0] < q.shape[0] else 1
    return q.double() * _spread_scales(s.double(), q.shape[0], q.shape[1], high)
