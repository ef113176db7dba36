"""The feed-forward operators in 16 bits as a user's program calls them, and their plain forms.

Four operators that belong together, the two products of a feed-forward block with all that stands around them:

* ``linear``: y = act(x W^T + bias) + residual, from one token to a training batch, and what the backward pass needs of
  it (the values before the activation), kept in the inputs' type or in 8 bits;
* ``linear_backward``: the gradients of x, W and the bias from either;
* ``gated``: h = act(x Wg^T) * (x Wu^T), both products in one kernel, and both kept in either way;
* ``gated_backward``: the gradients of x and both weights, and h once more for the product behind it.

Each case is measured as a user's call makes it (``own`` true) and as elementary torch operations in 32 bits
(``own`` false).
"""
import math

import torch

own = False

GROUP = 128                      # values of a row that share a scale where they are kept in 8 bits
SCALE_FLOOR = 2.0 ** -64         # the least scale
FMAX = 448.0                     # the largest value of E4M3
REAL = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"f16": 2, "bf16": 2, "f32": 4}
ACTIVATIONS = ["relu", "gelu", "gelu_tanh", "silu", "sigmoid"]


def listed():
    return [
        # one token through a square projection with its residual: the latency of single-token decoding
        linear("token_4096", 1, 4096, 4096, "bf16", bias=True, residual=True),
        # a prompt of ragged sizes through an activated projection
        linear("prompt_1000_ragged", 1000, 776, 2056, "f16", "gelu", bias=True, residual=True),
        # the forward product of a training step (the repository's 8192 x 8192 x 4096 workload)
        linear("forward_8192", 8192, 8192, 4096, "bf16", "gelu_tanh", bias=True),
        # a training step that keeps the values before the activation in 8 bits
        linear("forward_kept_8_bits", 4096, 8192, 2056, "bf16", "gelu", bias=True, keep="fp8"),
        # gradients of a square projection without an activation; the weight's in 32 bits, added to the one that is there
        linear_back("gradient_4096", 4096, 4096, 4096, "bf16", out="f32", add=True),
        # gradients of an activated projection for a short ragged batch
        linear_back("gradient_ragged", 200, 2056, 776, "f16", "gelu", keep="real", bias=True),
        # both projections of a gated block for one token
        gated("gated_token", 1, 8192, 4096, "bf16"),
        # and for a batch of sequences decoded together: the weights' bytes bound it
        gated("gated_decode_48", 48, 8192, 8192, "bf16"),
        # a short prompt of ragged sizes, kept as it is
        gated("gated_ragged", 333, 1000, 776, "f16", "gelu_tanh", keep="real"),
        # a training batch, kept in 8 bits
        gated("gated_forward_4096", 4096, 8192, 4096, "bf16", keep="fp8"),
        # its gradients from what was kept in 8 bits, with the product for the projection behind it
        gated_back("gated_gradient_4096", 4096, 8192, 4096, "bf16", keep="fp8", product=True),
        # gradients of the short ragged batch
        gated_back("gated_gradient_ragged", 333, 1000, 776, "f16", "gelu_tanh", keep="real"),
    ]


def linear(name, m, n, k, type, act="none", bias=False, residual=False, keep="none", tight=False):
    return dict(name=name, op="linear", m=m, n=n, k=k, type=type, act=act, bias=bias, residual=residual, keep=keep,
                tight=tight)


def linear_back(name, m, n, k, type, act="none", keep="none", bias=False, out="", add=False, tight=False):
    return dict(name=name, op="linear_back", m=m, n=n, k=k, type=type, act=act, keep=keep, bias=bias, out=out or type,
                add=add, tight=tight)


def gated(name, m, n, k, type, act="silu", keep="none", tight=False):
    return dict(name=name, op="gated", m=m, n=n, k=k, type=type, act=act, keep=keep, tight=tight)


def gated_back(name, m, n, k, type, act="silu", keep="real", product=False, tight=False):
    return dict(name=name, op="gated_back", m=m, n=n, k=k, type=type, act=act, keep=keep, product=product, tight=tight)


def draw(rng):
    """One more case: sizes spread over the logarithm, as odd as they come; rows on 16-byte boundaries in most, and
    as tight as they are in some."""
    def size(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return max(lo, min(hi, v))

    op = rng.choice(["linear", "linear", "linear_back", "gated", "gated", "gated_back"])
    type = rng.choice(["f16", "bf16", "bf16"])
    m, n, k = size(1, 8192), size(64, 8192), size(64, 8192)
    products = {"linear": 1, "linear_back": 2, "gated": 2, "gated_back": 4}[op]
    most = 2 * 4096 * 8192 * 4096 // products
    if m * n * k > most:
        m = max(1, most // (n * k))
    tight = rng.random() < 0.2
    act = rng.choice(ACTIVATIONS)
    if op == "linear":
        act = rng.choice([act, act, "none"])
        keep = rng.choice(["none", "none", "real", "fp8"]) if act != "none" else "none"
        case = linear("", m, n, k, type, act, rng.random() < 0.6, rng.random() < 0.4, keep, tight)
    elif op == "linear_back":
        if rng.random() < 0.5:
            case = linear_back("", m, n, k, type, bias=rng.random() < 0.5, out=rng.choice([type, "f32"]),
                               add=rng.random() < 0.5, tight=tight)
        else:
            case = linear_back("", m, n, k, type, act, rng.choice(["real", "fp8"]), rng.random() < 0.5, tight=tight)
    elif op == "gated":
        case = gated("", m, n, k, type, act, rng.choice(["none", "none", "real", "fp8"]), tight)
    else:
        case = gated_back("", m, n, k, type, act, rng.choice(["real", "fp8"]), rng.random() < 0.5, tight)
    del case["name"]
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _rows(x, tight, align=8):
    """`x` with rows that begin on 16-byte boundaries, as a program lays its buffers out once; `tight`: without a gap."""
    rows, cols = x.shape
    ld = -(-cols // align) * align
    if ld == cols or tight:
        return x.contiguous()
    wide = torch.zeros(rows, ld, dtype=x.dtype, device=x.device)
    wide[:, :cols].copy_(x)
    return wide[:, :cols]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    m, n, k, type, tight = case["m"], case["n"], case["k"], REAL[case["type"]], case["tight"]

    def normal(rows, cols, spread=1.0):
        return torch.randn(rows, cols, generator=g, device="cuda").mul_(spread)

    def tokens(cols, spread):
        """Normal values, each row at its own level; a row of zeros where a token only pads the batch."""
        x = normal(m, cols, spread).mul_(torch.exp(0.3 * normal(m, 1)))
        if m > 8:
            x[m // 3] = 0.0
        return _rows(x.to(type), tight)

    def weight():
        return _rows(normal(n, k, 1.3 / math.sqrt(k)).to(type), tight)

    def kept():
        """Values before an activation, as the forward pass leaves them."""
        z = normal(m, n, 1.3)
        if case["keep"] == "real":
            return (_rows(z.to(type), False),)
        data, scales = quantize_plain(z)
        wide = torch.zeros(m, -(-n // 16) * 16, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
        wide[:, :n].copy_(data)
        return wide[:, :n], scales.t().contiguous().t()

    state = {"case": case, "x": tokens(k, 1.0)}
    op = case["op"]
    if op in ("linear", "linear_back"):
        state["weight"] = weight()
        if op == "linear":
            state["bias"] = normal(1, n, 0.3)[0].to(type) if case["bias"] else None
            state["residual"] = tokens(n, 3.0) if case["residual"] else None
        else:
            state["dy"] = tokens(n, 0.05)
            state["kept"] = kept() if case["act"] != "none" else None
            state["add"] = normal(n, k, 0.5).to(REAL[case["out"]]) if case["add"] else None
        return state
    state["gate"], state["up"] = weight(), weight()
    if op == "gated_back":
        state["dh"] = tokens(n, 0.05)
        state["kept"] = kept() + kept()
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
    act = None if case["act"] == "none" else case["act"]
    keep = None if case["keep"] == "none" else case["keep"]
    if op == "linear":
        return gp.linear(state["x"], state["weight"], state["bias"], activation=act, residual=state["residual"], keep=keep)
    if op == "linear_back":
        return gp.linear_backward(state["dy"], state["x"], state["weight"], activation=act, kept=state["kept"],
                                  bias_grad=case["bias"], out_dtype=REAL[case["out"]], addend=state["add"])
    if op == "gated":
        return gp.gated(state["x"], state["gate"], state["up"], activation=act, keep=keep)
    return gp.gated_backward(state["dh"], state["x"], state["gate"], state["up"], state["kept"], activation=act,
                             product=case["product"])


def _run_plain(state):
    case = state["case"]
    op = case["op"]
    act, keep, type = case["act"], case["keep"], state["x"].dtype
    x = state["x"].float()
    if op == "linear":
        z = x @ state["weight"].float().t()
        if state["bias"] is not None:
            z += state["bias"].float()
        y = activate(z, act)
        if state["residual"] is not None:
            y = y + state["residual"].float()
        y = y.to(type)
        return (y, keep_plain(z, keep, type)) if keep != "none" else y
    if op == "linear_back":
        dz = state["dy"].float()
        if act != "none":
            dz = dz * slope(held(state["kept"]), act)
        dx = dz @ state["weight"].float()
        dw = dz.t() @ x
        if state["add"] is not None:
            dw += state["add"].float()
        return dx.to(type), dw.to(REAL[case["out"]]), dz.sum(0) if case["bias"] else None
    if op == "gated":
        gate, up = x @ state["gate"].float().t(), x @ state["up"].float().t()
        h = (activate(gate, act) * up).to(type)
        return (h, keep_plain(gate, keep, type) + keep_plain(up, keep, type)) if keep != "none" else h
    half = len(state["kept"]) // 2
    gate, up, dh = held(state["kept"][:half]), held(state["kept"][half:]), state["dh"].float()
    a = activate(gate, act)
    dgate, dup = dh * up * slope(gate, act), dh * a
    dx = dgate @ state["gate"].float() + dup @ state["up"].float()
    got = dx.to(type), (dgate.t() @ x).to(type), (dup.t() @ x).to(type)
    return got + ((a * up).to(type),) if case["product"] else got


def activate(z, act):
    if act == "none":
        return z
    if act == "relu":
        return z.clamp(min=0.0)
    if act == "gelu":
        return z * 0.5 * torch.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    s = 1.0 / (1.0 + torch.exp(-z))
    return s if act == "sigmoid" else z * s


def slope(z, act):
    """The activation's derivative."""
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        s = 1.0 / (1.0 + torch.exp(-c * (z + 0.044715 * z * z * z)))
        return s + z * s * (1.0 - s) * c * (1.0 + 3 * 0.044715 * z * z)
    s = 1.0 / (1.0 + torch.exp(-z))
    return s * (1.0 - s) if act == "sigmoid" else s * (1.0 + z * (1.0 - s))


def _groups(x):
    """`x` padded with zeros and seen as [rows, groups along the row, 128]."""
    return torch.nn.functional.pad(x, (0, -x.shape[1] % GROUP)).view(x.shape[0], -1, GROUP)


def quantize_plain(x):
    """(8-bit values, scales) of a 32-bit matrix: scale = max|x| / 448 over each row's 128 values."""
    wide = _groups(x)
    s = (wide.abs().amax(2) / FMAX).clamp(min=SCALE_FLOOR)
    q = (wide * (1.0 / s)[:, :, None]).to(torch.float8_e4m3fn)
    return q.view(x.shape[0], -1)[:, :x.shape[1]], s


def keep_plain(z, keep, type):
    return (z.to(type),) if keep == "real" else quantize_plain(z)


def held(kept):
    """The values that were kept, in 32 bits."""
    if len(kept) == 1:
        return kept[0].float()
    data, scales = kept
    return data.float() * scales.repeat_interleave(GROUP, 1)[:, :data.shape[1]]


# ---------------------------------------------------------------------------
# what a pass cannot do without, and what it has to give
# ---------------------------------------------------------------------------
def work(case):
    m, n, k, op = case["m"], case["n"], case["k"], case["op"]
    wide = SIZE[case["type"]]
    z = {"none": 0, "real": m * n * wide, "fp8": m * n + 4 * m * -(-n // GROUP)}[case["keep"]]
    if op == "linear":
        values = m * k + n * k + (n if case["bias"] else 0) + m * n * (2 if case["residual"] else 1)
        return {"bytes": values * wide + z, "flops": 2 * m * n * k}
    if op == "gated":
        return {"bytes": (m * k + 2 * n * k + m * n) * wide + 2 * z, "flops": 4 * m * n * k}
    if op == "linear_back":
        dw = n * k * SIZE[case["out"]] * (2 if case["add"] else 1)
        return {"bytes": (m * n + 2 * m * k + n * k) * wide + z + dw + (4 * n if case["bias"] else 0), "flops": 4 * m * n * k}
    values = m * n * (2 if case["product"] else 1) + 2 * m * k + 4 * n * k
    return {"bytes": values * wide + 2 * z, "flops": 8 * m * n * k}


def exact(case, seed):
    """The outputs in 64 bits: 8-bit ones before their rounding."""
    state = prepare(case, seed)
    op, act, keep = case["op"], case["act"], case["keep"]
    x = state["x"].double()

    def product(a, b):
        return torch.einsum("mk,nk->mn", a, b.double())

    if op == "linear":
        z = product(x, state["weight"])
        if state["bias"] is not None:
            z = z + state["bias"].double()[None, :]
        y = value_exact(z, act)
        if state["residual"] is not None:
            y = state["residual"].double() + y
        return (y, keep_exact(z, keep)) if keep != "none" else y
    if op == "gated":
        gate, up = product(x, state["gate"]), product(x, state["up"])
        h = up * value_exact(gate, act)
        return (h, keep_exact(gate, keep) + keep_exact(up, keep)) if keep != "none" else h
    if op == "linear_back":
        dz = state["dy"].double()
        if act != "none":
            dz = slope_exact(held_exact(state["kept"]), act) * dz
        dx = torch.einsum("mn,nk->mk", dz, state["weight"].double())
        dw = torch.einsum("mn,mk->nk", dz, x)
        if state["add"] is not None:
            dw = state["add"].double() + dw
        return dx, dw, torch.einsum("mn->n", dz) if case["bias"] else None
    half = len(state["kept"]) // 2
    gate, up, dh = held_exact(state["kept"][:half]), held_exact(state["kept"][half:]), state["dh"].double()
    h = up * value_exact(gate, act)
    dgate, dup = slope_exact(gate, act) * up * dh, value_exact(gate, act) * dh
    both = torch.cat([dgate, dup], 1)
    dx = torch.einsum("mn,nk->mk", both, torch.cat([state["gate"], state["up"]], 0).double())
    dw = torch.einsum("mn,mk->nk", both, x)
    got = dx, dw[:case["n"]], dw[case["n"]:]
    return got + (h,) if case["product"] else got


def _phi(z):
    """The normal distribution's integral up to z."""
    return torch.special.ndtr(z)


def _inner(z):
    return math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3)


def value_exact(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return z * _phi(z)
    if act == "gelu_tanh":
        return z * torch.special.expit(2.0 * _inner(z))
    return torch.special.expit(z) if act == "sigmoid" else z * torch.special.expit(z)


def slope_exact(z, act):
    if act == "relu":
        return torch.where(z > 0, torch.ones_like(z), torch.zeros_like(z))
    if act == "gelu":
        return _phi(z) + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        t = torch.tanh(_inner(z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * math.sqrt(2.0 / math.pi) * (1.0 + 3.0 * 0.044715 * z ** 2)
    s = torch.special.expit(z)
    return s * torch.special.expit(-z) if act == "sigmoid" else s + z * s * torch.special.expit(-z)


def keep_exact(z, keep):
    if keep == "real":
        return (z,)
    rows, cols = z.shape
    s = torch.stack([z[:, j:j + GROUP].abs().max(1).values for j in range(0, cols, GROUP)], 1)
    s = torch.clamp(s / FMAX, min=SCALE_FLOOR)
    at = torch.arange(cols, device=z.device) // GROUP
    return z / s[:, at], s


def held_exact(kept):
    if len(kept) == 1:
        return kept[0].double()
    data, scales = kept
    at = torch.arange(data.shape[1], device=data.device) // GROUP
    return data.double() * scales.double()[:, at]
