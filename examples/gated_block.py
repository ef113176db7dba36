"""A gated feed-forward block in bfloat16, trained and then run token by token.

    h   = silu(x Wg^T) * (x Wu^T)       one kernel; both products kept in 8 bits
    out = h Wd^T + x                    the residual in the product's epilogue

Training keeps the weights in float32 beside their bfloat16 copies, and adds
their gradients up in float32.  Between the passes a token costs two bytes for
each of the block's inner values (g and u in 8 bits); h is worked out again where
the last weight's gradient needs it.  Decoding is the same two calls on one row.

    python examples/gated_block.py [--tokens 512] [--width 1024] [--inner 2048] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import software_pipelined_tiled_pipeline_gb300 as gp  # noqa: E402

BF16 = torch.bfloat16


class Block:
    """The block's weights in float32, their gradients, and their copies in bfloat16."""

    def __init__(self, width, inner, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        sizes = ((inner, width), (inner, width), (width, inner))
        self.master = [torch.randn(n, k, generator=g, device="cuda") * k ** -0.5 for n, k in sizes]
        self.grad = [torch.zeros_like(w) for w in self.master]
        self.copy()

    def copy(self):
        self.gate, self.up, self.down = (w.to(BF16) for w in self.master)

    def forward(self, x):
        """out, and what the backward pass needs beside x."""
        h, kept = gp.gated(x, self.gate, self.up, keep="fp8")
        return gp.linear(h, self.down, residual=x), kept

    def backward(self, dout, x, kept):
        """The gradient of x, adding to those of the weights."""
        dh, _, _ = gp.linear_backward(dout, None, self.down, weight_grad=False)
        both = self.grad[:2]
        dx, _, _, h = gp.gated_backward(dh, x, self.gate, self.up, kept, product=True, addend=both, out=both)
        gp.linear_backward(dout, h, self.down, input_grad=False, addend=self.grad[2], out=self.grad[2])
        return dx + dout                       # dout also reaches x past the block

    def step(self, rate):
        for w, g in zip(self.master, self.grad):
            w -= rate * g
            g.zero_()
        self.copy()

    def token(self, x):
        """One token (or a few): what a decoding loop calls."""
        return gp.linear(gp.gated(x, self.gate, self.up), self.down, residual=x)


def reference(block, x, dout):
    """out, dx and the weights' gradients of the same block in float64."""
    x, d, (wg, wu, wd) = x.double(), dout.double(), [w.double() for w in (block.gate, block.up, block.down)]
    g, u = x @ wg.t(), x @ wu.t()
    s = torch.sigmoid(g)
    a = g * s
    dh = d @ wd
    dg, du = dh * u * (s + a * (1 - s)), dh * a
    return (a * u) @ wd.t() + x, dg @ wg + du @ wu + d, dg.t() @ x, du.t() @ x, d.t() @ (a * u)


def distance(a, b):
    return float((a.double() - b).norm() / b.norm())


def run(tokens=512, width=1024, inner=2048, steps=20, rate=0.02):
    """How far one pass is from float64, the losses of some steps towards a fixed target, and how far tokens one by one
    are from the batch."""
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(BF16)

    block = Block(width, inner)
    x, dout, target = normal(tokens, width), normal(tokens, width), normal(tokens, width)
    out, kept = block.forward(x)
    dx = block.backward(dout, x, kept)
    far = [distance(a, b) for a, b in zip([out, dx] + block.grad, reference(block, x, dout))]
    for grad in block.grad:
        grad.zero_()
    losses = []
    for _ in range(steps):
        out, kept = block.forward(x)
        error = out.float() - target.float()
        losses.append(float(error.square().mean()))
        block.backward((error / tokens).to(BF16), x, kept)
        block.step(rate)
    whole, _ = block.forward(x[:8])
    alone = torch.cat([block.token(x[i:i + 1]) for i in range(8)])
    return losses, far, distance(alone, whole.double())


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=2048)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    losses, far, apart = run(a.tokens, a.width, a.inner, a.steps)
    print("against float64: out %.4f  dx %.4f  dWg %.4f  dWu %.4f  dWd %.4f" % tuple(far))
    print("loss %.4f -> %.4f in %d steps" % (losses[0], losses[-1], len(losses)))
    print("eight tokens one by one against together: %.1e" % apart)


if __name__ == "__main__":
    main()
