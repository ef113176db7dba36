"""A residual block with 8-bit products, trained and then run token by token.

    h = x + residual
    y = norm(h) * g            RMS norm, straight to 8 bits
    z = y W^T                  8-bit product
    out = h + z                (the next block's residual stream)

Training keeps W in float32 and quantises it after each step, in 128 x 128
blocks and both ways round; the backward pass is three more 8-bit products and
the norm's gradient.  Decoding is the same two calls on one row.

    python examples/fp8_block.py [--tokens 512] [--width 1024] [--steps 20]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import software_pipelined_tiled_pipeline_gb300 as gp  # noqa: E402


class Block:
    """One block: its parameters in float32, and W in 8 bits as it stands and transposed."""

    def __init__(self, width, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.W = torch.randn(width, width, generator=g, device="cuda") * width ** -0.5
        self.g = torch.ones(width, device="cuda")
        self.dW = torch.zeros_like(self.W)
        self.quantise()

    def quantise(self):
        """After each change of W: its blocks for z = y W^T and, transposed, for dy = dz W."""
        self.w, self.w_s, self.wt, self.wt_s = gp.quantize_fp8(self.W, "blocks", transpose=True)

    def forward(self, x, residual):
        """out, and what the backward pass needs (y itself in 16 bits, for W's gradient)."""
        q, s, h, rstd, y = gp.rmsnorm_fp8(x, self.g, residual, normed=True)
        out = gp.gemm_fp8(q, s, self.w, self.w_s, out_dtype=x.dtype, addend=h)
        return out, (h, rstd, y)

    def backward(self, dout, saved):
        """Gradient of x and of the residual (the same), adding to dW; the gradient of g."""
        h, rstd, y = saved
        # dout along its rows for dy, and along its columns (over tokens) for dW; y over tokens too
        d, d_s, dt, dt_s = gp.quantize_fp8(dout, "rows", format="e5m2", transpose=True)
        yt, yt_s = gp.quantize_fp8(y, "rows", transpose="only")
        dy = gp.gemm_fp8(d, d_s, self.wt, self.wt_s, out_dtype=dout.dtype)
        gp.gemm_fp8(dt, dt_s, yt, yt_s, out=self.dW, addend=self.dW)
        return gp.rmsnorm_backward(dy, h, self.g, rstd, dout)      # dout also reaches h past the norm

    def step(self, dg, rate):
        self.W -= rate * self.dW
        self.g -= rate * dg
        self.dW.zero_()
        self.quantise()

    def token(self, x, residual):
        """One token (or a few): what a decoding loop calls."""
        q, s, h, _ = gp.rmsnorm_fp8(x, self.g, residual)
        return gp.gemm_fp8(q, s, self.w, self.w_s, out_dtype=x.dtype, addend=h)


def reference(block, x, residual, dout):
    """out, dx, dW and dg of the same block in float64, W unquantised."""
    h = x.double() + residual.double()
    rstd = torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6)
    y = h * rstd * block.g.double()
    out = h + y @ block.W.double().t()
    d = dout.double()
    dy = d @ block.W.double()
    scaled = dy * block.g.double()
    dx = rstd * (scaled - h * rstd * (scaled * h * rstd).mean(1, keepdim=True)) + d
    return out, dx, d.t() @ y, (dy * h * rstd).sum(0)


def distance(a, b):
    return float((a.double() - b).norm() / b.norm())


def run(tokens=512, width=1024, steps=20, rate=None):
    """Trains the block towards a fixed target, then decodes; returns the losses and how far one pass is from float64."""
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    if rate is None:
        # descent is stable below 2 / (the largest eigenvalue of y^T y / tokens), which for normal y is near this square
        rate = 1.0 / (1.0 + (width / tokens) ** 0.5) ** 2
    block = Block(width)
    x, residual, dout = normal(tokens, width), normal(tokens, width), normal(tokens, width)
    out, saved = block.forward(x, residual)
    dx, dg = block.backward(dout, saved)
    far = [distance(a, b) for a, b in zip((out, dx, block.dW, dg), reference(block, x, residual, dout))]
    block.dW.zero_()

    target = normal(tokens, width)
    losses = []
    for _ in range(steps):
        out, saved = block.forward(x, residual)
        error = out.float() - target.float()
        losses.append(float(error.square().mean()))
        dx, dg = block.backward((error / tokens).to(torch.bfloat16), saved)
        block.step(dg, rate)

    whole, _ = block.forward(x[:8], residual[:8])
    alone = torch.cat([block.token(x[i:i + 1], residual[i:i + 1]) for i in range(8)])
    return losses, far, distance(alone, whole.double())


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    losses, far, apart = run(a.tokens, a.width, a.steps)
    print("against float64 with W unquantised: out %.3f  dx %.3f  dW %.3f  dg %.3f" % tuple(far))
    print("loss %.4f -> %.4f in %d steps" % (losses[0], losses[-1], len(losses)))
    print("eight tokens one by one against together: %.1e" % apart)


if __name__ == "__main__":
    main()
