"""The example of the 8-bit operators together: a block's forward and backward
pass close to float64, its loss falling, its tokens one by one as together."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,width", [(300, 512), (130, 648)])
def test_block_trains_and_decodes(tokens, width):
    spec = importlib.util.spec_from_file_location("fp8_block", os.path.join(ROOT, "examples", "fp8_block.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, far, apart = example.run(tokens, width, steps=12)
    # a code of E4M3 is within 2^-4 of its value and uniform inside that (2^-4 / sqrt(3) = 0.036 root mean square at
    # most), one of E5M2 within 2^-3 (0.072); a product's relative error is at most the two operands' together, and
    # each output below has one product in it, the norm's gradient after it
    e4m3, e5m2 = 2.0 ** -4 / 3 ** 0.5, 2.0 ** -3 / 3 ** 0.5
    out, dx, dW, dg = far
    assert out < 2 * e4m3
    assert dx < e4m3 + e5m2 and dW < e4m3 + e5m2 and dg < e4m3 + e5m2
    assert all(b < a for a, b in zip(losses, losses[1:]))
    # the same codes and scales; only the tiling, and with it the order of FP32 sums, may differ: BF16 outputs
    assert apart < 2.0 ** -8
