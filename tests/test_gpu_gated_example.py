"""The example of the feed-forward operators together: a gated block's forward
and backward pass close to float64, its steps, its tokens one by one as together."""
import importlib.util
import math
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,width,inner", [(300, 512, 1024), (130, 328, 760)])
def test_block_trains_and_decodes(tokens, width, inner):
    spec = importlib.util.spec_from_file_location("gated_block", os.path.join(ROOT, "examples", "gated_block.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, far, apart = example.run(tokens, width, inner, steps=5)
    # forward: h and out are rounded to BF16 once each, 2^-8 of their values at most
    # backward: a code of E4M3 is within 2^-4 of its value and uniform inside that (2^-4 / sqrt(3) root mean square at
    # most); the products' gradients and h each have u, and silu or its slope of g, as factors, which move by at most 1.1
    # times that (the largest slope of silu, against values no smaller), and are rounded to BF16
    bf16, e4m3 = 2.0 ** -8, 2.0 ** -4 / 3 ** 0.5
    out, dx, dWg, dWu, dWd = far
    assert out < 2 * bf16
    assert max(dx, dWg, dWu, dWd) < 2.2 * e4m3 + 3 * bf16
    assert len(losses) == 5 and all(math.isfinite(v) for v in losses)
    # only the tiling, and with it the order of FP32 sums, may differ: BF16 values
    assert apart < 2 * bf16
