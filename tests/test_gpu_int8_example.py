"""The mixture-of-experts example runs and stays near the block in 64 bits.

An int8 code is off by at most half a step, a step being a row's largest
magnitude over 127: for normal rows, whose largest of about 1000 is near 3.3
deviations, 0.5/sqrt(3) * 3.3/127 = 0.75% of the deviation in the root mean
square.  Four quantised operands (activations and weights, twice) add up as
squares to 1.5% of the expert output, which the second norm scales to its gate's
share of the residual; the last projection's two operands add 1.1%.  bf16 adds
0.4% at most at each of five roundings.  3% holds all of it."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("tokens", [1, 64, 777])
def test_example(gpu, tokens):
    spec = importlib.util.spec_from_file_location("int8_moe_block", os.path.join(ROOT, "examples", "int8_moe_block.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    block = ex.Int8MoEBlock()
    g = torch.Generator(device="cuda").manual_seed(tokens)
    x, res = (torch.randn(tokens, 1024, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    r, out, expert = block(x, res)
    want_r, want = block.reference(x, res, expert)
    for got, ref in ((r, want_r), (out, want)):
        assert got.shape == ref.shape and bool(got.isfinite().all())
        assert float((got.double() - ref).norm() / ref.norm()) < 0.03
