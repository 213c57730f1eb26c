"""The README's 8-bit-integer example runs as written, after the one before it
whose names it uses."""
import os
import re

import pytest
import torch

from tests import _int8 as T

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_int8_example(gpu):
    text = open(os.path.join(ROOT, "README.md")).read()
    blocks = re.findall(r"```python\n(.*?)```", text, re.S)
    torch.manual_seed(0)
    env = {}
    for code in blocks[:2]:
        exec(compile(code, "README.md", "exec"), env)
    torch.cuda.synchronize()
    d = {"A": env["q"].cpu(), "a_s": env["s"].cpu(), "B": env["w8"].cpu(), "b_s": env["w_s"].cpu(), "bias": None}
    T.assert_gemm(env["C8"], d, "bf16")
    assert torch.equal(env["Cg8"], env["C8"])       # both experts hold the same weight
