"""The README's example of routing, dispatch, combine and adapters runs as
written, after the two before it whose names it uses."""
import os
import re

import pytest
import torch

from tests import _tokens as T

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_tokens_example(gpu):
    text = open(os.path.join(ROOT, "README.md")).read()
    blocks = re.findall(r"```python\n(.*?)```", text, re.S)
    torch.manual_seed(0)
    env = {}
    for code in blocks[:3]:
        exec(compile(code, "README.md", "exec"), env)
    torch.cuda.synchronize()
    c = {k: v.cpu() for k, v in env.items() if torch.is_tensor(v)}
    T.assert_route((c["weights"], c["experts"]), T.route(c["logits"], 1, "sigmoid", scale=2.5))
    rows, rows_s, offsets, slots = T.dispatch(c["experts"], 2, c["q"], c["s"])
    assert torch.equal(c["rows"], rows) and torch.equal(c["rows_s"], rows_s)
    assert torch.equal(c["offsets"], offsets) and torch.equal(c["slots"], slots)
    # both experts hold the shared projection's weight, so each token's row is that of C8
    assert torch.equal(c["y8"][c["slots"][:, 0].long()], c["C8"])
    ref, tol = T.combine(c["y8"], c["slots"], c["weights"], c["C8"])
    T.assert_close(c["h8"], ref, tol, "bf16")
    ref, tol, rms = T.adapters(c["C8"], c["x"], c["Al"], c["Bl"], c["ids"])
    T.assert_close(c["Cl"], ref, tol, "bf16", "adapters", rms)
