"""Rows that leave lanes of a wave without a column, with more choices than lanes
that have one: each choice's slot and weight is held by a lane of its own."""
import pytest
import torch

from tests import _tokens as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp32"), ("fp32", "fp32"), ("fp32", "bf16")])
@pytest.mark.parametrize("D", [1, 3, 4, 9, 33, 65, 129, 200, 256, 257, 264, 505, 511, 512, 513, 521, 1025, 2049, 2056, 4099])
@pytest.mark.parametrize("topk", [9, 33, 63, 64])
def test_choices_past_the_lanes_with_columns(gpu, dtype, out, D, topk):
    tokens = 7
    g = torch.Generator().manual_seed(D + topk)
    rows = torch.randn(tokens * topk, D, generator=g).to(T.DTYPES[dtype])
    slots = torch.randperm(tokens * topk, generator=g).view(tokens, topk).to(torch.int32)
    weights = torch.randn(tokens, topk, generator=g)
    base = torch.randn(tokens, D, generator=g).to(T.DTYPES[out])
    ref, tol = T.combine(rows, slots, weights, base)
    buf = torch.full((tokens + 2, D + 40), 3.0, dtype=T.DTYPES[out], device=DEV)
    view = buf[1:-1, 20:D + 20]
    view.copy_(base)
    gpu.combine_experts(rows.to(DEV), slots.to(DEV), weights.to(DEV), base=view, out=view)
    T.assert_close(view, ref, tol, out, (dtype, out, D, topk))
    assert bool((buf[[0, -1]] == 3).all()) and bool((buf[:, :20] == 3).all()) and bool((buf[:, D + 20:] == 3).all())
