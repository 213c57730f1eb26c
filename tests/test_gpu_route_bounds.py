"""What routing may call settled in 32 bits, at sums of any size: the last chosen
expert against all that is no candidate.  The choice is that of the sums in 64
bits."""
import numpy as np
import pytest
import torch

from tests import _tokens as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _ordered(v):
    b = np.float32(v).view(np.int32)
    return int(b) ^ ((int(b) >> 31) & 0x7fffffff)


def _value(k):
    return float(np.int32(k ^ ((k >> 31) & 0x7fffffff)).view(np.float32))


def _near_one_border(rows, E, place, centre, width, above, score, seed):
    """(logits, bias, c): per row, `above` experts far above; then, of fp32's numbers
    in runs of `place` (what a comparison that keeps an expert's place in the last
    bits tells apart), one whose sum is next to the border between the last number
    of a run and the first of the next one, another there too, and between them in
    order of their places one in the middle of the run."""
    rng = np.random.default_rng(seed)
    run = _ordered(centre) & ~(place - 1)
    border = (_value(run + place - 1) + _value(run + place)) / 2
    first, last, middle = (rng.permutation(E // place)[:3] * place).tolist()
    if seed % 2:
        first, last = last, first
    last += place - 1
    c = np.full((rows, E), centre - 5.0)
    c[:, first] = border + width * rng.standard_normal(rows)
    c[:, last] = border + width * rng.standard_normal(rows)
    c[:, middle] = _value(run + 1)
    others = [e for e in range(E) if e not in (first, last, middle)][:above]
    c[:, others] = centre + 1 + 0.1 * np.arange(above)
    top = 1e-3 if score == "softmax" else 0.5
    s = np.full(E, top)
    s[[first, last, middle]] = top * (0.7 + 0.6 * rng.random(3))
    bias = (c[0] - s).astype(np.float32)
    near = [first, last, middle]
    want = c[:, near] - bias[near].astype(np.float64)
    z = np.zeros((rows, E))
    if score == "softmax":  # the others' logits are zeros
        total = (E - 3) / (1 - want.sum(axis=1, keepdims=True))
        z[:, near] = np.log(want * total)
    else:
        z[:, near] = np.log(want / (1 - want))
    z = z.astype(np.float32)
    zd = z.astype(np.float64)
    e = np.exp(zd - zd.max(axis=1, keepdims=True))
    got = (e / e.sum(axis=1, keepdims=True) if score == "softmax" else 1 / (1 + np.exp(-zd))) + bias.astype(np.float64)
    clear = np.abs(got[:, first] - got[:, last]) > 4 * np.finfo(np.float64).eps * abs(centre)
    assert clear.mean() > 0.9
    return torch.from_numpy(z[clear]), torch.from_numpy(bias)


@pytest.mark.parametrize("centre", [0.75, 1.2, 16.5, 70.0, 1000.0, -1.2, -16.5, -70.0])
@pytest.mark.parametrize("E,place,rows", [(256, 4, 4000), (256, 16, 6000), (1024, 16, 3000), (48, 4, 4000)])
@pytest.mark.parametrize("score,width", [("sigmoid", 4e-8), ("softmax", 2e-11)])
def test_the_last_chosen(gpu, centre, E, place, rows, score, width):
    for seed, above in ((1, 0), (2, 0), (3, 5)):
        z, bias = _near_one_border(rows, E, place, centre, width, above, score, seed)
        got = gpu.route_experts(z.to(DEV), above + 1, score=score, bias=bias.to(DEV))
        T.assert_route(got, T.route(z, above + 1, score=score, bias=bias), (centre, E, score, seed))
