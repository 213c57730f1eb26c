"""What routing may call settled in 32 bits, at sums of any size: the last chosen
expert against all that is no candidate, and groups whose two best cancel.  The
choice is that of the sums in 64 bits."""
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


def _check(gpu, z, bias, topk, what, score="sigmoid", groups=1, topk_groups=1):
    """All rows' experts against the sums in 64 bits, some rows' weights too."""
    kw = dict(score=score, groups=groups, topk_groups=topk_groups, group_score="top2")
    weights, experts = gpu.route_experts(z.to(DEV), topk, bias=bias.to(DEV), **kw)
    zd = z.double().numpy()
    with np.errstate(over="ignore"):
        e = np.exp(zd - zd.max(axis=1, keepdims=True))
        s = e / e.sum(axis=1, keepdims=True) if score == "softmax" else 1 / (1 + np.exp(-zd))
    c = s + bias.double().numpy()
    order = np.argsort(-c, axis=1, kind="stable")
    if groups > 1:
        best = np.sort(c.reshape(len(c), groups, -1), axis=2)[:, :, -2:].sum(axis=2)
        dropped = np.ones((len(c), groups), bool)
        np.put_along_axis(dropped, np.argsort(-best, axis=1, kind="stable")[:, :topk_groups], False, axis=1)
        out = np.take_along_axis(dropped, order // (c.shape[1] // groups), axis=1)
        order = np.take_along_axis(order, np.argsort(out, axis=1, kind="stable"), axis=1)
    wrong = (experts.cpu().numpy() != order[:, :topk]).any(axis=1)
    assert not wrong.any(), (what, int(wrong.sum()), experts.cpu().numpy()[wrong][:2], order[wrong, :topk][:2])
    T.assert_route((weights[:20], experts[:20]), T.route(z[:20], topk, bias=bias, **kw), what)


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
        _check(gpu, z, bias, above + 1, (centre, E, score, seed), score)

def _cancelling(rows, E, groups, sizes, spread, seed):
    """Logits and a bias by which each group's two best sum to about one half; group
    g's biases are +sizes[g] and -sizes[g] and the rest of it far below."""
    rng = np.random.default_rng(seed)
    n = E // groups
    size = np.asarray(sizes, np.float64)[np.arange(groups) % len(sizes)]
    bias = np.empty((groups, n), np.float32)
    bias[:] = -2 * size[:, None] - 3
    bias[:, 0], bias[:, n - 1] = size, -size
    for g in range(groups):
        bias[g] = rng.permutation(bias[g])
    best, second = bias.argmax(axis=1), np.empty(groups, int)
    for g in range(groups):
        second[g] = np.argsort(-bias[g], kind="stable")[1]
    z = rng.standard_normal((rows, groups, n))
    s = 0.3 + 0.2 * rng.random((rows, groups))
    at = np.arange(groups)
    total = 0.9 + spread * rng.standard_normal((rows, groups))
    z[:, at, best] = np.log(s / (1 - s))
    z[:, at, second] = np.log((total - s) / (1 - total + s))
    z = z.reshape(rows, E).astype(np.float32)
    bias = bias.reshape(E)
    c = 1 / (1 + np.exp(-z.astype(np.float64))) + bias.astype(np.float64)
    v = np.sort(np.sort(c.reshape(rows, groups, n), axis=2)[:, :, -2:].sum(axis=2), axis=1)
    clear = np.diff(v, axis=1).min(axis=1) > 1e-15 * max(sizes) + 1e-14
    assert clear.mean() > 0.9
    return torch.from_numpy(z[clear]), torch.from_numpy(bias)


@pytest.mark.parametrize("sizes,spread", [((0.3,), 2e-7), ((8.0,), 1e-6), ((100.0,), 3e-6), ((30.0, 90.0), 3e-6),
                                          ((0.1, 1e3, 0.1, 1e5), 3e-3), ((1e5, 0.2), 3e-3), ((1e5, 1e5, 0.2, 0.2), 1e-3)])
@pytest.mark.parametrize("E,groups,rows", [(8, 4, 4000), (64, 8, 1500), (64, 8, 3000), (256, 8, 3000), (256, 8, 5500),
                                           (60, 5, 3000), (250, 10, 5500), (1000, 20, 2000)])
def test_two_best_that_cancel(gpu, sizes, spread, E, groups, rows):
    z, bias = _cancelling(rows, E, groups, sizes, spread, E + groups)
    for keep in sorted({1, groups // 2, groups - 1}):
        # One choice need not tell the groups apart; as many as two of each kept group do.
        for topk in (1, 2 * keep):
            _check(gpu, z, bias, topk, (sizes, E, keep, topk), groups=groups, topk_groups=keep)


@pytest.mark.parametrize("rows", [5, 5000])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_two_best_past_the_largest_fp32(gpu, rows, score):
    """Sums of two that fp32 cannot hold, of either sign, next to groups of -infinity."""
    z = torch.randn(rows, 32, generator=torch.Generator().manual_seed(rows))
    for sign in (1.0, -1.0):
        bias = torch.full((8, 4), -3.4e38)
        for g, (best, second) in enumerate(((2.0, 1.9), (2.1, 1.9), (2.0, 1.8), (1.9, 1.9), (2.2, 1.7), (1.8, 1.8))):
            bias[g, 1], bias[g, 3] = sign * best * 1e38, sign * second * 1e38
        bias[6] = -float("inf")
        bias[7, 1:] = -float("inf")
        bias = bias.view(32)
        for keep in (1, 2, 3, 5, 6, 7):
            _check(gpu, z, bias, 2, (sign, keep), score, 8, keep)
