"""Routing to experts on the GPU against its 64-bit form: experts equal, weights
within their roundings' bound."""
import numpy as np
import pytest
import torch

from tests import _tokens as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
CONFIGS = [dict(score="softmax"), dict(score="sigmoid"), dict(score="softmax", bias=True),
           dict(score="sigmoid", bias=True, scale=2.5), dict(score="softmax", renormalize=False),
           dict(score="sigmoid", renormalize=False, scale=0.5)]


def _logits(rows, E, dtype, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    return (spread * torch.randn(rows, E, generator=g)).to(T.DTYPES[dtype])


def _check(gpu, logits, topk, pad=0, what="", **kw):
    bias = kw.pop("bias", None)
    if bias is True:
        bias = 0.1 * torch.randn(logits.shape[1], generator=torch.Generator().manual_seed(5))
    mask = kw.pop("mask", None)
    wide = torch.full((logits.shape[0], logits.shape[1] + pad), float("nan"), dtype=logits.dtype, device=DEV)
    wide[:, :logits.shape[1]] = logits.to(DEV)
    got = gpu.route_experts(wide[:, :logits.shape[1]], topk, bias=None if bias is None else bias.to(DEV),
                            mask=None if mask is None else mask.to(DEV), **kw)
    T.assert_route(got, T.route(logits, topk, bias=bias, mask=mask, **kw), what)
    return got


@pytest.mark.parametrize("E", [1, 2, 7, 8, 31, 60, 64, 65, 100, 127, 128, 129, 160, 255, 256, 257, 384, 511, 512, 513,
                               1000, 1024])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_experts(gpu, E, dtype):
    for i, kw in enumerate(CONFIGS):
        for topk in sorted({1, min(2, E), min(8, E), min(64, E)}):
            _check(gpu, _logits(9, E, dtype, E + i), topk, pad=(0, 3)[i % 2], what=(E, dtype, kw, topk), **kw)


@pytest.mark.parametrize("E,groups", [(8, 2), (64, 8), (60, 4), (256, 8), (256, 64), (160, 8), (256, 4), (96, 3),
                                      (35, 7), (64, 64), (1024, 16), (1000, 8), (512, 32), (256, 2), (128, 16)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_groups(gpu, E, groups, group_score):
    for i, kw in enumerate(CONFIGS):
        for keep in sorted({1, max(1, groups // 2), groups - 1, groups}):
            topk = min(8, E // groups * keep)
            _check(gpu, _logits(7, E, ("fp32", "bf16", "fp16")[i % 3], E + keep), topk, what=(E, groups, keep, kw),
                   groups=groups, topk_groups=keep, group_score=group_score, **kw)


@pytest.mark.parametrize("rows", [1, 3, 4, 5, 17, 64, 333, 2049, 5000])
def test_rows(gpu, rows):
    for E, kw in ((256, dict(score="sigmoid", bias=True, groups=8, topk_groups=4, group_score="top2")),
                  (256, dict(score="softmax")), (60, dict(score="softmax")), (16, dict(score="sigmoid", bias=True))):
        _check(gpu, _logits(rows, E, "fp32", rows), 6, what=(rows, E), **kw)
        mask = torch.rand(rows, generator=torch.Generator().manual_seed(rows)) < 0.4
        _check(gpu, _logits(rows, E, "bf16", rows), 6, what=(rows, E, "masked"), mask=mask, **kw)


def test_all_masked(gpu):
    w, e = _check(gpu, _logits(5, 64, "bf16", 0), 4, mask=torch.ones(5, dtype=torch.bool))
    assert bool((e == -1).all()) and bool((w == 0).all())


@pytest.mark.parametrize("E", [5, 64, 200, 256, 1024])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups", [1, 5, 4])
def test_ties(gpu, E, bias, groups):
    """Few different values: the lowest of equals, among experts and groups."""
    if E % groups:
        pytest.skip("groups do not divide E")
    g = torch.Generator().manual_seed(E)
    b = torch.randint(0, 2, (E,), generator=g).float() * 0.25 if bias else None
    for score in ("softmax", "sigmoid"):
        for values in (1, 2, 5):
            z = torch.randint(0, values, (33, E), generator=g).float()
            for group_score in ("max", "top2"):
                _check(gpu, z, min(8, E // groups), score=score, bias=b, groups=groups, topk_groups=1,
                       group_score=group_score, what=(E, values))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_infinities_and_nan(gpu, score, dtype):
    inf, nan = float("inf"), float("nan")
    for E, topk in ((6, 3), (64, 8), (256, 8), (300, 8)):
        z = _logits(12, E, dtype, E)
        z[0] = -inf
        z[1, 2:] = -inf                   # fewer finite logits than topk
        z[2, 3] = nan
        z[3, 0], z[3, 1] = inf, -inf
        z[4] = nan
        z[5, E - 1] = nan
        z[6] = torch.finfo(z.dtype).min   # a mask of the type's lowest value
        z[7, 1:] = torch.finfo(z.dtype).min
        z[8, :E - 1] = -inf
        z[9] = torch.finfo(z.dtype).max
        for kw in (dict(), dict(bias=True), dict(renormalize=False)):
            _check(gpu, z, topk, score=score, what=(E, kw), **kw)
            if E % 2 == 0:
                for gs in ("max", "top2"):
                    _check(gpu, z, min(topk, E // 2), score=score, groups=2, topk_groups=1, group_score=gs, **kw)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_bias_that_is_not_finite(gpu, value):
    b = torch.zeros(64)
    b[[3, 40]] = value
    for score in ("softmax", "sigmoid"):
        _check(gpu, _logits(6, 64, "fp32", 1), 8, score=score, bias=b)
        _check(gpu, _logits(6, 64, "fp32", 1), 8, score=score, bias=b, groups=8, topk_groups=2, group_score="top2")
    if value == float("-inf"):            # more experts asked for than are left
        b[:60] = value
        _check(gpu, _logits(6, 64, "fp32", 1), 8, score="sigmoid", bias=b)


@pytest.mark.parametrize("E", [64, 256, 512])
def test_scores_next_to_one_another(gpu, E):
    """Biases that put all sums within fp32's rounding of one value: the order is
    that of the sums in 64 bits, whose gaps here are far above its own rounding."""
    g = torch.Generator().manual_seed(E)
    for score in ("sigmoid", "softmax"):
        z = torch.randn(1, E, generator=g)
        s = torch.sigmoid(z.double()) if score == "sigmoid" else torch.softmax(z.double(), 1)
        bias = (0.75 - s[0]).float()
        sums = np.sort((s[0] + bias.double()).numpy())
        assert sums[-1] - sums[0] < 2.0 ** -23 and np.diff(sums)[-9:].min() > 1e-13
        _check(gpu, z, 8, score=score, bias=bias, what=E)
        # Rows that differ by little: 64 of them, each decided on its own.
        rows = z.repeat(64, 1) * (1 + 2.0 ** -20 * torch.randn(64, 1, generator=g))
        c = np.sort(((torch.sigmoid(rows.double()) if score == "sigmoid" else torch.softmax(rows.double(), 1))
                     + bias.double()).numpy(), axis=1)
        clear = torch.from_numpy(np.diff(c, axis=1)[:, -9:].min(axis=1) > 1e-13)
        _check(gpu, rows[clear], 8, score=score, bias=bias, what=(E, "rows"))
        for groups in (4, 8):
            v = np.sort((s[0] + bias.double()).numpy().reshape(groups, -1), axis=1)[:, -2:].sum(axis=1)
            if np.diff(np.sort(v)).min() > 1e-13:
                _check(gpu, z, 8, score=score, bias=bias, groups=groups, topk_groups=groups // 2, group_score="top2")


@pytest.mark.parametrize("E", [48, 256])
def test_many_rows_next_to_one_another(gpu, E):
    """The same in calls of many tokens: pairs, heaps and exact ties, with and without
    a bias, in and between groups."""
    g = torch.Generator().manual_seed(E)
    for score in ("sigmoid", "softmax"):
        near = lambda z: torch.sigmoid(z.double()) if score == "sigmoid" else torch.softmax(z.double(), 1)  # noqa: E731
        z = torch.randn(1500, E, generator=g)
        bias = 0.75 - near(z[:1])[0].float()
        z[1:500] = z[:1] * (1 + 2.0 ** -21 * torch.randn(499, 1, generator=g))          # all near
        z[500:1000, 1::2] = z[500:1000, ::2]                                            # equal pairs
        z[1000:1200, 1::2] = z[1000:1200, ::2] * (1 + 2.0 ** -23)                       # the next number
        c = np.sort((near(z) + bias.double()).numpy(), axis=1)
        clear = torch.from_numpy(np.diff(c, axis=1)[:, -10:].min(axis=1) > 1e-13)
        assert int(clear[:500].sum()) > 300
        for groups in (1, 4, 6 if E % 6 == 0 else 8):
            for group_score in ("max", "top2"):
                kw = dict(score=score, groups=groups, topk_groups=max(1, groups // 2), group_score=group_score)
                if groups > 1:   # rows whose groups are as near as their experts are left out
                    v = np.sort((near(z) + bias.double()).numpy().reshape(1500, groups, -1), axis=2)
                    v = np.sort(v[:, :, -1] if group_score == "max" else v[:, :, -2:].sum(axis=2), axis=1)
                    keep = clear & torch.from_numpy(np.diff(v, axis=1).min(axis=1) > 1e-13)
                else:
                    keep = clear
                rows = z[keep].repeat(2, 1)
                assert len(rows) > 1024
                _check(gpu, rows, 8, bias=bias, what=(E, kw), **kw)
                _check(gpu, z if groups == 1 else rows, 8, what=(E, kw, "no bias"), **kw)


@pytest.mark.parametrize("E,rows", [(48, 2500), (256, 4500)])
def test_rows_next_to_one_another_four_to_a_wave(gpu, E, rows):
    """Calls above the number of tokens from which four share a wave: near sums, pairs
    and exact ties among ordinary rows, between groups too."""
    g = torch.Generator().manual_seed(E + 1)
    for score in ("sigmoid", "softmax"):
        near = lambda z: torch.sigmoid(z.double()) if score == "sigmoid" else torch.softmax(z.double(), 1)  # noqa: E731
        z = torch.randn(rows, E, generator=g)
        bias = 0.75 - near(z[:1])[0].float()
        z[1:500] = z[:1] * (1 + 2.0 ** -21 * torch.randn(499, 1, generator=g))
        z[500:1000, 1::2] = z[500:1000, ::2]
        z[1000:1200, 1::2] = z[1000:1200, ::2] * (1 + 2.0 ** -23)
        c = (near(z) + bias.double()).numpy()
        clear = torch.from_numpy(np.diff(np.sort(c, axis=1), axis=1)[:, -10:].min(axis=1) > 1e-13)
        assert int(clear[:500].sum()) > 300
        for groups in (1, 4, 6 if E % 6 == 0 else 8):
            for group_score in ("max", "top2"):
                kw = dict(score=score, groups=groups, topk_groups=max(1, groups // 2), group_score=group_score)
                v = np.sort(c.reshape(rows, groups, -1), axis=2)
                v = np.sort(v[:, :, -1] if group_score == "max" else v[:, :, -2:].sum(axis=2), axis=1)
                keep = clear if groups == 1 else clear & torch.from_numpy(np.diff(v, axis=1).min(axis=1) > 1e-13)
                some = z[keep].repeat(2, 1)[:rows]   # as many as before: all near rows, some others twice
                assert len(some) > (2048 if E <= 64 else 4096)
                _check(gpu, some, 8, bias=bias, what=(E, kw), **kw)
                _check(gpu, z if groups == 1 else some, 8, what=(E, kw, "no bias"), **kw)


@pytest.mark.parametrize("E,rows", [(64, 2048), (64, 2049), (60, 3001), (65, 4096), (65, 4097), (256, 4099), (250, 5001)])
def test_both_sides_of_four_to_a_wave(gpu, E, rows):
    for i, kw in enumerate(CONFIGS):
        for groups in (1, 4 if E % 4 == 0 else 5):
            if E % groups:
                continue
            group_score = ("max", "top2")[i % 2]
            mask = torch.rand(rows, generator=torch.Generator().manual_seed(i)) < 0.2 if i % 3 else None
            _check(gpu, _logits(rows, E, ("fp32", "bf16", "fp16")[i % 3], E + i), 6, pad=i % 2, what=(E, rows, kw, groups),
                   groups=groups, topk_groups=groups - groups // 2, group_score=group_score, mask=mask, **kw)


def test_two_best_without_a_bias(gpu):
    """The groups' values are sums of scores, not of logits."""
    z = torch.tensor([[5.0, -9.0, 4.0, 3.9, -1.0, -1.0, 0.0, 0.0]])
    for score in ("softmax", "sigmoid"):
        _check(gpu, z, 2, score=score, groups=4, topk_groups=1, group_score="top2")
        _check(gpu, z, 2, score=score, groups=4, topk_groups=1, group_score="max")


def test_outputs_of_the_caller_and_streams(gpu):
    z = _logits(50, 256, "bf16", 3).to(DEV)
    want = gpu.route_experts(z, 8)
    w = torch.full((52, 8), 7.0, device=DEV)
    e = torch.full((52, 8), 7, dtype=torch.int32, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = gpu.route_experts(z, 8, weights=w[1:51], experts=e[1:51], stream=s)
    s.synchronize()
    assert got[0].data_ptr() == w[1:51].data_ptr()
    assert torch.equal(w[1:51], want[0]) and torch.equal(e[1:51], want[1])
    assert bool((w[[0, 51]] == 7).all()) and bool((e[[0, 51]] == 7).all())


def test_refusals(gpu):
    z = _logits(4, 64, "fp32", 0).to(DEV)
    for kw, err in ((dict(topk=65), gpu.FP8BGError), (dict(topk=8, groups=3), gpu.FP8BGError),
                    (dict(topk=-1), ValueError), (dict(topk=8, score="max"), ValueError),
                    (dict(topk=8, group_score="sum"), ValueError), (dict(topk=8, bias=torch.zeros(63, device=DEV)), ValueError),
                    (dict(topk=8, bias=torch.zeros(64)), ValueError), (dict(topk=8, bias=torch.zeros(64, device=DEV).half()), TypeError),
                    (dict(topk=8, mask=torch.zeros(3, dtype=torch.bool, device=DEV)), ValueError),
                    (dict(topk=8, mask=torch.zeros(4, device=DEV)), TypeError),
                    (dict(topk=8, weights=torch.zeros(4, 7, device=DEV)), ValueError),
                    (dict(topk=8, experts=torch.zeros(4, 8, dtype=torch.int64, device=DEV)), TypeError)):
        with pytest.raises(err):
            gpu.route_experts(z, **kw)
    with pytest.raises(TypeError):
        gpu.route_experts(z.double(), 8)
    with pytest.raises(ValueError):
        gpu.route_experts(z.t(), 2)
    w, e = gpu.route_experts(z[:0], 8)
    assert w.shape == (0, 8) and e.shape == (0, 8)
    w, e = gpu.route_experts(z, 0)
    assert w.shape == (4, 0)
