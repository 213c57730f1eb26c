"""Adapters with infinities and NaN in their tokens, weights and scales, and with
values next to the largest ones: what the formula gives, element by element."""
import pytest
import torch

from tests import _tokens as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF, NAN = float("inf"), float("nan")


def _reference(d):
    """The formula in 64 bits, each product and sum as written: 0 * inf is NaN.  Beside
    it where an infinite scale's sign is not settled: B (A x), in fp32 off by at most
    (K + R + 64) U32 of the sum of its terms' magnitudes (see T.adapters), may have
    either sign, or be 0, where it is no larger than that."""
    R, K = d["A"].shape[1:]
    either = torch.zeros(d["y"].shape, dtype=torch.bool)
    ref, tol, _ = T.adapters(d["y"], d["x"], d["A"], d["B"], d["ids"], d["scales"])
    for m in range(len(d["ids"])):
        a = int(d["ids"][m])
        if 0 <= a < len(d["A"]) and not bool(ref[m].isfinite().all()):
            h = (d["A"][a].double() * d["x"][m].double()).sum(1)
            product = (d["B"][a].double() * h).sum(1)
            ref[m] = d["y"][m].double() + float(d["scales"][a]) * product
            if abs(float(d["scales"][a])) == INF:
                size = d["B"][a].double().abs() @ (d["A"][a].double().abs() @ d["x"][m].double().abs())
                either[m] = product.abs() <= (K + R + 64) * T.U32 * size
    return ref, tol, either


def _check(gpu, d, out, what):
    ref, tol, either = _reference(d)
    dev = {k: v.to(DEV) for k, v in d.items()}
    for in_place in (False, True):
        y = dev["y"].clone()
        got = gpu.add_adapters(y, dev["x"], dev["A"], dev["B"], dev["ids"], dev["scales"],
                               out=None if in_place else torch.empty_like(y)).cpu()
        most = torch.finfo(T.DTYPES[out]).max
        assert not bool(got[either].isfinite().any()), what
        assert torch.equal(got.isnan() & ~either, ref.isnan() & ~either), what
        large = (ref.abs() > 1.01 * most) & ~either           # infinities, and what the output's type makes one of
        assert torch.equal(got[large].double(), ref[large].sign() * INF), what
        ok = (ref.abs() < 0.99 * most) & ~either
        T.assert_close(got[ok], ref[ok], tol[ok], out, what)
        bare = d["ids"] < 0
        assert torch.equal(got[bare], d["y"][bare]), what


def _make(M, N, K, R, dtype, out, seed):
    g = torch.Generator().manual_seed(seed)
    t = T.DTYPES[dtype]
    d = {"x": torch.randn(M, K, generator=g).to(t), "A": (torch.randn(3, R, K, generator=g) / K ** 0.5).to(t),
         "B": (0.3 * torch.randn(3, N, R, generator=g)).to(t), "y": torch.randn(M, N, generator=g).to(T.DTYPES[out]),
         "scales": 0.5 + torch.rand(3, generator=g), "ids": torch.randint(-1, 3, (M,), generator=g).to(torch.int32)}
    d["ids"][:5] = torch.tensor([0, 1, 2, 0, -1], dtype=torch.int32)[:M]
    return d


FORMS = [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32")]


@pytest.mark.parametrize("dtype,out", FORMS)
@pytest.mark.parametrize("R", [1, 3, 8, 10, 16, 40, 64, 100, 256])
@pytest.mark.parametrize("M,N,K", [(6, 200, 72), (70, 600, 1100), (3400, 330, 40)])
def test_tokens(gpu, dtype, out, R, M, N, K):
    """An infinite h: of one sign where the weights are, NaN where they are not or are zero."""
    d = _make(M, N, K, R, dtype, out, R)
    d["A"][0, :, 3] = 1.0                                     # every rank sees column 3 with this sign
    d["x"][0, 3], d["x"][3, 3] = INF, -INF
    d["B"][0, ::3] = d["B"][0, ::3].abs() + 0.01
    d["B"][0, 1::3] = -d["B"][0, 1::3].abs() - 0.01
    d["B"][0, 5] = 0.0
    d["x"][1, 0], d["x"][4] = NAN, NAN
    _check(gpu, d, out, (M, R))


@pytest.mark.parametrize("dtype,out", FORMS)
@pytest.mark.parametrize("R", [1, 3, 8, 10, 16, 40, 64, 100, 256])
@pytest.mark.parametrize("M,N,K", [(6, 200, 72), (70, 600, 1100), (3400, 330, 40)])
def test_weights(gpu, dtype, out, R, M, N, K):
    """An infinite weight makes its column infinite, by the sign of each token's h."""
    d = _make(M, N, K, R, dtype, out, R + 1)
    d["B"][0, 0, R - 1] = INF
    d["B"][0, 65, 0], d["B"][1, N - 1, R // 2], d["B"][1, 130] = -INF, -INF, INF
    d["B"][2, 7, 0] = NAN
    d["A"][2, 0, :] = 0.0                                     # 0 * inf
    d["B"][2, 9, 0] = INF
    _check(gpu, d, out, (M, R))


@pytest.mark.parametrize("dtype,out", FORMS)
@pytest.mark.parametrize("R", [1, 7, 16, 40, 100])
@pytest.mark.parametrize("M,N,K", [(6, 200, 72), (3400, 330, 40)])
def test_scales(gpu, dtype, out, R, M, N, K):
    """A scale multiplies the product: padded ranks stay out of an infinite one's, and
    one that passes the largest number with h, but not with the weights, is as any."""
    d = _make(M, N, K, R, dtype, out, R + 2)
    d["A"][:, R // 2 + 1:], d["B"][:, :, R // 2 + 1:] = 0.0, 0.0
    d["scales"][:] = torch.tensor([INF, -INF, 0.0])
    d["B"][2, 11, 0] = INF                                    # 0 * inf
    _check(gpu, d, out, (M, R, "infinite"))
    d = _make(M, N, K, R, dtype, out, R + 3)
    d["A"] *= 1000
    d["B"] = (d["B"].float() * 1e-4).to(d["B"].dtype)
    d["scales"][:] = torch.tensor([3e38, -2e38, 1e-38])
    if out == "fp32":
        d["x"] *= 0.01
    _check(gpu, d, out, (M, R, "large"))


@pytest.mark.parametrize("out", ["bf16", "fp32", "fp16"])
@pytest.mark.parametrize("R", [1, 5, 16, 40, 72])
@pytest.mark.parametrize("M", [6, 3400])
def test_next_to_the_largest(gpu, out, R, M):
    """An h that bf16 would round to infinity."""
    d = _make(M, 100, 64, R, "bf16", out, R)
    d["A"][0] = 0.0
    d["A"][0, :, 2], d["A"][0, :, 3] = 1.9921875, 2.0 ** -8
    d["x"][0], d["x"][3] = 0.0, 0.0
    d["x"][0, 2:4] = 2.0 ** 127
    d["x"][3, 2:4] = -2.0 ** 127
    d["B"] = torch.where(torch.arange(3)[:, None, None] == 0, d["B"].float() * 2.0 ** -124, d["B"].float()).bfloat16()
    h = d["A"][0].double() @ d["x"][0].double()
    assert bool((h < torch.finfo(torch.float32).max).all()) and bool(h.float().bfloat16().isinf().all())
    others = d["ids"] == 0
    others[0] = others[3] = False
    d["x"][others] *= 2.0 ** 100
    _check(gpu, d, out, (M, R))
