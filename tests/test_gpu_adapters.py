"""Low-rank adapters on the GPU against their 64-bit form."""
import pytest
import torch

from tests import _tokens as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _make(M, N, K, R, L, dtype, out, seed, pad=0, lead=0, bare=0.2, exact=False):
    """Inputs; `exact`: small integers, whose sums fp32 holds exactly."""
    g = torch.Generator().manual_seed(seed)
    t = T.DTYPES[dtype]

    def v(*shape):
        return torch.randint(-2, 3, shape, generator=g).float() if exact else torch.randn(*shape, generator=g)

    d = {"x": v(M, K + pad).to(t)[:, lead:lead + K], "A": (v(L, R, K) * (1 if exact else K ** -0.5)).to(t),
         "B": (v(L, N, R) * (1 if exact else 0.3)).to(t), "y": v(M, N + pad).to(T.DTYPES[out])[:, lead:lead + N],
         "scales": torch.randint(1, 3, (L,), generator=g).float() if exact else 0.5 + torch.rand(L, generator=g)}
    ids = torch.randint(0, L, (M,), generator=g)
    d["ids"] = torch.where(torch.rand(M, generator=g) < bare, -1, ids).to(torch.int32)
    return d


def _dev(t):
    if t._base is None:
        return t.to(DEV)
    return t._base.to(DEV)[:, t.storage_offset():t.storage_offset() + t.shape[1]]


def _run(gpu, d, in_place=False, scales=True):
    y = _dev(d["y"])
    out = None if in_place else torch.empty_like(y)
    got = gpu.add_adapters(y, _dev(d["x"]), d["A"].to(DEV), d["B"].to(DEV), d["ids"].to(DEV),
                           d["scales"].to(DEV) if scales else None, out=out)
    assert got.data_ptr() == (y if in_place else out).data_ptr()
    if not in_place:
        assert torch.equal(y.cpu(), d["y"])
    return got


def _check(gpu, d, out, what="", **kw):
    got = _run(gpu, d, **kw)
    ref, tol, rms = T.adapters(d["y"], d["x"], d["A"], d["B"], d["ids"], d["scales"] if kw.get("scales", True) else None)
    T.assert_close(got, ref, tol, out, what, rms)
    bare = (d["ids"] < 0) | (d["ids"] >= d["A"].shape[0])
    assert torch.equal(got.cpu()[bare], d["y"][bare])
    return got


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 33, 64, 100, 300])
@pytest.mark.parametrize("R", [1, 4, 7, 8, 10, 16, 17, 32, 33, 64, 65, 100, 128, 200, 256])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("fp16", "fp32")])
def test_tokens_and_ranks(gpu, M, R, dtype, out):
    _check(gpu, _make(M, 200, 328, R, 5, dtype, out, M + R), out, (M, R))


@pytest.mark.parametrize("K", [1, 7, 8, 31, 32, 33, 100, 128, 1000, 1024, 1027, 4096, 8200])
@pytest.mark.parametrize("N", [1, 5, 8, 31, 32, 33, 128, 129, 1000, 1537])
@pytest.mark.parametrize("pad,lead", [(0, 0), (5, 1)])
def test_widths(gpu, K, N, pad, lead):
    dtype, out = (("bf16", "fp32"), ("fp16", "fp16"), ("bf16", "fp16"), ("fp16", "bf16"))[(K + N) % 4]
    _check(gpu, _make(19, N, K, 12, 3, dtype, out, K + N, pad, lead), out, (K, N))


@pytest.mark.parametrize("M,N,K,R,L", [(64, 512, 4096, 16, 16), (1, 4096, 4096, 16, 1), (700, 1024, 1024, 64, 4),
                                       (2000, 640, 512, 16, 9), (3000, 264, 2048, 8, 64), (130, 4096, 512, 128, 2),
                                       (5000, 520, 256, 16, 3), (2500, 72, 520, 40, 100)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32")])
def test_exact_integers(gpu, M, N, K, R, L, dtype, out):
    """Sums that fp32 holds exactly: bit for bit, one rounding at the end."""
    d = _make(M, N, K, R, L, dtype, out, M + K, exact=True)
    d["A"] *= (torch.rand(d["A"].shape, generator=torch.Generator().manual_seed(1)) < 64 / K)  # h below 2^9
    ref = T.adapters(d["y"], d["x"], d["A"], d["B"], d["ids"], d["scales"])[0]
    assert float(ref.abs().max()) < 2.0 ** 16
    want = ref.float().to(T.DTYPES[out])
    assert torch.equal(_run(gpu, d).cpu(), want)
    assert torch.equal(_run(gpu, d, in_place=True).cpu(), want)


@pytest.mark.parametrize("M", [16, 50, 1000])
def test_runs_and_alternations(gpu, M):
    """Adapters in runs, each token its own, one for all, none at all, and ids
    that no adapter has."""
    L = 40
    d = _make(M, 264, 520, 16, L, "bf16", "fp32", M)
    m = torch.arange(M)
    for ids in (m // 7 % L, m % L, torch.full((M,), 3), torch.full((M,), -1), torch.full((M,), L),
                torch.where(m % 3 == 0, 2 ** 31 - 1, torch.where(m % 3 == 1, -2 ** 31, m % L))):
        d["ids"] = ids.to(torch.int32)
        _check(gpu, d, "fp32", ids[:4])
        _check(gpu, d, "fp32", ids[:4], in_place=True, scales=False)


@pytest.mark.parametrize("R", [1, 3, 4, 7, 8, 16, 24, 30, 32, 33, 64, 65, 128, 200, 256])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32")])
def test_many_tokens(gpu, R, dtype, out):
    """Prefills: runs of one adapter and tokens that change theirs, columns that no
    block divides, out of place and in place."""
    for M, N, K, L in ((3333, 136, 72, 3), (4100, 345, 40, 7)):
        d = _make(M, N, K, R, L, dtype, out, M + R, pad=3 * (R % 2), lead=R % 2)
        m = torch.arange(M)
        for ids in (d["ids"], (m // 100 % (L + 1) - 1), torch.where(m % 1000 < 500, m // 64 % L, -1)):
            d["ids"] = ids.to(torch.int32)
            _check(gpu, d, out, (M, R), in_place=R % 2 == 0)


@pytest.mark.parametrize("M,R", [(496, 64), (497, 64), (240, 128), (250, 128), (112, 256), (113, 256), (816, 40),
                                 (817, 40), (999, 36), (640, 200), (3200, 16), (3201, 16), (512, 32), (513, 30)])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "fp32")])
@pytest.mark.parametrize("in_place", [False, True])
def test_both_sides_of_many_tokens(gpu, M, R, dtype, out, in_place):
    """Tokens of 21 adapters in any order, more of them per workgroup than it has workers."""
    _check(gpu, _make(M, 328, 264, R, 21, dtype, out, M + R), out, (M, R), in_place=in_place)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M", [20, 3400])
@pytest.mark.parametrize("R", [16, 48, 100])
def test_ranks_of_unlike_sizes(gpu, dtype, M, R):
    """Ranks whose values differ by up to 2^12, with weights that make up for it: none
    may lose its small ones, within 32 ranks or between them."""
    d = _make(M, 72, 128, R, 2, dtype, "fp32", R)
    size = torch.exp2(-(torch.arange(R) % 13).float())
    d["A"] = (d["A"].float() * size[None, :, None]).to(d["A"].dtype)
    d["B"] = (d["B"].float() / size / 64).to(d["B"].dtype)
    d["x"] *= 16
    _check(gpu, d, "fp32", (M, R))


def test_infinities_stay_with_their_tokens(gpu):
    """A NaN or infinity in one token, or in an adapter that others use, reaches
    no other token."""
    for M in (40, 600, 3500):
        d = _make(M, 96, 256, 16, 4, "bf16", "fp32", 1, bare=0.3)
        d["x"][5] = float("nan")
        d["x"][6, 3] = float("inf")
        d["A"][2, 4, 7], d["B"][3, 9, 2] = float("nan"), float("inf")
        d["ids"][5], d["ids"][6], d["ids"][7] = 0, 1, -1
        d["x"][7] = float("nan")                      # a token without an adapter
        got = _run(gpu, d).cpu()
        clean = (d["ids"] == 0) | (d["ids"] == 1)
        clean[5] = clean[6] = False
        ref, tol, _ = T.adapters(d["y"], d["x"], d["A"], d["B"], d["ids"], d["scales"])
        T.assert_close(got[clean], ref[clean], tol[clean], "fp32")
        bare = d["ids"] < 0
        assert torch.equal(got[bare], d["y"][bare])
        assert bool(got[5].isnan().all()) and not bool(got[6].isfinite().all())
        third = d["ids"] == 3
        assert bool(got[third][:, :9].isfinite().all()) and not bool(got[third][:, 9].isfinite().any())


def test_padded_ranks_and_zeros(gpu):
    """An adapter padded with zeros is the adapter; sizes of zero leave y."""
    d = _make(30, 100, 64, 8, 3, "fp16", "fp32", 2)
    want = _run(gpu, d)
    d["A"] = torch.cat([d["A"], torch.zeros(3, 24, 64, dtype=torch.float16)], 1)
    d["B"] = torch.cat([d["B"], torch.zeros(3, 100, 24, dtype=torch.float16)], 2)
    assert torch.equal(_run(gpu, d), want)
    for M, N, K, R, L in ((0, 8, 8, 4, 2), (5, 0, 8, 4, 2), (5, 8, 0, 4, 2), (5, 8, 8, 0, 2), (5, 8, 8, 4, 0)):
        y = torch.randn(M, N, device=DEV)
        args = (torch.zeros(M, K, device=DEV).half(), torch.zeros(L, R, K, device=DEV).half(),
                torch.zeros(L, N, R, device=DEV).half(), torch.zeros(M, dtype=torch.int32, device=DEV))
        assert torch.equal(gpu.add_adapters(y, *args, out=torch.full_like(y, 9.0)), y)
        keep = y.clone()
        assert torch.equal(gpu.add_adapters(y, *args), keep)


def test_around_the_output(gpu):
    d = _make(37, 77, 64, 8, 3, "bf16", "bf16", 4)
    buf = torch.full((40, 100), 3.0, dtype=torch.bfloat16, device=DEV)
    buf[1:38, 9:86] = d["y"].to(DEV)
    gpu.add_adapters(buf[1:38, 9:86], d["x"].to(DEV), d["A"].to(DEV), d["B"].to(DEV), d["ids"].to(DEV), d["scales"].to(DEV))
    ref, tol, rms = T.adapters(d["y"], d["x"], d["A"], d["B"], d["ids"], d["scales"])
    T.assert_close(buf[1:38, 9:86], ref, tol, "bf16")
    assert bool((buf[0] == 3).all()) and bool((buf[38:] == 3).all())
    assert bool((buf[:, :9] == 3).all()) and bool((buf[:, 86:] == 3).all())


def test_refusals(gpu):
    def call(**kw):
        a = {"y": torch.zeros(4, 24, device=DEV), "x": torch.zeros(4, 16, device=DEV).half(),
             "A": torch.zeros(2, 8, 16, device=DEV).half(), "B": torch.zeros(2, 24, 8, device=DEV).half(),
             "adapters": torch.zeros(4, dtype=torch.int32, device=DEV), **kw}
        return gpu.add_adapters(**a)

    assert call().shape == (4, 24)
    for kw, err in (({"x": torch.zeros(4, 16, device=DEV)}, TypeError), ({"A": torch.zeros(2, 8, 16, device=DEV).bfloat16()}, TypeError),
                    ({"A": torch.zeros(2, 8, 15, device=DEV).half()}, ValueError), ({"B": torch.zeros(2, 24, 7, device=DEV).half()}, ValueError),
                    ({"B": torch.zeros(2, 8, 24, device=DEV).half().transpose(1, 2)}, ValueError),
                    ({"adapters": torch.zeros(4, dtype=torch.int64, device=DEV)}, TypeError),
                    ({"adapters": torch.zeros(3, dtype=torch.int32, device=DEV)}, ValueError),
                    ({"scales": torch.zeros(3, device=DEV)}, ValueError), ({"x": torch.zeros(3, 16, device=DEV).half()}, ValueError),
                    ({"out": torch.zeros(4, 24, device=DEV).half()}, TypeError),
                    ({"A": torch.zeros(2, 257, 16, device=DEV).half(), "B": torch.zeros(2, 24, 257, device=DEV).half()}, gpu.FP8BGError)):
        with pytest.raises(err):
            call(**kw)
