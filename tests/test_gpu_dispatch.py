"""The way into expert order (exact) and back (within fp32's roundings) on the
GPU against their plain forms."""
import pytest
import torch

from tests import _tokens as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _ids(n, topk, E, seed, kind="even"):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":
        return torch.full((n, topk), E - 1, dtype=torch.int32)      # the same expert, more than once per token
    ids = torch.randint(-1 if kind == "some" else 0, E + (2 if kind == "some" else 0), (n, topk), generator=g)
    return ids.to(torch.int32)


def _x(n, K, dtype, seed, pad=0, lead=0):
    g = torch.Generator().manual_seed(seed)
    if dtype in (torch.int8, torch.float8_e4m3fn, torch.uint8):
        v = torch.randint(0, 256, (n, K + pad), generator=g, dtype=torch.uint8).view(dtype)
    else:
        v = torch.randn(n, K + pad, generator=g).to(dtype)
    return v[:, lead:lead + K]


def _dev(t):
    """The same slice of the same buffer on the GPU."""
    base = t if t._base is None else t._base
    return base.to(DEV)[:, t.storage_offset():t.storage_offset() + t.shape[1]] if t._base is not None else t.to(DEV)


def _same(a, b):
    assert a.dtype == b.dtype and a.shape == b.shape
    assert torch.equal(a.cpu().contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def _check(gpu, ids, E, x, x_scale=None, first=0, **kw):
    rows, scale, offsets, slots = gpu.dispatch_tokens(ids.to(DEV), E, _dev(x), None if x_scale is None else x_scale.to(DEV),
                                                      first_expert=first, **kw)
    wr, ws, wo, wl = T.dispatch(ids, E, x, x_scale, first)
    assert torch.equal(offsets.cpu(), wo), (offsets.cpu(), wo)
    assert torch.equal(slots.cpu(), wl)
    n = int(wo[-1])
    assert rows.shape == (ids.numel(), x.shape[1])
    _same(rows[:n], wr)
    if x_scale is None:
        assert scale is None
    else:
        _same(scale[:n], ws)
    return rows, scale, n


@pytest.mark.parametrize("tokens", [1, 2, 63, 64, 65, 200, 511, 512, 513, 1025, 3000])
@pytest.mark.parametrize("topk,E", [(1, 1), (8, 256), (2, 8), (6, 60), (3, 1024), (64, 100), (9, 64), (5, 257)])
@pytest.mark.parametrize("kind", ["even", "some", "one"])
def test_order(gpu, tokens, topk, E, kind):
    ids = _ids(tokens, topk, E, tokens + E, kind)
    _check(gpu, ids, E, _x(tokens, 40, torch.int8, 1), torch.rand(tokens))


@pytest.mark.parametrize("tokens,topk", [(1024, 1), (1025, 1), (724, 2), (725, 2), (512, 4), (513, 4), (323, 5), (324, 5),
                                         (256, 8), (257, 8), (90, 64), (91, 64)])
@pytest.mark.parametrize("E", [16, 1000])
@pytest.mark.parametrize("kind", ["even", "some", "one"])
def test_both_sides_of_few_choices(gpu, tokens, topk, E, kind):
    _check(gpu, _ids(tokens, topk, E, tokens, kind), E, _x(tokens, 515, torch.bfloat16, 2), torch.rand(tokens, 3))


@pytest.mark.parametrize("tokens,topk,E", [(40000, 8, 256), (20001, 3, 1000), (131072, 1, 16), (4096, 8, 128)])
@pytest.mark.parametrize("kind", ["even", "some", "one"])
def test_many_tokens(gpu, tokens, topk, E, kind):
    _check(gpu, _ids(tokens, topk, E, 1, kind), E, _x(tokens, 16, torch.int8, 1), torch.rand(tokens))


@pytest.mark.parametrize("K", [1, 3, 15, 16, 17, 100, 128, 1000, 1024, 1027, 4096, 4100, 9000, 20000])
@pytest.mark.parametrize("dtype", [torch.int8, torch.float8_e4m3fn, torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("pad,lead", [(0, 0), (16, 0), (3, 1)])
@pytest.mark.parametrize("tokens", [21, 1500])
def test_rows(gpu, K, dtype, pad, lead, tokens):
    if tokens > 100 and K > 4096:
        tokens = 1100
    S = None if K % 128 else K // 128
    scale = torch.rand(tokens, S) if S else torch.rand(tokens) if K % 2 else None
    _check(gpu, _ids(tokens, 8, 16, K, "some"), 16, _x(tokens, K, dtype, K, pad, lead), scale, first=1)


@pytest.mark.parametrize("first", [0, 16, 240, 250, 300, 2 ** 31 - 1 - 1024])
def test_share_of_the_experts(gpu, first):
    """Experts held elsewhere, and ids that no expert has, get no row."""
    ids = _ids(100, 4, 256, 3)
    ids[3, 0], ids[4, 1], ids[5, 2], ids[6, 3] = -1, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1024
    for tokens in (100, 3000):
        _check(gpu, ids.repeat(tokens // 100, 1), 16, _x(tokens, 64, torch.int8, 2), torch.rand(tokens, 3), first=first)


@pytest.mark.parametrize("tokens", [100, 3000])
def test_rows_of_the_caller(gpu, tokens):
    """What lies behind the last row, beside and around the buffers is left."""
    ids, x, s = _ids(tokens, 4, 32, 5), _x(tokens, 50, torch.int8, 3), torch.rand(tokens)
    buf = torch.full((tokens * 4 + 2, 70), 77, dtype=torch.int8, device=DEV)
    sc = torch.full((tokens * 4 + 2,), 7.0, device=DEV)
    rows, scale, n = _check(gpu, ids, 8, x, s, first=8, rows=buf[1:-1, 9:59], row_scale=sc[1:-1])
    assert 0 < n < tokens * 4 and rows.data_ptr() == buf[1:-1, 9:59].data_ptr()
    assert bool((buf[0] == 77).all()) and bool((buf[n + 1:] == 77).all())
    assert bool((buf[:, :9] == 77).all()) and bool((buf[:, 59:] == 77).all())
    assert bool((sc[0] == 7).all()) and bool((sc[n + 1:] == 7).all())


def test_empty(gpu):
    for tokens, topk, E, K in ((0, 8, 16, 64), (5, 0, 16, 64), (5, 4, 0, 64), (5, 4, 16, 0), (3000, 4, 0, 8), (3000, 4, 8, 0)):
        rows, scale, n = _check(gpu, _ids(tokens, topk, max(E, 1), 0), E, _x(tokens, K, torch.int8, 0), torch.rand(tokens))
        assert rows.shape == (tokens * topk, K)
    _check(gpu, _ids(5, 4, 16, 0), 16, _x(5, 8, torch.int8, 0), torch.rand(5, 0))


def test_int8_rows_are_padded(gpu):
    rows = gpu.dispatch_tokens(_ids(10, 2, 4, 0).to(DEV), 4, _x(10, 100, torch.int8, 0).to(DEV))[0]
    assert rows.stride(0) % 16 == 0


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp16", "bf16"),
                                       ("fp32", "bf16"), ("fp32", "fp32"), ("fp32", "fp16"), ("bf16", "fp16")])
@pytest.mark.parametrize("D", [1, 7, 8, 100, 512, 513, 1027, 4096, 5000])
@pytest.mark.parametrize("topk", [1, 2, 6, 8, 11, 64])
def test_combine(gpu, dtype, out, D, topk):
    for tokens, base in ((1, None), (37, "rows"), (300, "out")):
        g = torch.Generator().manual_seed(D + topk)
        rows = torch.randn(tokens * topk + 3, D + 3, generator=g).to(T.DTYPES[dtype])[:, 1:D + 1]
        slots = torch.randint(-1, tokens * topk + 4, (tokens, topk), generator=g).to(torch.int32)
        slots[0] = -1                                              # a token without a row
        weights = torch.randn(tokens, topk, generator=g)
        weights[slots < 0] = float("nan")                          # weighs nothing
        b = None if base is None else torch.randn(tokens, D + 2, generator=g).to(T.DTYPES[dtype if base == "rows" else out])[:, :D]
        got = gpu.combine_experts(_dev(rows), slots.to(DEV), weights.to(DEV), base=None if b is None else _dev(b),
                                  out_dtype=T.DTYPES[out])
        ref, tol = T.combine(rows, slots, weights, b)
        T.assert_close(got, ref, tol, out, (dtype, out, D, topk, tokens))


@pytest.mark.parametrize("tokens", [5, 4000])
def test_combine_into_a_slice_and_in_place(gpu, tokens):
    g = torch.Generator().manual_seed(2)
    rows, w = torch.randn(tokens * 2, 96, generator=g), torch.rand(tokens, 2, generator=g)
    slots = torch.randperm(tokens * 2, generator=g).view(tokens, 2).to(torch.int32)
    buf = torch.full((tokens + 2, 130), 5.0, device=DEV)
    view = buf[1:-1, 7:103]
    view.copy_(torch.randn(tokens, 96, generator=g))
    base = view.cpu().clone()
    got = gpu.combine_experts(rows.to(DEV), slots.to(DEV), w.to(DEV), base=view, out=view)
    assert got.data_ptr() == view.data_ptr()
    ref, tol = T.combine(rows, slots, w, base)
    T.assert_close(view, ref, tol, "fp32")
    assert bool((buf[[0, -1]] == 5).all()) and bool((buf[:, :7] == 5).all()) and bool((buf[:, 103:] == 5).all())


def test_combine_empty_and_infinite(gpu):
    w, i = torch.ones(3, 2, device=DEV), torch.zeros(3, 2, dtype=torch.int32, device=DEV)
    none = gpu.combine_experts(torch.zeros(0, 16, device=DEV), i, w)
    assert bool((none == 0).all())
    base = torch.randn(3, 16, device=DEV)
    assert torch.equal(gpu.combine_experts(torch.zeros(0, 16, device=DEV), i, w, base=base), base)
    assert torch.equal(gpu.combine_experts(torch.zeros(4, 16, device=DEV), i[:, :0], w[:, :0], base=base), base)
    rows = torch.full((4, 16), float("inf"), device=DEV)
    rows[1] = 1.0
    i[0, 0], i[0, 1] = -1, 1
    got = gpu.combine_experts(rows, i, w).cpu()
    assert bool((got[0] == 1).all()) and bool((got[1:] == float("inf")).all())
    assert gpu.combine_experts(rows, i[:0], w[:0]).shape == (0, 16)


def test_refusals(gpu):
    ids, x = _ids(8, 2, 4, 0).to(DEV), torch.zeros(8, 32, device=DEV)
    for args, kw, err in (((ids, -1, x), {}, ValueError), ((ids, 1025, x), {}, gpu.FP8BGError),
                          ((ids.long(), 4, x), {}, TypeError), ((ids[:7], 4, x), {}, ValueError),
                          ((ids.t(), 4, x[:2]), {}, ValueError), ((ids, 4, x.double()), {}, TypeError),
                          ((ids, 4, x, torch.zeros(7, device=DEV)), {}, ValueError),
                          ((ids, 4, x, torch.zeros(8, 2, 2, device=DEV)), {}, ValueError),
                          ((ids, 4, x), {"row_scale": torch.zeros(16, device=DEV)}, ValueError),
                          ((ids, 4, x), {"rows": torch.zeros(15, 32, device=DEV)}, ValueError),
                          ((ids, 4, x), {"rows": torch.zeros(16, 32, device=DEV).half()}, TypeError)):
        with pytest.raises(err):
            gpu.dispatch_tokens(*args, **kw)
    rows, w = torch.zeros(16, 32, device=DEV), torch.zeros(8, 2, device=DEV)
    for args, kw, err in (((rows, ids.long(), w), {}, TypeError), ((rows, ids, w[:7]), {}, ValueError),
                          ((rows, ids, w.half()), {}, TypeError), ((rows.double(), ids, w), {}, TypeError),
                          ((rows, ids, w), {"base": torch.zeros(8, 31, device=DEV)}, ValueError),
                          ((rows, ids, w), {"base": torch.zeros(8, 32, device=DEV).half()}, TypeError),
                          ((rows, ids, w), {"out": rows[:8]}, gpu.FP8BGError),
                          ((rows, ids, w), {"out": torch.zeros(8, 32, device=DEV), "out_dtype": torch.float16}, TypeError)):
        with pytest.raises(err):
            gpu.combine_experts(*args, **kw)
