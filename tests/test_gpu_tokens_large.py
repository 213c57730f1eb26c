"""Offsets past 32 bits: tensors of more than 2^32 bytes, checked at both ends and
in between."""
import pytest
import torch

from tests import _tokens as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


def _some(n, k=40):
    g = torch.Generator().manual_seed(n)
    return torch.cat([torch.arange(k), n - 1 - torch.arange(k), torch.randint(0, n, (k,), generator=g)])


def test_route(gpu):
    rows, E = 9_000_000, 256
    z = torch.randn(rows, E, device=DEV, dtype=torch.bfloat16)
    assert z.numel() * 2 > 2 ** 32
    bias = 0.1 * torch.randn(E)
    for kw in (dict(), dict(score="sigmoid", bias=bias, groups=8, topk_groups=4, group_score="top2")):
        b = kw.get("bias")
        w, e = gpu.route_experts(z, 8, **{**kw, **({"bias": b.to(DEV)} if b is not None else {})})
        at = _some(rows)
        T.assert_route((w[at.to(DEV)], e[at.to(DEV)]), T.route(z[at.to(DEV)].cpu(), 8, **kw))


def test_dispatch_and_combine(gpu):
    tokens, topk, K, E = 150_000, 8, 4096, 64
    g = torch.Generator(device=DEV).manual_seed(1)
    experts = torch.randint(0, E, (tokens, topk), generator=g, device=DEV, dtype=torch.int32)
    x = torch.randint(-128, 128, (tokens, K), generator=g, device=DEV, dtype=torch.int8)
    scale = torch.rand(tokens, generator=g, device=DEV)
    rows, row_scale, offsets, slots = gpu.dispatch_tokens(experts, E, x, scale)
    assert rows.numel() > 2 ** 32
    flat = experts.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    want = torch.empty_like(flat)
    want[order] = torch.arange(len(flat), device=DEV, dtype=torch.int32)
    assert torch.equal(slots.reshape(-1), want)
    assert torch.equal(offsets[1:], torch.bincount(flat, minlength=E).cumsum(0).to(torch.int32))
    assert torch.equal(row_scale, scale[order // topk])
    for i in range(0, len(order), 100_000):
        assert torch.equal(rows[i:i + 100_000], x[order[i:i + 100_000] // topk])
    del rows, x
    weights = torch.rand(tokens, topk, generator=g, device=DEV)
    values = torch.randn(tokens * topk, 2048, generator=g, device=DEV, dtype=torch.float32).bfloat16()
    assert values.numel() * 2 > 2 ** 32
    out = gpu.combine_experts(values, slots, weights, out_dtype=torch.float32)
    at = _some(tokens).to(DEV)
    rows = values[slots[at].long().reshape(-1)].cpu()
    ref, tol = T.combine(rows, torch.arange(len(rows), dtype=torch.int32).view(len(at), topk), weights[at].cpu())
    T.assert_close(out[at], ref, tol, "fp32")


@pytest.mark.parametrize("R", [16, 72])
def test_adapters(gpu, R):
    M, N, K, L = 700_000, 4096, 64, 3
    g = torch.Generator(device=DEV).manual_seed(2)
    rn = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    x, A, B = rn(M, K), rn(L, R, K), rn(L, N, R)
    y = torch.randn(1000, N, generator=g, device=DEV).bfloat16().repeat(700, 1)
    assert y.numel() * 2 > 2 ** 32
    ids = (torch.arange(M, device=DEV) // 1000 % (L + 1) - 1).to(torch.int32)
    at = _some(M).to(DEV)
    d = {"y": y[at].cpu(), "x": x[at].cpu(), "A": A.cpu(), "B": B.cpu(), "ids": ids[at].cpu()}
    got = gpu.add_adapters(y, x, A, B, ids)
    ref, tol, rms = T.adapters(d["y"], d["x"], d["A"], d["B"], d["ids"])
    T.assert_close(got[at], ref, tol, "bf16", rms=rms)
    bare = (d["ids"] < 0).nonzero()[:, 0]
    assert len(bare) and torch.equal(got[at].cpu()[bare], d["y"][bare])
