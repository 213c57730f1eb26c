"""The token operators at the sizes where 32-bit arithmetic on the host or a
grid's dimension ends."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOP = 2 ** 31 - 1 - 1024


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("D", [TOP - 1022, TOP - 1, TOP])
def test_combine_of_the_longest_rows(gpu, D):
    rows = torch.randint(-100, 100, (1, D), dtype=torch.int8, device=DEV).to(torch.bfloat16)
    slots = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    out = gpu.combine_experts(rows, slots, torch.full((1, 1), 2.0, device=DEV))
    rows *= 2
    assert torch.equal(out, rows)


@pytest.mark.parametrize("rows,E,topk,bias", [(2 ** 24 + 333, 4, 2, False), (2 ** 24 + 333, 4, 1, True),
                                              (2 ** 22 + 5, 260, 3, False), (2 ** 22 + 5, 64, 63, True)])
def test_route_past_2_20_workgroups(gpu, rows, E, topk, bias):
    """16 tokens to a workgroup, and four: by one kernel up to 62 choices, by another above."""
    g = torch.Generator(device=DEV).manual_seed(rows)
    z = torch.randn(rows, E, generator=g, device=DEV)
    b = torch.randn(E, generator=g, device=DEV) if bias else None
    w, e = gpu.route_experts(z, topk, score="sigmoid", bias=b, renormalize=False)
    for at in range(0, rows, 1 << 21):
        part = z[at:at + (1 << 21)].double()
        s = torch.sigmoid(part)
        c = part if b is None else s + b.double()
        order = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :topk]
        assert torch.equal(e[at:at + (1 << 21)].long(), order), at
        want = s.gather(1, order)
        # fp32's sigmoid: 1.5 |z| of exp's argument and a few roundings, of s.
        assert bool(((w[at:at + (1 << 21)].double() - want).abs() <= 2.0 ** -24 * (8 + 2 * part.abs().amax()) * want).all())


@pytest.mark.parametrize("tokens,K", [(2 ** 22 + 7, 24), (2 ** 20 + 7, 1040)])
def test_dispatch_past_2_20_workgroups(gpu, tokens, K):
    """A wave to a token, and four."""
    g = torch.Generator(device=DEV).manual_seed(K)
    experts = torch.randint(-1, 9, (tokens, 1), generator=g, device=DEV, dtype=torch.int32)
    x = torch.randint(-128, 128, (tokens, K), generator=g, device=DEV, dtype=torch.int8)
    rows, _, offsets, slots = gpu.dispatch_tokens(experts, 8, x)
    flat = experts[:, 0]
    here = (flat >= 0) & (flat < 8)
    order = torch.sort(torch.where(here, flat, 8), stable=True).indices[:int(here.sum())]
    want = torch.full_like(flat, -1)
    want[order] = torch.arange(len(order), device=DEV, dtype=torch.int32)
    assert torch.equal(slots[:, 0], want)
    assert torch.equal(offsets[1:], torch.bincount(flat[here], minlength=8).cumsum(0).to(torch.int32))
    assert torch.equal(rows[:len(order)], x[order])


@pytest.mark.parametrize("R", [12, 40])
def test_adapters_past_2_15_tiles(gpu, R):
    """Tiles of 64 tokens past a grid's second dimension."""
    M, N, K, L = 2 ** 21 + 1000, 64, 32, 5
    g = torch.Generator(device=DEV).manual_seed(R)
    v = lambda *s: torch.randint(-2, 3, s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    x, A, B, y = v(M, K), v(L, R, K), v(L, N, R), v(M, N).float()
    ids = (torch.arange(M, device=DEV) // 300 % (L + 1) - 1).to(torch.int32)
    got = gpu.add_adapters(y, x, A, B, ids, out=torch.empty_like(y))
    want = y.clone()
    for a in range(L):   # whole numbers that fp32 holds: exact
        t = (ids == a).nonzero()[:, 0]
        want[t] += (x[t].float() @ A[a].float().t().contiguous()) @ B[a].float().t().contiguous()
    assert torch.equal(got, want)
