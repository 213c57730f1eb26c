"""The token operators together as a block runs them: a projection with its
requests' adapters, the router, rows into expert order, the experts' products
in int8 and in E4M3, and the way back; eagerly, on another stream, captured into
a graph and replayed, and two graphs that share nothing."""
import pytest
import torch

from tests import _tokens as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D, F, E, TOPK, L, R = 256, 128, 16, 4, 5, 8


def _weights(gpu):
    g = torch.Generator().manual_seed(7)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    w = {"proj": rn(D, D) / D ** 0.5, "router": rn(E, D) / D ** 0.5, "bias": 0.02 * rn(E),
         "up": rn(E, F, D) / D ** 0.5, "A": (rn(L, R, D) / D ** 0.5).bfloat16(), "B": (0.3 * rn(L, D, R)).bfloat16(),
         "scales": 1 + torch.rand(L, generator=g)}
    w = {k: v.to(DEV) for k, v in w.items()}
    w["proj8"] = gpu.quantize_tokens(w["proj"])
    up, s = gpu.quantize_tokens(w["up"].view(E * F, D))
    w["up8"] = up.view(E, F, D), s.view(E, F)
    f = [gpu.quantize_blocks(w["up"][e].bfloat16()) for e in range(E)]
    w["up_f8"] = torch.stack([a for a, _ in f]), torch.stack([b for _, b in f])
    return w


def _block(gpu, w, x, ids, mask, fmt, stream=None):
    """Every value on the way, so that each can be checked from those before it."""
    q, s = gpu.quantize_tokens(x, stream=stream)
    y = gpu.int8_gemm(q, s, *w["proj8"], out_dtype=torch.bfloat16, stream=stream)
    base = y.clone()
    gpu.add_adapters(y, x, w["A"], w["B"], ids, w["scales"], stream=stream)
    logits = y.float() @ w["router"].t()
    weights, experts = gpu.route_experts(logits, TOPK, score="sigmoid", bias=w["bias"], groups=4, topk_groups=2,
                                         group_score="top2", scale=2.5, mask=mask, stream=stream)
    if fmt == "int8":
        codes, scale = gpu.quantize_tokens(y, stream=stream)
        rows, row_scale, offsets, slots = gpu.dispatch_tokens(experts, E, codes, scale, stream=stream)
        up = gpu.int8_grouped_gemm(rows, row_scale, *w["up8"], offsets, out_dtype=torch.float32, stream=stream)
    else:
        codes, scale = gpu.quantize_rows(y, stream=stream)
        rows, row_scale, offsets, slots = gpu.dispatch_tokens(experts, E, codes, scale, stream=stream)
        up = gpu.grouped_gemm(rows, row_scale, *w["up_f8"], offsets, out_dtype=torch.float32, stream=stream)
    out = gpu.combine_experts(up, slots, weights, out_dtype=torch.float32, stream=stream)
    return dict(base=base, y=y, logits=logits, weights=weights, experts=experts, codes=codes, scale=scale, rows=rows,
                row_scale=row_scale, offsets=offsets, slots=slots, up=up, out=out)


def _inputs(tokens, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(tokens, D, generator=g).bfloat16()
    ids = torch.randint(-1, L, (tokens,), generator=g).to(torch.int32)
    mask = torch.rand(tokens, generator=g) < 0.2           # a padded batch
    return x.to(DEV), ids.to(DEV), mask.to(DEV)


def _check(v, w, x, ids, mask, fmt):
    c = {k: t.cpu() for k, t in v.items()}
    ref, tol, rms = T.adapters(c["base"], x.cpu(), w["A"].cpu(), w["B"].cpu(), ids.cpu(), w["scales"].cpu())
    T.assert_close(c["y"], ref, tol, "bf16", "adapters", rms)
    T.assert_route((c["weights"], c["experts"]),
                   T.route(c["logits"], TOPK, "sigmoid", w["bias"].cpu(), 4, 2, "top2", True, 2.5, mask.cpu()))
    rows, row_scale, offsets, slots = T.dispatch(c["experts"], E, c["codes"], c["scale"])
    n = int(offsets[-1])
    assert n == TOPK * int((~mask).sum())
    assert torch.equal(c["offsets"], offsets) and torch.equal(c["slots"], slots)
    assert torch.equal(c["rows"][:n].view(torch.uint8), rows.view(torch.uint8))
    assert torch.equal(c["row_scale"][:n], row_scale)
    # The combined output from the products' rows, and those against the weights that the codes stand for.
    ref, tol = T.combine(c["up"], c["slots"], c["weights"])
    T.assert_close(c["out"], ref, tol, "fp32", "combine")
    assert bool((c["out"][mask.cpu()] == 0).all())
    if fmt == "int8":
        codes, scales = (t.cpu().double() for t in w["up8"])
        a = rows.double() * row_scale.double()[:, None]
        weight = codes * scales[..., None]
    else:
        codes, scales = w["up_f8"][0].cpu().float().double(), w["up_f8"][1].cpu().double()
        a = rows.float().double() * row_scale.double().repeat_interleave(128, 1)
        weight = codes * scales.repeat_interleave(128, 1).repeat_interleave(128, 2)[:, :F]
    for e in range(E):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        want = a[lo:hi] @ weight[e].t()
        lim = (D + 8) * T.U32 * (a[lo:hi].abs() @ weight[e].abs().t())
        assert bool(((c["up"][lo:hi].double() - want).abs() <= lim).all()), e


@pytest.mark.parametrize("fmt", ["int8", "fp8"])
@pytest.mark.parametrize("tokens", [1, 7, 64, 600, 3000])
def test_block(gpu, fmt, tokens):
    w = _weights(gpu)
    args = _inputs(tokens, tokens)
    _check(_block(gpu, w, *args, fmt), w, *args, fmt)


def test_another_stream(gpu):
    """The operators on a stream of the caller's; torch's own steps go there too."""
    w = _weights(gpu)
    args = _inputs(700, 3)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        v = _block(gpu, w, *args, "int8", stream=s)
    s.synchronize()
    _check(v, w, *args, "int8")


@pytest.mark.parametrize("tokens", [5, 2500])
def test_captured_and_replayed(gpu, tokens):
    """Two graphs of one block over inputs of their own, replayed in turn with
    eager work between, new inputs each time: every replay equals the eager
    result, and leaves the other graph's."""
    w = _weights(gpu)
    ins = [tuple(t.clone() for t in _inputs(tokens, i)) for i in range(2)]
    _block(gpu, w, *ins[0], "int8")
    graphs, outs = [], []
    for a in ins:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(_block(gpu, w, *a, "int8"))
        graphs.append(graph)
    for step in range(3):
        want = []
        for i in range(2):
            new = _inputs(tokens, 10 + 2 * step + i)
            for t, u in zip(ins[i], new):
                t.copy_(u)
            want.append({k: t.clone() for k, t in _block(gpu, w, *new, "int8").items()})
        for i in (1, 0):
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            n = int(want[i]["offsets"][-1])
            for k, t in want[i].items():
                cut = slice(0, n) if k in ("rows", "row_scale", "up") else slice(None)
                assert torch.equal(outs[i][k][cut].view(torch.uint8), t[cut].view(torch.uint8)), (step, i, k)


def test_two_streams_at_once(gpu):
    """Calls that overlap on two streams share no memory."""
    w = _weights(gpu)
    ins = [_inputs(3000, 20 + i) for i in range(2)]
    want = [{k: t.clone() for k, t in _block(gpu, w, *a, "fp8").items()} for a in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(_block(gpu, w, *ins[i], "fp8"))
    torch.cuda.synchronize()
    for i in range(2):
        n = int(want[i]["offsets"][-1])
        for v in got[i]:
            for k in ("y", "weights", "experts", "offsets", "slots", "out"):
                assert torch.equal(v[k], want[i][k]), (i, k)
            assert torch.equal(v["rows"][:n].view(torch.uint8), want[i]["rows"][:n].view(torch.uint8))
