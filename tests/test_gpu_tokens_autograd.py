"""The token operators are forward only: while gradients are recorded they write into no
tensor of the caller's if one of theirs requires a gradient, and what they write
counts as written, so that a backward pass does not take it for what was saved."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T, E, K, N, R, L, TOPK = 6, 8, 32, 24, 4, 2, 2


def _calls(gpu):
    """name -> (call, its tensors, which of them it writes)"""
    r = lambda *s: torch.randn(*s, device=DEV)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device=DEV)  # noqa: E731
    h = lambda *s: torch.randn(*s, device=DEV).bfloat16()  # noqa: E731
    a = dict(y=r(T, N), x=h(T, K), A=h(L, R, K), B=h(L, N, R), adapters=i(T), scales=r(L))
    c = dict(rows=r(T * TOPK, N), slots=i(T, TOPK), weights=r(T, TOPK), base=r(T, N), out=r(T, N))
    d = dict(experts=i(T, TOPK), x=r(T, K), x_scale=r(T), rows=r(T * TOPK, K), row_scale=r(T * TOPK))
    return {
        "adapters in place": (gpu.add_adapters, {**a}, ["y"]),
        "adapters": (gpu.add_adapters, {**a, "out": r(T, N)}, ["out"]),
        "combine": (gpu.combine_experts, {**c}, ["out"]),
        "dispatch": (lambda **kw: gpu.dispatch_tokens(E=E, **kw), {**d}, ["rows", "row_scale"]),
        "dispatch, rows alone": (lambda **kw: gpu.dispatch_tokens(E=E, **kw), {k: d[k] for k in ("experts", "x", "rows")}, ["rows"]),
        "route": (lambda **kw: gpu.route_experts(topk=TOPK, **kw),
                  dict(logits=r(T, E), bias=r(E), weights=r(T, TOPK), experts=i(T, TOPK)), ["weights", "experts"]),
    }


NAMES = ["adapters in place", "adapters", "combine", "dispatch", "dispatch, rows alone", "route"]


@pytest.mark.parametrize("name", NAMES)
def test_refused_while_gradients_are_recorded(gpu, name):
    call, args, written = _calls(gpu)[name]
    call(**args)
    for k, t in args.items():
        if not t.is_floating_point():
            continue
        before = {w: args[w].clone() for w in written}
        some = {**args, k: t.clone().requires_grad_()}
        with pytest.raises(ValueError, match="no_grad"):
            call(**some)
        view = {**args, k: (t.clone().requires_grad_() * 1.0)}     # not a leaf: of a graph
        with pytest.raises(ValueError, match="no_grad"):
            call(**view)
        torch.cuda.synchronize()
        assert all(torch.equal(args[w], before[w]) for w in written)
        with torch.no_grad():
            call(**some)
    with torch.inference_mode():
        call(**{k: t.clone() for k, t in args.items()})
        call(**args)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_of_the_call_hang_on_no_graph(gpu, name):
    call, args, written = _calls(gpu)[name]
    if name == "adapters in place":
        return
    own = {k: t if not t.is_floating_point() else t.clone().requires_grad_()
           for k, t in args.items() if k not in written}
    if name == "adapters":
        own["out"] = torch.empty(T, N, device=DEV)                 # its default is y
        own = {k: t.detach() for k, t in own.items()}
    got = call(**own)
    assert not any(t.requires_grad for t in (got if isinstance(got, tuple) else (got,)) if t is not None)


@pytest.mark.parametrize("name", NAMES)
def test_a_write_is_counted(gpu, name):
    call, args, written = _calls(gpu)[name]
    for k in written:
        before = {n: t._version for n, t in args.items()}
        call(**args)
        assert args[k]._version > before[k]
        assert all(t._version == before[n] for n, t in args.items() if n not in written)
        if not args[k].is_floating_point():
            continue
        p = torch.ones_like(args[k]).requires_grad_()
        out = (p * args[k]).sum()                                  # saves it for the backward pass
        with torch.no_grad():
            call(**args)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            out.backward()


def test_a_projection_with_gradients(gpu):
    """The call that lost the adapters' gradients without a word."""
    _, a, _ = _calls(gpu)["adapters in place"]
    w = torch.randn(N, K, device=DEV, requires_grad=True)
    y = a["x"].float() @ w.t()
    with pytest.raises(ValueError, match="no_grad"):
        gpu.add_adapters(**{**a, "y": y})
    y.sum().backward()
    assert torch.allclose(w.grad, a["x"].float().sum(0).expand(N, K), atol=1e-4)
