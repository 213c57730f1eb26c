"""The token quantiser (bit for bit) and the block norm (within the bound that
its roundings allow) on the GPU against their plain forms."""
import pytest
import torch

from tests import _int8 as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
WIDTHS = [1, 2, 7, 63, 64, 100, 128, 129, 256, 511, 512, 1000, 1024, 1027, 2048, 4096, 4104, 5000, 8192, 9001, 16384,
          20000, 40001]


def _slice(t, pad, lead=0):
    """t as columns lead .. of rows `pad` elements wider, NaN around it."""
    if t is None:
        return None
    if not pad:
        return t.to(DEV)
    buf = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), dtype=t.dtype, device=DEV)
    buf[:, lead:lead + t.shape[1]] = t.to(DEV)
    return buf[:, lead:lead + t.shape[1]]


def _x(M, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp(torch.randn(M, 1, generator=g))
    if M > 2:
        x[1] = 0.0            # an empty row
        x[2] *= 1e-30         # all below the smallest scale
    return x.to(T.DTYPES[dtype])


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("pad,lead", [(0, 0), (8, 0), (3, 1)])
def test_quantize(gpu, K, dtype, pad, lead):
    M = 5 if K > 4096 else 37
    x = _x(M, K, dtype, K + pad)
    q, s = gpu.quantize_tokens(_slice(x, pad, lead))
    wq, ws = T.quantize(x)
    assert torch.equal(s.cpu(), ws)
    assert torch.equal(q.cpu(), wq)
    assert q.stride(0) % 16 == 0


def test_quantize_into_a_slice(gpu):
    x = _x(20, 300, "bf16", 1)
    buf = torch.full((22, 333), 5, dtype=torch.int8, device=DEV)
    q, s = gpu.quantize_tokens(x.to(DEV), q=buf[1:21, 7:307])
    assert torch.equal(q.cpu(), T.quantize(x)[0])
    assert bool((buf[0] == 5).all()) and bool((buf[21] == 5).all())
    assert bool((buf[:, :7] == 5).all()) and bool((buf[:, 307:] == 5).all())


@pytest.mark.parametrize("K", [1, 64, 4096, 20000])
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_quantize_non_finite_rows(gpu, K, dtype):
    """A NaN or an infinity shows in its row's scale and leaves the others."""
    x = _x(6, K, dtype, 3)
    x[0, K // 2], x[3, K - 1], x[4, 0] = float("nan"), float("inf"), float("-inf")
    q, s = gpu.quantize_tokens(x.to(DEV))
    q, s = q.cpu(), s.cpu()
    assert bool(s[0].isnan()) and s[3] == float("inf") and s[4] == float("inf")
    assert not bool(q[[0, 3, 4]].any())
    wq, ws = T.quantize(x)
    for m in (1, 2, 5):
        assert torch.equal(q[m], wq[m]) and s[m] == ws[m]
    w = torch.ones(3, K, dtype=torch.int8, device=DEV)
    C = gpu.int8_gemm(q.to(DEV), s.to(DEV), w, torch.ones(3, device=DEV), out_dtype=torch.float32).cpu()
    assert bool(C[[0, 3, 4]].isnan().all()) and bool(C[[1, 2, 5]].isfinite().all())


def test_quantize_ties_and_edges(gpu):
    """Quotients at .5 go to even; the scale is exact here."""
    row = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5, -127.0, 0.0, -0.0, 0.49999997])
    q, s = gpu.quantize_tokens(row[None].to(DEV))
    assert s.item() == 1.0
    assert q[0].tolist() == [127, 0, 2, 2, 0, -2, -2, 126, -127, 0, 0, 0]


def test_quantize_empty(gpu):
    q, s = gpu.quantize_tokens(torch.zeros(0, 64, device=DEV))
    assert q.shape == (0, 64) and s.shape == (0,)
    q, s = gpu.quantize_tokens(torch.zeros(3, 0, device=DEV))
    assert q.shape == (3, 0) and torch.equal(s.cpu(), T.quantize(torch.zeros(3, 0))[1])


def _norm_inputs(M, D, dtype, gate, seed, wtype=None):
    g = torch.Generator().manual_seed(seed)
    t = T.DTYPES[dtype]
    rn = lambda *s: torch.randn(*s, generator=g)
    h, x = (0.5 * rn(M, D)).to(t), (2 * rn(M, D)).to(t)
    if M > 3:
        h[1] = 0
        x[2] = 0
        h[3] = 0
        x[3] = 0               # nothing left: r is zero, y is zero, not NaN
    shape = {"none": None, "channel": (D,), "token": (M, 1), "full": (M, D), "row": (1, D)}[gate]
    w = T.DTYPES[wtype or dtype]
    return h, x, None if shape is None else rn(*shape).to(t), (1 + 0.1 * rn(D)).to(w), (1 + 0.1 * rn(D)).to(w)


def _check_norm(gpu, M, D, dtype, gate, quant=None, use_x=True, use_post=True, pad=0, lead=0, alpha=0.875, eps=1e-6,
                offset=0.0, wtype=None, seed=None):
    h, x, g, post, pre = _norm_inputs(M, D, dtype, gate, seed if seed is not None else D + M, wtype)
    x, post = x if use_x else None, post if use_post else None
    gd = None if g is None else (_slice(g, pad, lead) if gate == "full" else g.to(DEV))
    got = gpu.block_norm(_slice(h, pad, lead), _slice(x, pad, lead), post_weight=None if post is None else post.to(DEV),
                         gate=gd, pre_weight=pre.to(DEV), residual_scale=alpha, eps=eps, weight_offset=offset,
                         quantize=quant)
    torch.cuda.synchronize()
    r, y, tr, ty = T.block_norm(h, x, post, g, pre, alpha, eps, offset)
    what = f"{M}x{D} {dtype} gate {gate} quant {quant}"
    T.assert_close(got[0], r, tr, dtype, what + " r")
    if quant is None:
        T.assert_close(got[1], y, ty, dtype, what + " y")
    else:
        T.assert_codes(got[1], got[2], y, ty, quant, what)
    return got


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
def test_norm(gpu, D, dtype, gate):
    _check_norm(gpu, 5 if D > 2048 else 21, D, dtype, gate)


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("quant", ["int8", "fp8"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_norm_quantised(gpu, D, quant, dtype):
    if quant == "fp8" and D % 128:
        with pytest.raises(gpu.FP8BGError) as e:
            _check_norm(gpu, 4, D, dtype, "none", quant)
        assert e.value.status == gpu.UNSUPPORTED
        return
    _check_norm(gpu, 6, D, dtype, "full", quant)


@pytest.mark.parametrize("use_x,use_post", [(False, True), (True, False), (False, False)])
@pytest.mark.parametrize("D", [100, 1024, 30000])
def test_norm_without_a_residual_or_a_post_norm(gpu, use_x, use_post, D):
    _check_norm(gpu, 6, D, "bf16", "row", use_x=use_x, use_post=use_post)
    _check_norm(gpu, 6, D, "fp16", "token", "int8", use_x=use_x, use_post=use_post)


@pytest.mark.parametrize("D", [128, 1000, 4096, 17000])
@pytest.mark.parametrize("pad,lead", [(8, 0), (8, 8), (1, 1)])
def test_norm_of_slices(gpu, D, pad, lead):
    _check_norm(gpu, 7, D, "bf16", "full", pad=pad, lead=lead)
    _check_norm(gpu, 7, D, "fp32", "full", "int8", pad=pad, lead=lead)


@pytest.mark.parametrize("D", [256, 1001])
def test_norm_options(gpu, D):
    _check_norm(gpu, 9, D, "bf16", "channel", wtype="fp32")
    _check_norm(gpu, 9, D, "fp16", "channel", wtype="fp32", offset=1.0)
    _check_norm(gpu, 9, D, "bf16", "token", offset=1.0, alpha=-2.0, eps=0.1)
    _check_norm(gpu, 1, D, "bf16", "token")
    _check_norm(gpu, 400, D, "bf16", "channel")


def test_norm_without_a_second_norm(gpu):
    h, x, g, post, _ = _norm_inputs(9, 300, "bf16", "channel", 2)
    r, y = gpu.block_norm(h.to(DEV), x.to(DEV), post_weight=post.to(DEV), gate=g.to(DEV))
    assert y is None
    ref, _, tr, _ = T.block_norm(h, x, post, g, None, 1.0, 1e-6, 0.0)
    T.assert_close(r, ref, tr, "bf16")


@pytest.mark.parametrize("D", [64, 4096, 33000])
def test_norm_non_finite_values_stay_in_their_row(gpu, D):
    h, x, g, post, pre = _norm_inputs(6, D, "fp32", "full", 7)
    clean = gpu.block_norm(h.to(DEV), x.to(DEV), post.to(DEV), g.to(DEV), pre.to(DEV), quantize="int8")
    h[0, D // 2], x[4, 0] = float("nan"), float("inf")
    got = gpu.block_norm(h.to(DEV), x.to(DEV), post.to(DEV), g.to(DEV), pre.to(DEV), quantize="int8")
    assert bool(got[2][0].isnan()) and bool(got[2][4].isnan())
    assert not bool(got[1][0].any()) and not bool(got[1][4].any())
    for m in (1, 2, 3, 5):
        assert all(torch.equal(a[m], b[m]) for a, b in zip(got, clean))


def test_norm_quantised_outputs_feed_the_products(gpu):
    """int8 codes into int8_gemm and E4M3 codes into gemm, as a block does."""
    h, x, g, post, pre = _norm_inputs(33, 512, "bf16", "channel", 11)
    w = torch.randn(200, 512, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    _, y, _, ty = T.block_norm(h, x, post, g, pre, 1.0, 1e-6, 0.0)
    args = [t.to(DEV) for t in (h, x, post, g, pre)]
    r, q, s = gpu.block_norm(*args, quantize="int8")
    B, b_s = gpu.quantize_tokens(w.to(DEV))
    C = gpu.int8_gemm(q, s, B, b_s, out_dtype=torch.float32).cpu().double()
    # Half a step on either operand's codes, in the worst case all one way.
    ya, wa = s.cpu().double()[:, None] * q.cpu().double(), b_s.cpu().double()[:, None] * B.cpu().double()
    assert float((C - ya @ wa.t()).abs().max()) <= 8 * T.U32 * float((ya.abs() @ wa.abs().t()).max())
    da, dw = (ya - y).abs(), (wa - w.double()).abs()
    assert bool(((C - y @ w.double().t()).abs() <= da @ wa.abs().t() + y.abs() @ dw.t() + 1e-4).all())
    r8, q8, s8 = gpu.block_norm(*args, quantize="fp8")
    assert torch.equal(r8, r)
    A8, a8 = gpu.quantize_blocks(w.to(DEV))
    C8 = gpu.gemm(q8, s8, A8, a8, out_dtype=torch.float32).cpu().double()
    y8 = (q8.float().cpu().double().view(33, 4, 128) * s8.cpu().double()[..., None]).view(33, 512)
    w8 = A8.float().cpu().double()
    w8 = w8 * a8.cpu().double().repeat_interleave(128, 0)[:200].repeat_interleave(128, 1)
    # 512 products and 4 folds in fp32.
    assert bool(((C8 - y8 @ w8.t()).abs() <= 600 * T.U32 * (y8.abs() @ w8.abs().t())).all())


def test_more_rows_than_one_grid_dimension(gpu):
    """Rows past 2^20 workgroups: the grid's second dimension."""
    M, K = (1 << 23) + 5000, 32           # eight rows to a workgroup
    x = torch.randn(M, K, device=DEV, dtype=torch.bfloat16)
    q, s = gpu.quantize_tokens(x)
    r, y = gpu.block_norm(x, pre_weight=torch.ones(K, device=DEV, dtype=torch.bfloat16))
    for lo in (0, (1 << 23) - 7, M - 20):
        wq, ws = T.quantize(x[lo:lo + 20].cpu())
        assert torch.equal(q[lo:lo + 20].cpu(), wq) and torch.equal(s[lo:lo + 20].cpu(), ws)
        assert torch.equal(r[lo:lo + 20], x[lo:lo + 20])
        _, ref, _, tol = T.block_norm(x[lo:lo + 20].cpu(), None, None, None, torch.ones(K, dtype=torch.bfloat16), 1.0, 1e-6, 0.0)
        T.assert_close(y[lo:lo + 20], ref, tol, "bf16")


def test_large_residuals(gpu):
    """A residual of more than 4 MB takes another kind of store when y is asked for."""
    for M, D in ((1030, 4096), (1031, 4099), (1030, 8192), (601, 16390)):
        x, h = (torch.randn(M, D, device=DEV, dtype=torch.bfloat16) for _ in range(2))
        w = torch.ones(D, device=DEV, dtype=torch.bfloat16)
        r, c, cs = gpu.block_norm(h, x, post_weight=w, pre_weight=w, quantize="int8")
        assert torch.equal(r, gpu.block_norm(h, x, post_weight=w)[0])
        rows = torch.tensor([0, 1, 2, 3, M // 2, M - 5, M - 1])
        ref_r, ref_y, tr, ty = T.block_norm(h[rows].cpu(), x[rows].cpu(), w.cpu(), None, w.cpu(), 1.0, 1e-6, 0.0)
        T.assert_close(r[rows], ref_r, tr, "bf16")
        T.assert_codes(c[rows], cs[rows], ref_y, ty, "int8")


def test_rows_without_columns_have_a_scale(gpu):
    """The scales of rows of no columns are written (their products are zero, not what the memory held)."""
    want = T.quantize(torch.zeros(3, 0))[1]
    for n in (3, 5000):
        full = torch.full((n,), float("nan"), device=DEV)  # its memory is what the call below allocates
        del full
        h, w = torch.zeros(n, 0, device=DEV, dtype=torch.bfloat16), torch.zeros(0, device=DEV, dtype=torch.bfloat16)
        r, q, s = gpu.block_norm(h, h, post_weight=w, pre_weight=w, quantize="int8")
        assert r.shape == (n, 0) and q.shape == (n, 0) and torch.equal(s.cpu(), want[:1].expand(n))
        c = gpu.int8_gemm(q, s, torch.zeros(4, 0, device=DEV, dtype=torch.int8), torch.ones(4, device=DEV))
        assert torch.equal(c.cpu(), torch.zeros(n, 4, dtype=torch.bfloat16))
