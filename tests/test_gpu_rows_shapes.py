"""The row operators in every split of a row over threads that many rows take
(512 and more: two or four chunks of 16 bytes per thread), in every type, with
every kind of gate and every output.  Bounds and bit patterns as in
tests/test_gpu_rows.py; the norms are checked on rows picked from all of them."""
import pytest
import torch

from tests import _int8 as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
# Chunks to a row on either side of every step: half a wave, 64, 128, 256 and
# 512 threads of two chunks (of four past 512 chunks), 1024 of four.
CHUNKS = [20, 32, 33, 64, 65, 128, 129, 256, 257, 512, 513, 1024, 1025, 2048, 2049, 4096]


def _per_chunk(dtype):
    return 4 if dtype == "fp32" else 8


def _rows(M):
    g = torch.Generator().manual_seed(M)
    return torch.cat([torch.arange(9), torch.randint(9, M - 9, (14,), generator=g).sort().values, torch.arange(M - 9, M)])


@pytest.mark.parametrize("chunks", CHUNKS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("less,pad", [(0, 0), (3, 5)])
def test_quantize(gpu, chunks, dtype, less, pad):
    M, K = 513, chunks * _per_chunk(dtype) - less
    g = torch.Generator().manual_seed(chunks)
    x = (torch.randn(M, K + pad, generator=g) * torch.exp(torch.randn(M, 1, generator=g))).to(T.DTYPES[dtype])
    q, s = gpu.quantize_tokens(x.to(DEV)[:, :K])
    wq, ws = T.quantize(x[:, :K])
    assert torch.equal(s.cpu(), ws) and torch.equal(q.cpu(), wq)


def _gate(kind, M, D, dtype, g):
    """(the gate, its values as [M, D] or a shape that broadcasts to it)"""
    t = lambda *s: torch.randn(*s, generator=g).to(T.DTYPES[dtype]).to(DEV)
    if kind == "none":
        return None
    if kind == "channel":
        return t(D)
    if kind == "token":
        return t(M, 1)
    if kind == "full":
        return t(M, D)
    if kind == "every_other":             # columns two apart
        return t(M, 2 * D)[:, ::2]
    if kind == "channel_apart":           # three apart, one for all rows
        return t(3 * D)[::3]
    assert kind == "columns_first"
    return t(D, M).t()


GATES = ["none", "channel", "token", "full", "every_other", "channel_apart", "columns_first"]


def _check(gpu, M, D, dtype, gate, quant, pad=0):
    g = torch.Generator().manual_seed(M + D)
    t = T.DTYPES[dtype]
    wide = lambda: torch.randn(M, D + pad, generator=g).to(t).to(DEV)[:, :D]
    h, x, gt = wide(), wide(), _gate(gate, M, D, dtype, g)
    post, pre = ((1 + 0.1 * torch.randn(D, generator=g)).to(t).to(DEV) for _ in range(2))
    got = gpu.block_norm(h, x, post_weight=post, gate=gt, pre_weight=pre, residual_scale=0.875, quantize=quant)
    at = _rows(M)
    some = lambda v: v[at.to(DEV)].cpu()
    gr = None if gt is None else (some(gt) if gt.dim() == 2 else gt.cpu())
    r, y, tr, ty = T.block_norm(some(h), some(x), post.cpu(), gr, pre.cpu(), 0.875, 1e-6, 0.0)
    what = f"{M}x{D} {dtype} gate {gate} quant {quant}"
    T.assert_close(some(got[0]), r, tr, dtype, what + " r")
    if quant is None:
        T.assert_close(some(got[1]), y, ty, dtype, what + " y")
    else:
        T.assert_codes(some(got[1] if quant == "int8" else got[1].float()), some(got[2]), y, ty, quant, what)


@pytest.mark.parametrize("chunks", CHUNKS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("quant", [None, "int8", "fp8"])
def test_norm(gpu, chunks, dtype, quant):
    """D whole chunks and, where the output allows it, odd; a residual of less
    and of more than 4 MB (other stores)."""
    i = CHUNKS.index(chunks)
    D = chunks * _per_chunk(dtype)
    if quant == "fp8":
        D = -(-D // 128) * 128
    size = D * (4 if dtype == "fp32" else 2)
    for j, M in enumerate((513, (4 << 20) // size + 600)):
        _check(gpu, M, D, dtype, GATES[(i + j) % 4], quant)
        if quant != "fp8":
            _check(gpu, M, D - 3, dtype, GATES[(i + j + 2) % 4], quant, pad=5)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D", [128, 1027, 4096, 33280])
def test_norm_gates(gpu, gate, dtype, D):
    """Few rows, many, and rows that are read again for every pass (33280)."""
    for M in ((20,) if D > 10000 else (20, 777)):
        _check(gpu, M, D, dtype, gate, None)
        _check(gpu, M, D, dtype, gate, "int8", pad=3)
        if D % 128 == 0:
            _check(gpu, M, D, dtype, gate, "fp8")
