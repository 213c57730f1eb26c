"""Codes whose rows are padded, as quantize_tokens makes them at a K that is no
multiple of 16, are weights of the grouped product like any others."""
import importlib.util
import os

import pytest
import torch

from tests import _int8 as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _check(gpu, A, a_s, B, b_s, counts, out="fp32"):
    off = torch.tensor([0, *counts], device=DEV).cumsum(0).to(torch.int32)
    C = gpu.int8_grouped_gemm(A, a_s, B, b_s, off, out_dtype=T.DTYPES[out])
    assert torch.equal(C, gpu.int8_grouped_gemm(A, a_s, B.contiguous(), b_s, off, out_dtype=T.DTYPES[out]))
    lo = 0
    for e, n in enumerate(counts):
        d = {"A": A[lo:lo + n].cpu(), "a_s": a_s[lo:lo + n].cpu(), "B": B[e].cpu(), "b_s": b_s[e].cpu(), "bias": None}
        T.assert_gemm(C[lo:lo + n], d, out, f"expert {e}")
        lo += n


@pytest.mark.parametrize("K", [5, 17, 776, 1000, 1001, 1024])
@pytest.mark.parametrize("counts", [[3, 0, 1, 2], [70, 1, 0, 200], [300]])
def test_quantised_weights(gpu, K, counts):
    E, N, M = len(counts), 70, sum(counts)
    g = torch.Generator(device=DEV).manual_seed(K)
    w, w_s = gpu.quantize_tokens(torch.randn(E * N, K, generator=g, device=DEV))
    q, s = gpu.quantize_tokens(torch.randn(M, K, generator=g, device=DEV))
    _check(gpu, q, s, w.view(E, N, K), w_s.view(E, N), counts)


@pytest.mark.parametrize("K,pitch", [(336, 352), (336, 333 + 4), (2048, 4096), (11, 40)])
@pytest.mark.parametrize("N", [1, 96])
@pytest.mark.parametrize("counts", [[3, 0, 1, 2], [70, 1, 0, 200], [40]])
def test_weights_in_wider_rows(gpu, K, pitch, N, counts):
    """Slices of the columns of wider weights; what lies between the rows does
    not get into the sums."""
    E = len(counts)
    g = torch.Generator(device=DEV).manual_seed(K + N)
    codes = lambda *s: torch.randint(-128, 128, s, generator=g, device=DEV, dtype=torch.int8)
    _check(gpu, codes(sum(counts), K), torch.rand(sum(counts), generator=g, device=DEV), codes(E, N, pitch)[:, :, :K],
           torch.rand(E, N, generator=g, device=DEV), counts, "bf16")


def test_weights_that_do_not_follow_one_another_are_refused(gpu):
    i = lambda *s: torch.zeros(*s, dtype=torch.int8, device=DEV)
    A, a_s, b_s = i(4, 64), torch.zeros(4, device=DEV), torch.zeros(2, 10, device=DEV)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    for B in (i(2, 12, 64)[:, :10], i(2, 64, 10).transpose(1, 2), i(10, 2, 64).transpose(0, 1), i(1, 10, 64).expand(2, 10, 64),
              i(2, 10, 128)[:, :, ::2]):
        with pytest.raises(ValueError):
            gpu.int8_grouped_gemm(A, a_s, B, b_s, off)
    with pytest.raises(gpu.FP8BGError) as e:      # rows that overlap
        gpu.int8_grouped_gemm(A, a_s, i(100000).as_strided((2, 10, 64), (320, 32, 1)), b_s, off)
    assert e.value.status == gpu.INVALID_VALUE


def test_example_at_widths_that_are_no_multiple_of_16(gpu):
    """The bound is the one that tests/test_gpu_int8_example.py derives."""
    spec = importlib.util.spec_from_file_location("int8_moe_block", os.path.join(ROOT, "examples", "int8_moe_block.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    block = ex.Int8MoEBlock(D=1000, F=500, out=1000)
    g = torch.Generator(device="cuda").manual_seed(5)
    x, res = (torch.randn(64, 1000, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    r, out, expert = block(x, res)
    for got, ref in zip((r, out), block.reference(x, res, expert)):
        assert got.shape == ref.shape and bool(got.isfinite().all())
        assert float((got.double() - ref).norm() / ref.norm()) < 0.03
