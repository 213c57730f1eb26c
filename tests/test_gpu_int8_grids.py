"""Products of more workgroups than one launch holds (2^32 threads)."""
import pytest
import torch

from tests._gpu import forced_config

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _codes(*s):
    g = torch.Generator(device=DEV).manual_seed(s[0])
    return torch.randint(-128, 128, s, generator=g, device=DEV, dtype=torch.int8)


def _check(C, A, a_s, w, w_s):
    """All of a one-column product, some rows at a time: the sums are below
    2^24, so fp32 holds them exactly.  w, w_s: a row of weights for each row of
    A, or for all."""
    M, step = A.shape[0], 1 << 24
    for lo in range(0, M, step):
        part = slice(lo, min(lo + step, M))
        each = w.shape[0] == M
        acc = (A[part].float() * (w[part] if each else w).float()).sum(dim=1)
        want = ((a_s[part] * (w_s[part] if each else w_s)) * acc).to(torch.bfloat16)
        assert torch.equal(C[part, 0], want), lo


@pytest.mark.parametrize("cfg,rows,K,lda", [(2, 8, 16, 16), (1, 32, 17, 17), (None, 64, 17, 17)])
def test_product(gpu, cfg, rows, K, lda):
    M = rows * (1 << 23) + 5
    if cfg is None:
        assert gpu.int8_plan(M, 1, K)["grid"] > 1 << 23
    A, a_s = _codes(M, K), torch.rand(M, device=DEV)
    B, b_s = _codes(1, K), torch.rand(1, device=DEV)
    with forced_config(cfg):
        C = gpu.int8_gemm(A, a_s, B, b_s)
    _check(C, A, a_s, B, b_s)


def test_columns(gpu):
    N, K = 16 * (1 << 23) + 7, 16
    A, a_s = _codes(1, K), torch.rand(1, device=DEV)
    B, b_s = _codes(N, K), torch.rand(N, device=DEV)
    with forced_config(3):
        C = gpu.int8_gemm(A, a_s, B, b_s)
    _check(C.t(), B, b_s, A, a_s)


def test_experts(gpu):
    """One row to an expert."""
    E, K = (1 << 23) + 9, 16
    A, a_s = _codes(E, K), torch.rand(E, device=DEV)
    B, b_s = _codes(E + 1, K)[1:].contiguous(), torch.rand(E, device=DEV)
    off = torch.arange(E + 1, device=DEV, dtype=torch.int32)
    with forced_config(2):
        C = gpu.int8_grouped_gemm(A, a_s, B[:, None], b_s[:, None], off)
    _check(C, A, a_s, B, b_s)
