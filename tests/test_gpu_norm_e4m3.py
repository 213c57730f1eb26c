"""The block norm's E4M3 output where a quotient is no ordinary number: both of
its kernels (rows in registers, and rows too long for them) give the codes that
the interface states."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TYPES = [torch.bfloat16, torch.float16, torch.float32]
WIDTHS = [256, 4096, 33024]     # on a wave, on a workgroup, read again for every pass


def _inputs(M, D, dtype):
    g = torch.Generator().manual_seed(D)
    return [torch.randn(*s, generator=g).to(dtype).to(DEV) for s in ((M, D), (M, D), (D,))]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype", TYPES)
def test_groups_with_an_infinity_or_a_nan(gpu, D, dtype):
    """Their scale is one, their codes are zero, so that their products are NaN;
    every other group is what it was."""
    h, x, w = _inputs(5, D, dtype)
    _, clean_q, clean_s = gpu.block_norm(h, x, pre_weight=w, quantize="fp8")
    w[130], h[3, D // 2] = float("inf"), float("nan")
    _, q, s = gpu.block_norm(h, x, pre_weight=w, quantize="fp8")
    fine = [0, 1, 2, 4]
    assert bool(s[fine, 1].isinf().all()) and bool(s[3].isnan().all())
    codes, want = q.view(torch.uint8).clone(), clean_q.view(torch.uint8).clone()
    want[:, 128:256] = 0
    want[3] = 0
    assert torch.equal(codes, want)
    others = [g for g in range(D // 128) if g != 1]
    assert torch.equal(s[fine][:, others], clean_s[fine][:, others])
    B, b_s = gpu.quantize_blocks(torch.randn(64, D, device=DEV).to(torch.bfloat16))
    assert bool(gpu.gemm(q, s, B, b_s, out_dtype=torch.float32).isnan().all())


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype", TYPES)
def test_zeros_keep_their_sign(gpu, D, dtype):
    """x / scale of a negative zero is a negative zero, as in the activation
    quantiser's codes."""
    _, x, w = _inputs(4, D, dtype)
    x[:, ::3] = 0
    _, q, _ = gpu.block_norm(x, pre_weight=w, quantize="fp8")
    want = torch.where(w < 0, 128, 0).to(torch.uint8).expand(4, D)
    assert torch.equal(q.view(torch.uint8)[:, ::3], want[:, ::3])
    flat = torch.tensor([-0.0, 0.0] * 64, device=DEV, dtype=torch.bfloat16)[None]
    codes, _ = gpu.quantize_rows(flat)
    assert codes.view(torch.uint8)[0, :2].tolist() == [128, 0]
