"""What the values between the adapters' two products lose, seen where y cancels
the product: nothing, 2^-17 of a value, or 2^-22 of the largest of a token's 32."""
import pytest
import torch

from tests import _tokens as T

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _inputs(M, N, R, dtype, out, seed):
    """Token m's only rank that counts, m % R, is a sum of three weights that fp32 holds
    with all of its 24 bits; its column's weight is a power of two, and y is the
    output's nearest to the product, negative."""
    g = torch.Generator().manual_seed(seed)
    t = T.DTYPES[dtype]
    bits = 8 if dtype == "bf16" else 11
    last = 24 - 2 * bits if dtype == "fp16" else bits
    lead = 1 + torch.randint(0, 2 ** (bits - 1), (R,), generator=g) * 2.0 ** (1 - bits)
    mid = torch.randint(2 ** (bits - 1), 2 ** bits, (R,), generator=g) * 2.0 ** (1 - 2 * bits)
    low = torch.randint(2 ** (last - 1), 2 ** last, (R,), generator=g) * 2.0 ** -23
    sign = torch.randint(0, 2, (3, R), generator=g) * 2.0 - 1
    A = (torch.stack([lead, mid, low]) * sign).t()[None].contiguous()                # [1, R, 3]
    # All ranks are there; a token's others have weights of zero in every column.
    h = A[0].double().sum(1)
    assert torch.equal(h.float().double(), h) and torch.equal(A.to(t).float(), A)
    B = torch.zeros(1, N, R)
    n = torch.arange(N)
    B[0, n, n % R] = 2.0 ** (n % 4).float()
    delta = (B[0].double() @ h).expand(M, N)
    y = (-delta).to(T.DTYPES[out])
    return y, torch.ones(M, 3, dtype=t), A.to(t), B.to(t), delta, h


@pytest.mark.parametrize("M", [3, 700, 3400])
@pytest.mark.parametrize("R", [1, 5, 16, 32, 48, 64, 100, 256])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("bf16", "fp16"), ("bf16", "fp32"), ("fp16", "fp16"),
                                       ("fp16", "bf16"), ("fp16", "fp32")])
def test_what_is_left_where_y_cancels(gpu, M, R, dtype, out):
    N = 300
    y, x, A, B, delta, h = _inputs(M, N, R, dtype, out, R)
    ids = torch.zeros(M, dtype=torch.int32)
    got = gpu.add_adapters(y.to(DEV), x.to(DEV), A.to(DEV), B.to(DEV), ids.to(DEV)).cpu().double()
    ref = y.double() + delta
    if dtype == "bf16":
        off = 0.0 if out == "fp32" else 2.0 ** -17 * delta.abs()
    else:  # every |h| is in [1 - 2^-10, 2 + 2^-10], so the largest of 32 is below 2.01
        off = 2.0 ** -22 * 2.01 * B[0].double().abs().sum(1)
    # The products' fp32 sums: two or three terms of one rank and zeros, the last addition
    # rounded; then y's, and the output's own rounding.
    lim = off + 2 * T.U32 * (delta.abs() + ref.abs())
    if dtype == "bf16" and out == "fp32":  # all of it fits in 24 bits: exact
        lim = torch.zeros_like(ref)
    lim = lim + (ref.abs() + lim) * (0 if out == "fp32" else T.U_OUT[out]) + (0 if out == "fp32" else T.TINY[out])
    err = (got - ref).abs()
    assert bool((err <= lim).all()), (float((err - lim).max()), (err > lim).nonzero()[:4].tolist())
