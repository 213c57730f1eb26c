"""fbg_int8_plan and the int8 products agree on which sizes they take."""
import pytest

import block_scaled_fp8_gemm_amd as fbg

P = 0x10000000
TOP = 2 ** 31 - 1 - 1024     # the products' largest extent


def _plan_status(**kw):
    try:
        fbg.int8_plan(**kw)
        return fbg.SUCCESS
    except fbg.FP8BGError as e:
        return e.status


@pytest.mark.parametrize("M,N,K", [(2 ** 31 - 1, 64, 256), (TOP + 1, 64, 256), (64, TOP + 1, 256), (64, 2 ** 31 - 1, 256),
                                   (16, 64, 131072), (-1, 64, 256), (16, -1, 256), (16, 64, -1)])
def test_the_plan_refuses_what_the_products_refuse(M, N, K):
    call = fbg.load().fbg_int8_gemm(P, max(K, 1), 2 * P, 3 * P, max(K, 1), 4 * P, None, 5 * P, max(N, 1), M, N, K, 0, None)
    assert call != fbg.SUCCESS and _plan_status(M=M, N=N, K=K) == call
    if M >= 0 and N >= 0:
        grouped = fbg.load().fbg_int8_grouped_gemm(P, max(K, 1), 2 * P, 3 * P, 4 * P, 5 * P, max(N, 1), 6 * P, 2, M, N, K,
                                                   0, None)
        assert _plan_status(M=M, N=N, K=K, E=2) == grouped


def test_too_many_experts():
    call = fbg.load().fbg_int8_grouped_gemm(P, 64, 2 * P, 3 * P, 4 * P, 5 * P, 1, 6 * P, TOP + 1, 4, 1, 64, 0, None)
    assert call == fbg.UNSUPPORTED and _plan_status(M=4, N=1, K=64, E=TOP + 1) == call


def test_more_tiles_than_32_bits():
    """No memory holds such outputs; the plan says so and names no grid."""
    assert _plan_status(M=TOP, N=TOP, K=64) == fbg.UNSUPPORTED
    assert _plan_status(M=TOP, N=TOP, K=64, E=TOP) == fbg.UNSUPPORTED
    for M, N in ((TOP, 1), (1, TOP), (2 ** 29, 1), (600000000, 1)):
        p = fbg.int8_plan(M, N, 17)
        assert 0 < p["grid"] < 2 ** 31
        assert p["grid"] == -(-M // p["tile_m"]) * -(-N // p["tile_n"])
