"""Small experts, all rows in one of them: a workgroup takes one tile of rows,
so the grid has room for every tile wherever the rows are."""
import pytest

import block_scaled_fp8_gemm_amd as fbg


@pytest.mark.parametrize("E,M,N,K", [(64, 512, 128, 4096), (8, 64, 512, 4096), (32, 128, 256, 4096), (256, 3072, 128, 1001),
                                     (64, 512, 128, 1001), (8, 96, 515, 776)])
def test_the_grid_holds_any_distribution_of_the_rows(E, M, N, K):
    p = fbg.int8_plan(M, N, K, E=E)
    assert p["config"] in (2, 3, 4)
    across = -(-N // p["tile_n"])
    assert p["grid"] == (M // p["tile_m"] + E) * across
    # the experts' first tiles, and the rest of one that has all the rows
    assert p["grid"] >= (E - 1 + -(-M // p["tile_m"])) * across
