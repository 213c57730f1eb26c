"""Grouped products whose rows are spread unevenly over the experts."""
import numpy as np
import pytest
import torch

from tests import _int8 as T
from tests._gpu import forced_config

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _counts(kind, E, M):
    c = np.zeros(E, dtype=int)
    if kind == "one":
        c[E // 2] = M
    elif kind == "last":
        c[-1] = M
    elif kind == "half":
        c[0] = M // 2
        c += np.bincount(np.arange(M - M // 2) % E, minlength=E)
    else:
        c += np.bincount(np.minimum(np.random.default_rng(E + M).geometric(0.3, M) - 1, E - 1), minlength=E)
    return c


SIZES = [(64, 512, 128, 4096), (8, 63, 200, 2048), (8, 96, 515, 776), (300, 1500, 33, 1001), (1, 50, 64, 2048), (3, 7, 70, 2064)]


@pytest.mark.parametrize("cfg,size", [(c, s) for c in (None, 2, 3, 4) for s in SIZES if c not in (2, 3) or s[3] % 16 == 0])
@pytest.mark.parametrize("kind", ["one", "last", "half", "falling"])
def test_skewed(gpu, cfg, kind, size):
    E, M, N, K = size
    counts = _counts(kind, E, M)
    d = T.make_gemm(M, N, K, seed=E + M, experts=E)
    off = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    with forced_config(cfg):
        C = gpu.int8_grouped_gemm(*[d[k].to(DEV) for k in ("A", "a_s", "B", "b_s")], off)
    lo = 0
    for e, n in enumerate(counts):
        if n:
            T.assert_gemm(C[lo:lo + n], {"A": d["A"][lo:lo + n], "a_s": d["a_s"][lo:lo + n], "B": d["B"][e],
                                         "b_s": d["b_s"][e], "bias": None}, "bf16", f"{kind} expert {e}")
        lo += n
