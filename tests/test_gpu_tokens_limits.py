"""The token operators at the sizes where 32-bit arithmetic on the host or a
grid's dimension ends."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
TOP = 2 ** 31 - 1 - 1024


@pytest.fixture(autouse=True)
def _free():
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("D", [TOP - 1022, TOP - 1, TOP])
def test_combine_of_the_longest_rows(gpu, D):
    rows = torch.randint(-100, 100, (1, D), dtype=torch.int8, device=DEV).to(torch.bfloat16)
    slots = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    out = gpu.combine_experts(rows, slots, torch.full((1, 1), 2.0, device=DEV))
    rows *= 2
    assert torch.equal(out, rows)
