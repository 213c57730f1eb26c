"""FBG_LOG=1 prints each call's plan, the int8 products' too."""
import pytest
import torch

from tests._gpu import forced_config

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_log(gpu, capfd, monkeypatch):
    monkeypatch.setenv("FBG_LOG", "1")
    A, s = torch.zeros(5, 64, dtype=torch.int8, device=DEV), torch.zeros(5, device=DEV)
    off = torch.tensor([0, 2, 5], dtype=torch.int32, device=DEV)
    gpu.int8_gemm(A, s, A, s)
    gpu.int8_grouped_gemm(A, s, torch.stack([A, A]), torch.stack([s, s]), off, out_dtype=torch.float32)
    with forced_config(6):
        gpu.int8_gemm(A, s, A, s)
    gpu.int8_gemm(A[:, :9], s, A[:, :9], s)
    p, g = gpu.int8_plan(5, 5, 64), gpu.int8_plan(5, 5, 64, E=2)
    lines = [l for l in capfd.readouterr().err.splitlines() if l.startswith("fp8bg int8")]
    assert lines == [f"fp8bg int8: E=0 M=5 N=5 K=64 out=0 -> cfg={p['config']} grid={p['grid']}",
                     f"fp8bg int8: E=2 M=5 N=5 K=64 out=2 -> cfg={g['config']} grid={g['grid']}",
                     "fp8bg int8: E=0 M=5 N=5 K=64 out=0 -> cfg=6 grid=1",
                     "fp8bg int8: E=0 M=5 N=5 K=9 out=0 -> cfg=-1 grid=0"]
    monkeypatch.setenv("FBG_LOG", "0")
    gpu.int8_gemm(A, s, A, s)
    assert "fp8bg" not in capfd.readouterr().err
