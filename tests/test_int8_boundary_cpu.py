"""Host-side checks of the int8 and row entry points: every case fails
validation, or is empty, before any HIP call, so the pointers are never used."""
import ctypes
import os
import re

import pytest
import torch

import block_scaled_fp8_gemm_amd as fbg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x10000000  # made-up addresses, far apart


def _gemm(A=P, lda=256, a_s=2 * P, B=3 * P, ldb=256, b_s=4 * P, bias=None, C=5 * P, ldc=64, M=16, N=64, K=256, out=0):
    return fbg.load().fbg_int8_gemm(A, lda, a_s, B, ldb, b_s, bias, C, ldc, M, N, K, out, None)


def _grouped(A=P, lda=256, a_s=2 * P, B=3 * P, b_s=4 * P, C=5 * P, ldc=64, off=6 * P, E=4, M=16, N=64, K=256, out=0):
    return fbg.load().fbg_int8_grouped_gemm(A, lda, a_s, B, b_s, C, ldc, off, E, M, N, K, out, None)


def _quant(x=P, ldx=256, dtype=0, M=16, K=256, q=2 * P, ldq=256, scale=3 * P):
    return fbg.load().fbg_quantize_tokens(x, ldx, dtype, M, K, q, ldq, scale, None)


def _norm(h=P, ldh=256, x=2 * P, ldx=256, gate=None, grow=0, gcol=0, post=3 * P, pre=4 * P, dtype=0, wdtype=0, M=16,
          D=256, r=5 * P, ldr=256, y=6 * P, ldy=256, ys=7 * P, quant=0):
    return fbg.load().fbg_block_norm(h, ldh, x, ldx, gate, grow, gcol, post, pre, dtype, wdtype, M, D, 1.0, 1e-6, 0.0,
                                     r, ldr, y, ldy, ys, quant, None)


def test_every_declared_function_is_exported():
    text = open(os.path.join(ROOT, "include", "fp8bg.h")).read()
    names = set(re.findall(r"^int (fbg_\w+)\(", text, re.M))
    assert names == {"fbg_int8_gemm", "fbg_int8_grouped_gemm", "fbg_quantize_tokens", "fbg_block_norm",
                     "fbg_int8_plan"}
    for n in names:
        assert isinstance(getattr(fbg.load(), n), ctypes._CFuncPtr)


def test_gemm_refusals():
    bad, unsup = fbg.INVALID_VALUE, fbg.UNSUPPORTED
    for kw in ({"A": None}, {"a_s": None}, {"B": None}, {"b_s": None}, {"C": None}):
        assert _gemm(**kw) == bad, kw
    for kw in ({"M": -1}, {"N": -1}, {"K": -1}, {"out": 3}, {"out": -1}):
        assert _gemm(**kw) == bad, kw
    for kw in ({"lda": 255}, {"ldb": 255}, {"ldc": 63}, {"lda": 0}, {"ldb": -256}):
        assert _gemm(**kw) == bad, kw
    assert _gemm(K=131072, lda=131072, ldb=131072) == unsup          # the int32 sum could overflow
    assert _gemm(M=1 << 31) == unsup and _gemm(N=1 << 31, ldc=1 << 31) == unsup
    assert _gemm(M=(1 << 31) - 1000) == unsup                        # rounding up to a tile would pass 32 bits
    assert _quant(M=(1 << 31) - 1) == unsup and _norm(D=(1 << 31) - 1, ldh=1 << 31, ldx=1 << 31, ldr=1 << 31, ldy=1 << 31) == unsup
    assert _gemm(lda=1 << 24) == unsup and _gemm(ldb=1 << 24) == unsup
    assert _gemm(a_s=2 * P + 2) == unsup and _gemm(b_s=4 * P + 1) == unsup and _gemm(bias=8 * P + 3) == unsup
    assert _gemm(C=5 * P + 1) == unsup and _gemm(C=5 * P + 2, out=2) == unsup
    assert _gemm(C=P + 128) == bad and _gemm(C=3 * P) == bad and _gemm(C=2 * P) == bad and _gemm(C=4 * P) == bad
    assert _gemm(bias=5 * P + 64) == bad                             # C overlaps the bias
    assert _gemm(M=0, A=None, a_s=None, C=None) == fbg.SUCCESS
    assert _gemm(N=0, B=None, b_s=None, C=None) == fbg.SUCCESS


def test_grouped_refusals():
    bad, unsup = fbg.INVALID_VALUE, fbg.UNSUPPORTED
    for kw in ({"A": None}, {"a_s": None}, {"B": None}, {"b_s": None}, {"C": None}, {"off": None}, {"E": -1},
               {"M": -1}, {"K": -1}, {"out": 7}, {"lda": 100}, {"ldc": 10}):
        assert _grouped(**kw) == bad, kw
    assert _grouped(off=6 * P + 2) == unsup
    assert _grouped(E=1 << 30, N=1 << 30, ldc=1 << 30) == unsup      # E * N * K overflows
    assert _grouped(C=3 * P + 4096) == bad                           # C overlaps B
    assert _grouped(C=6 * P - 64) == bad                             # C overlaps the offsets
    assert _grouped(M=0, A=None, a_s=None, C=None) == fbg.SUCCESS


def test_quantize_refusals():
    bad, unsup = fbg.INVALID_VALUE, fbg.UNSUPPORTED
    for kw in ({"x": None}, {"q": None}, {"scale": None}, {"M": -1}, {"K": -1}, {"dtype": 3}, {"ldx": 255},
               {"ldq": 255}):
        assert _quant(**kw) == bad, kw
    assert _quant(x=P + 1) == unsup and _quant(x=P + 2, dtype=2) == unsup and _quant(scale=3 * P + 2) == unsup
    assert _quant(q=P + 64) == bad and _quant(scale=2 * P + 64) == bad and _quant(scale=P + 64) == bad
    assert _quant(M=0, x=None, q=None, scale=None) == fbg.SUCCESS


def test_norm_refusals():
    bad, unsup = fbg.INVALID_VALUE, fbg.UNSUPPORTED
    for kw in ({"h": None}, {"r": None}, {"y": None}, {"quant": 1, "ys": None}, {"quant": 3}, {"quant": -1},
               {"M": -1}, {"D": -1}, {"dtype": 3}, {"wdtype": 1}, {"ldh": 255}, {"ldx": 255}, {"ldr": 255},
               {"ldy": 255}, {"gate": 8 * P, "grow": -1}):
        assert _norm(**kw) == bad, kw
    assert _norm(quant=2, D=200) == unsup                            # E4M3 scales take 128 columns
    assert _norm(h=P + 1) == unsup and _norm(post=3 * P + 1) == unsup and _norm(ys=7 * P + 2, quant=1) == unsup
    assert _norm(r=2 * P) == bad and _norm(y=P + 512) == bad and _norm(r=6 * P + 512) == bad
    assert _norm(gate=5 * P, gcol=1) == bad                          # r overlaps the gate
    assert _norm(M=0, h=None, r=None, y=None) == fbg.SUCCESS
    assert _norm(D=0, h=None, r=None, y=None) == fbg.SUCCESS


def test_wrappers_refuse_host_tensors_and_wrong_types():
    A, s = torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4)
    with pytest.raises(ValueError):
        fbg.int8_gemm(A, s, A, s)
    with pytest.raises(ValueError):
        fbg.int8_gemm(A[0], s, A, s)
    with pytest.raises(ValueError):
        fbg.int8_grouped_gemm(A, s, A[None], s[None], torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        fbg.quantize_tokens(torch.zeros(4, 64))
    with pytest.raises(ValueError):
        fbg.block_norm(torch.zeros(4, 64))


def test_plan():
    for M, N, K, want in [(1, 4096, 4096, (2,)), (64, 4096, 4096, (11,)), (16384, 4096, 4096, (10,)), (128, 8192, 1024, (5, 6))]:
        p = fbg.int8_plan(M, N, K)
        assert p["variant_name"] == "int8" and p["config"] in want, (M, N, K, p)
        assert p["grid"] == -(-M // p["tile_m"]) * -(-N // p["tile_n"])
        assert p["split_k"] == 1 and p["workspace_bytes"] == 0
    # rows that are not whole 16-byte chunks never take the direct-to-LDS tiles
    for M in (1, 40, 300, 5000):
        assert fbg.int8_plan(M, 1000, 4096, aligned_rows=False)["config"] < 5
        assert fbg.int8_plan(M, 1000, 1001)["config"] < 5
    # small experts: long K over few of them on the skinny kernel; the grouped
    # grid bounds the experts' row tiles by floor(M / rows) + E
    assert fbg.int8_plan(64, 512, 4096, E=8)["config"] == 3
    assert fbg.int8_plan(8, 512, 4096, E=8)["config"] == 2
    p = fbg.int8_plan(512, 512, 4096, E=256)
    assert p["config"] == 12 and p["grid"] == (512 // 32 + 256) * 16
    p = fbg.int8_plan(512, 512, 1024, E=256)
    assert p["config"] == 5 and p["grid"] == (512 // 32 + 256) * 8
    assert fbg.int8_plan(32768, 512, 4096, E=256)["config"] >= 7
    assert fbg.int8_plan(0, 512, 4096)["config"] == -1 and fbg.int8_plan(7, 9, 15)["config"] == -1
    for kw in ({"M": -1}, {"E": -1}, {"cu_count": 0}):
        with pytest.raises(fbg.FP8BGError) as e:
            fbg.int8_plan(**{"M": 4, "N": 4, "K": 64, **kw})
        assert e.value.status == fbg.INVALID_VALUE
    with pytest.raises(fbg.FP8BGError) as e:
        fbg.int8_plan(4, 4, 131072)
    assert e.value.status == fbg.UNSUPPORTED


def test_every_configuration_is_chosen_for_some_shape():
    seen = set()
    for aligned in (True, False):
        for M in (1, 4, 12, 16, 24, 48, 100, 200, 400, 1000, 2048, 4096, 16384):
            for N in (64, 512, 1536, 4096, 8192):
                for K in (256, 1024, 4096):
                    seen.add(fbg.int8_plan(M, N, K, aligned_rows=aligned)["config"])
                    seen.add(fbg.int8_plan(M, N, K, E=64, aligned_rows=aligned)["config"])
    assert seen == set(range(13)), seen
