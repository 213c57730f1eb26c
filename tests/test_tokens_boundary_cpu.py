"""Host-side checks of the routing, dispatch, combine and adapter entry points:
every case fails validation, or is empty, before any HIP call, so the pointers
are never used."""
import ctypes
import os
import re

import pytest
import torch

import block_scaled_fp8_gemm_amd as fbg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 0x100000000  # made-up addresses, far apart
BAD, UNSUP, MEM = fbg.INVALID_VALUE, fbg.UNSUPPORTED, fbg.OUT_OF_MEMORY
TOP = 2 ** 31 - 1 - 1024


def _route(logits=P, ld=256, dtype=0, T=16, E=256, topk=8, score=0, bias=2 * P, groups=8, topk_groups=4,
           group_score=1, renorm=1, mask=3 * P, weights=4 * P, experts=5 * P):
    return fbg.load().fbg_route_experts(logits, ld, dtype, T, E, topk, score, bias, groups, topk_groups, group_score,
                                        renorm, 1.0, mask, weights, experts, None)


def _dispatch(experts=P, T=16, topk=8, first=0, E=64, x=2 * P, ldx=256, K=256, size=1, xs=3 * P, S=2, rows=4 * P,
              ldr=256, rs=5 * P, off=6 * P, slots=7 * P):
    return fbg.load().fbg_dispatch_tokens(experts, T, topk, first, E, x, ldx, K, size, xs, S, rows, ldr, rs, off, slots,
                                          None)


def _combine(rows=P, ldr=256, dtype=0, R=128, slots=2 * P, weights=3 * P, base=4 * P, ldb=256, bdtype=0, out=5 * P,
             ldo=256, odtype=0, T=16, topk=8, D=256):
    return fbg.load().fbg_combine_experts(rows, ldr, dtype, R, slots, weights, base, ldb, bdtype, out, ldo, odtype, T,
                                          topk, D, None)


def _adapters(y=P, ldy=256, x=2 * P, ldx=128, A=3 * P, B=4 * P, ids=5 * P, scales=6 * P, out=7 * P, ldo=256, M=16,
              N=256, K=128, R=16, L=4, dtype=0, odtype=0, ws=8 * P, wn=None):
    wn = 1 << 30 if wn is None else wn
    return fbg.load().fbg_add_adapters(y, ldy, x, ldx, A, B, ids, scales, out, ldo, M, N, K, R, L, dtype, odtype, ws, wn,
                                       None)


def test_every_declared_function_is_exported():
    text = open(os.path.join(ROOT, "include", "fp8bg_tokens.h")).read()
    names = set(re.findall(r"^(?:int|size_t) (fbg_\w+)\(", text, re.M))
    assert names == {"fbg_route_experts", "fbg_dispatch_tokens", "fbg_combine_experts",
                     "fbg_add_adapters", "fbg_add_adapters_workspace_size"}
    for n in names:
        assert isinstance(getattr(fbg.load(), n), ctypes._CFuncPtr)


def test_the_header_compiles_as_c_and_cpp(tmp_path):
    import subprocess
    src = tmp_path / "t.c"
    src.write_text('#include "fp8bg_tokens.h"\nint main(void) { return FBG_SCORE_SOFTMAX + FBG_GROUP_MAX; }\n')
    for cc in (["gcc", "-std=c99"], ["g++", "-std=c++17", "-x", "c++"]):
        subprocess.run([*cc, "-Wall", "-Werror", "-fsyntax-only", "-I", os.path.join(ROOT, "include"), str(src)],
                       check=True)


def test_route_refusals():
    for kw in ({"logits": None}, {"weights": None}, {"experts": None}, {"T": -1}, {"E": -8}, {"topk": -1}, {"dtype": 3},
               {"score": 2}, {"group_score": 2}, {"groups": 0}, {"groups": 7}, {"topk_groups": 0}, {"topk_groups": 9},
               {"ld": 255}, {"topk": 33, "topk_groups": 1}, {"E": 0, "ld": 0}):
        assert _route(**kw) == BAD, kw
    for kw in ({"E": 1032, "ld": 2000}, {"topk": 65}, {"groups": 128, "topk_groups": 128}, {"T": TOP + 1}):
        assert _route(**kw) == UNSUP, kw
    assert _route(logits=P + 1) == UNSUP and _route(logits=P + 2, dtype=2) == UNSUP
    assert _route(bias=2 * P + 2) == UNSUP and _route(weights=4 * P + 1) == UNSUP and _route(experts=5 * P + 2) == UNSUP
    assert _route(weights=P + 64) == BAD and _route(experts=P + 64) == BAD and _route(weights=2 * P + 64) == BAD
    assert _route(weights=3 * P) == BAD and _route(weights=5 * P + 4) == BAD
    assert _route(T=0, logits=None, weights=None, experts=None) == fbg.SUCCESS
    assert _route(topk=0, logits=None, weights=None, experts=None) == fbg.SUCCESS


def test_dispatch_refusals():
    for kw in ({"experts": None}, {"x": None}, {"rows": None}, {"rs": None}, {"off": None}, {"slots": None}, {"T": -1},
               {"topk": -1}, {"E": -1}, {"first": -1}, {"K": -1}, {"S": -1}, {"size": 3}, {"size": 8}, {"ldx": 255}, {"ldr": 255}):
        assert _dispatch(**kw) == BAD, kw
    for kw in ({"T": TOP + 1}, {"topk": 65}, {"E": 1025}, {"first": TOP + 1}, {"T": 2 ** 26, "topk": 33}, {"K": TOP + 1, "ldx": 2 ** 32, "ldr": 2 ** 32}):
        assert _dispatch(**kw) == UNSUP, kw
    assert _dispatch(experts=P + 2) == UNSUP and _dispatch(x=2 * P + 1, size=2) == UNSUP
    assert _dispatch(rows=4 * P + 2, size=4) == UNSUP and _dispatch(xs=3 * P + 1) == UNSUP
    assert _dispatch(rs=5 * P + 1) == UNSUP and _dispatch(off=6 * P + 2) == UNSUP and _dispatch(slots=7 * P + 3) == UNSUP
    assert _dispatch(rows=2 * P + 256) == BAD and _dispatch(rows=P) == BAD and _dispatch(rs=3 * P) == BAD
    assert _dispatch(off=7 * P + 8) == BAD and _dispatch(slots=P) == BAD and _dispatch(off=4 * P) == BAD


def test_combine_refusals():
    for kw in ({"rows": None}, {"slots": None}, {"weights": None}, {"out": None}, {"R": -1}, {"T": -1}, {"topk": -1},
               {"D": -1}, {"dtype": 3}, {"odtype": 3}, {"bdtype": 1}, {"ldr": 255}, {"ldb": 255}, {"ldo": 255}):
        assert _combine(**kw) == BAD, kw
    for kw in ({"T": TOP + 1}, {"R": TOP + 1}, {"topk": 65}, {"D": TOP + 1, "ldr": 2 ** 32, "ldb": 2 ** 32, "ldo": 2 ** 32}):
        assert _combine(**kw) == UNSUP, kw
    assert _combine(rows=P + 1) == UNSUP and _combine(slots=2 * P + 1) == UNSUP and _combine(weights=3 * P + 2) == UNSUP
    assert _combine(base=4 * P + 1) == UNSUP and _combine(out=5 * P + 2, odtype=2) == UNSUP
    assert _combine(out=P + 512) == BAD and _combine(out=2 * P) == BAD and _combine(out=3 * P) == BAD
    assert _combine(out=4 * P + 512) == BAD                              # near the base, but not the base
    assert _combine(out=4 * P, ldo=512) == BAD                           # the base with another pitch
    assert _combine(T=0, rows=None, slots=None, weights=None, out=None) == fbg.SUCCESS
    assert _combine(D=0, ldr=0, ldb=0, ldo=0, rows=None, out=None) == fbg.SUCCESS


def test_adapter_refusals():
    for kw in ({"y": None}, {"x": None}, {"A": None}, {"B": None}, {"ids": None}, {"out": None}, {"M": -1}, {"N": -1},
               {"K": -1}, {"R": -1}, {"L": -1}, {"dtype": 2}, {"dtype": -1}, {"odtype": 3}, {"ldy": 255}, {"ldx": 127},
               {"ldo": 255}):
        assert _adapters(**kw) == BAD, kw
    for kw in ({"M": TOP + 1}, {"N": TOP + 1, "ldy": 2 ** 32, "ldo": 2 ** 32}, {"R": 257}, {"K": 1 << 24, "ldx": 1 << 24}, {"L": TOP + 1}):
        assert _adapters(**kw) == UNSUP, kw
    assert _adapters(y=P + 1) == UNSUP and _adapters(x=2 * P + 1) == UNSUP and _adapters(A=3 * P + 1) == UNSUP
    assert _adapters(B=4 * P + 1) == UNSUP and _adapters(ids=5 * P + 2) == UNSUP and _adapters(scales=6 * P + 2) == UNSUP
    assert _adapters(out=7 * P + 2, odtype=2) == UNSUP and _adapters(ws=8 * P + 8) == UNSUP
    assert _adapters(out=P + 512) == BAD and _adapters(out=P, ldo=512) == BAD
    for p in (2, 3, 4, 5, 6):
        assert _adapters(out=p * P) == BAD, p
        assert _adapters(ws=p * P) == BAD, p
    assert _adapters(ws=7 * P) == BAD and _adapters(ws=P) == BAD
    need = fbg.load().fbg_add_adapters_workspace_size(16, 256, 128, 16)
    assert need > 0 and _adapters(wn=need - 1) == MEM and _adapters(ws=None) == MEM
    assert fbg.load().fbg_add_adapters_workspace_size(16, 256, 128, 257) == ctypes.c_size_t(-1).value
    assert _adapters(M=0, y=None, x=None, out=None) == fbg.SUCCESS
    assert _adapters(N=0, y=None, out=None) == fbg.SUCCESS
    for kw in ({"K": 0}, {"R": 0}, {"L": 0}):                            # in place, and nothing to add
        assert _adapters(out=P, x=None, A=None, B=None, ids=None, ws=None, **kw) == fbg.SUCCESS


def test_python_refuses_host_tensors():
    z = torch.zeros(4, 8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        fbg.route_experts(z, 2)
    with pytest.raises(ValueError, match="CUDA"):
        fbg.dispatch_tokens(i, 8, z)
    with pytest.raises(ValueError, match="CUDA"):
        fbg.combine_experts(z, i, torch.zeros(4, 2))
    with pytest.raises(ValueError, match="CUDA"):
        fbg.add_adapters(z, z, torch.zeros(1, 2, 8), torch.zeros(1, 8, 2), i[:, 0])
    with pytest.raises(TypeError, match="tensor"):
        fbg.route_experts(None, 2)
