"""The int8 products on the GPU against their plain form: bit for bit with the
stated roundings (the integer sum is exact, so that holds for every kernel),
and within the derived bound of the 64-bit product."""
import numpy as np
import pytest
import torch

from tests import _int8 as T
from tests._gpu import forced_config

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _to(t, pitch=None):
    """On the GPU; with `pitch`, as a slice of rows that far apart, the gaps
    and the bytes after the last row holding other values."""
    if t is None:
        return None
    if pitch is None:
        return t.to(DEV)
    buf = torch.full((t.shape[0], pitch), 77, dtype=t.dtype, device=DEV)
    buf[:, :t.shape[1]] = t.to(DEV)
    return buf[:, :t.shape[1]]


def _gemm(fbg, d, dtype, lda=None, ldb=None, **kw):
    C = fbg.int8_gemm(_to(d["A"], lda), d["a_s"].to(DEV), _to(d["B"], ldb), d["b_s"].to(DEV), bias=_to(d["bias"]),
                      out_dtype=T.DTYPES[dtype], **kw)
    torch.cuda.synchronize()
    return C


# Row counts around every tile height, columns around every tile width, K
# around the MFMA's depth, the step and the pipeline's length.
SHAPES = [(1, 1, 1), (1, 16, 64), (1, 512, 4096), (2, 33, 127), (3, 130, 128), (5, 96, 129), (7, 257, 1000),
          (8, 64, 256), (15, 48, 63), (16, 512, 256), (17, 100, 300), (31, 129, 2048), (33, 4096, 64), (48, 72, 192),
          (64, 512, 4096), (65, 63, 65), (100, 200, 300), (127, 255, 511), (128, 256, 1024), (129, 257, 1025),
          (184, 512, 256), (200, 1000, 16), (255, 128, 4000), (256, 256, 128), (257, 513, 384), (300, 700, 515),
          (513, 300, 640), (1030, 260, 272), (70, 2050, 144), (9, 8200, 80)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
def test_product(gpu, M, N, K, out):
    d = T.make_gemm(M, N, K, seed=M * 7 + N * 3 + K, bias=(M + N + K) % 2 == 0)
    T.assert_gemm(_gemm(gpu, d, out), d, out, f"{M}x{N}x{K}")


@pytest.mark.parametrize("lda,ldb", [(320, 320), (304, None), (301, 333), (None, 301)])
@pytest.mark.parametrize("M", [1, 20, 150])
def test_row_pitches(gpu, M, lda, ldb):
    """Slices of wider buffers: what lies between the rows is not read into
    the sums, and an output slice leaves its surroundings alone."""
    d = T.make_gemm(M, 140, 300, seed=M, bias=True)
    buf = torch.full((M + 2, 150), 7.0, device=DEV)
    C = _gemm(gpu, d, "fp32", lda, ldb, out=buf[1:M + 1, 3:143])
    T.assert_gemm(C, d, "fp32")
    assert bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all())
    assert bool((buf[:, :3] == 7).all()) and bool((buf[:, 143:] == 7).all())


@pytest.mark.parametrize("shift", [1, 4, 8])
@pytest.mark.parametrize("M", [1, 130])
def test_unaligned_base(gpu, M, shift):
    d = T.make_gemm(M, 70, 256, seed=shift)
    A = torch.zeros(M * 256 + 32, dtype=torch.int8, device=DEV)[shift:shift + M * 256].view(M, 256)
    A.copy_(d["A"])
    C = gpu.int8_gemm(A, d["a_s"].to(DEV), d["B"].to(DEV), d["b_s"].to(DEV), out_dtype=torch.float32)
    T.assert_gemm(C, d, "fp32")


@pytest.mark.parametrize("M", [1, 17, 300])
def test_largest_sums(gpu, M):
    """Every product is 2^14: the sums reach 2^31 - 2^14 at the largest K."""
    K = 131071
    A, B = torch.full((M, K), -128, dtype=torch.int8, device=DEV), torch.full((20, K), -128, dtype=torch.int8, device=DEV)
    B[1].fill_(127)
    one = torch.ones(max(M, 20), device=DEV)
    C = gpu.int8_gemm(A, one[:M], B, one[:20], out_dtype=torch.float32)
    assert bool((C[:, 0] == float(16384 * K)).all())
    assert bool((C[:, 1] == float(torch.tensor(-128 * 127 * K, dtype=torch.float64).float())).all())


def test_empty_extents(gpu):
    z = lambda *s: torch.zeros(*s, device=DEV)
    i = lambda *s: torch.zeros(*s, dtype=torch.int8, device=DEV)
    assert gpu.int8_gemm(i(0, 64), z(0), i(5, 64), z(5)).shape == (0, 5)
    assert gpu.int8_gemm(i(4, 64), z(4), i(0, 64), z(0)).shape == (4, 0)
    bias = torch.arange(5.0, device=DEV)
    C = gpu.int8_gemm(i(4, 0), z(4) + 1, i(5, 0), z(5) + 1, bias=bias, out_dtype=torch.float32)
    assert torch.equal(C, bias.expand(4, 5))
    assert bool((gpu.int8_gemm(i(4, 0), z(4) + 1, i(5, 0), z(5) + 1) == 0).all())
    C = gpu.int8_grouped_gemm(i(4, 64), z(4), i(0, 5, 64), z(0, 5), torch.zeros(1, dtype=torch.int32, device=DEV))
    assert C.shape == (4, 5) and bool((C == 0).all())


@pytest.mark.parametrize("M", [1, 40, 300])
def test_non_finite_scales_stay_in_their_row_and_column(gpu, M):
    d = T.make_gemm(M, 96, 256, seed=5)
    want = T.gemm_bits(d, "fp32")
    a_s, b_s = d["a_s"].clone(), d["b_s"].clone()
    a_s[M // 2], b_s[40] = float("nan"), float("inf")
    C = gpu.int8_gemm(d["A"].to(DEV), a_s.to(DEV), d["B"].to(DEV), b_s.to(DEV), out_dtype=torch.float32).cpu()
    assert bool(C[M // 2].isnan().all())
    keep = torch.ones(M, 96, dtype=torch.bool)
    keep[M // 2], keep[:, 40] = False, False
    assert torch.equal(C[keep], want[keep])


# ---------------------------------------------------------------------------
# Grouped
# ---------------------------------------------------------------------------
GROUPS = {
    "one": [37], "single_rows": [1] * 9, "empty_ends": [0, 0, 5, 0, 130, 0], "decode": [2, 0, 1, 3, 0, 0, 4, 1, 2, 2],
    "ragged": [65, 0, 300, 1, 64, 17, 129], "big": [513, 0, 700], "many": ([0, 3, 1, 0, 2, 7, 0] * 20), "mid": [33, 40, 20, 64],
    "hundreds": [100, 140, 128, 257, 0, 90],
}


def _grouped(fbg, d, counts, dtype, offsets=None, **kw):
    off = offsets if offsets is not None else np.concatenate([[0], np.cumsum(counts)])
    C = fbg.int8_grouped_gemm(d["A"].to(DEV), d["a_s"].to(DEV), d["B"].to(DEV), d["b_s"].to(DEV),
                              torch.tensor(off, dtype=torch.int32, device=DEV), out_dtype=T.DTYPES[dtype], **kw)
    torch.cuda.synchronize()
    return C


def _expert(d, e, lo, hi):
    return {"A": d["A"][lo:hi], "a_s": d["a_s"][lo:hi], "B": d["B"][e], "b_s": d["b_s"][e], "bias": None}


@pytest.mark.parametrize("name", list(GROUPS))
@pytest.mark.parametrize("N,K,out", [(64, 256, "bf16"), (40, 11, "fp32"), (33, 17, "bf16"), (515, 776, "fp32"), (130, 1001, "fp16"), (512, 1024, "bf16")])
def test_grouped(gpu, name, N, K, out):
    counts = GROUPS[name]
    d = T.make_gemm(sum(counts), N, K, seed=len(counts) + N, experts=len(counts))
    C = _grouped(gpu, d, counts, out)
    lo = 0
    for e, n in enumerate(counts):
        if n:
            T.assert_gemm(C[lo:lo + n], _expert(d, e, lo, lo + n), out, f"{name} expert {e}")
        lo += n


def test_grouped_rows_of_no_expert_and_malformed_offsets(gpu):
    d = T.make_gemm(50, 70, 192, seed=3, experts=3)
    buf = torch.full((50, 70), 9.0, device=DEV)
    C = _grouped(gpu, d, None, "fp32", offsets=[5, 20, 20, 40], out=buf)
    assert bool((C[:5] == 9).all()) and bool((C[40:] == 9).all())
    T.assert_gemm(C[5:20], _expert(d, 0, 5, 20), "fp32")
    T.assert_gemm(C[20:40], _expert(d, 2, 20, 40), "fp32")
    # Out of range and decreasing: clamped; experts whose clamped range is
    # whole and alone give their product, nothing outside C is written.
    guard = torch.full((52, 70), 9.0, device=DEV)
    C = _grouped(gpu, d, None, "fp32", offsets=[-7, 30, 10, 1000], out=guard[1:51])
    assert bool((guard[0] == 9).all()) and bool((guard[51] == 9).all())
    T.assert_gemm(C[:10], _expert(d, 0, 0, 10), "fp32")
    T.assert_gemm(C[30:], _expert(d, 2, 30, 50), "fp32")


def test_grouped_single_expert_equals_the_product(gpu):
    d = T.make_gemm(90, 200, 512, seed=8, experts=1)
    C = _grouped(gpu, d, [90], "bf16")
    one = gpu.int8_gemm(d["A"].to(DEV), d["a_s"].to(DEV), d["B"][0].to(DEV), d["b_s"][0].to(DEV))
    assert torch.equal(C, one)


def test_moe_sizes_on_sampled_experts(gpu):
    """256 experts of 512 x 4096, 64 and 4096 tokens picking 8 each."""
    E, N, K = 256, 512, 4096
    g = torch.Generator(device=DEV).manual_seed(1)
    B = torch.randint(-127, 128, (E, N, K), generator=g, device=DEV, dtype=torch.int8)
    b_s = torch.rand(E, N, generator=g, device=DEV) * 0.01
    for tokens in (64, 1024, 4096):
        M = tokens * 8
        cnt = torch.bincount(torch.rand(tokens, E, generator=g, device=DEV).topk(8, dim=1).indices.reshape(-1), minlength=E)
        off = torch.cat([cnt.new_zeros(1), cnt.cumsum(0)]).to(torch.int32)
        A = torch.randint(-127, 128, (M, K), generator=g, device=DEV, dtype=torch.int8)
        a_s = torch.rand(M, generator=g, device=DEV)
        C = gpu.int8_grouped_gemm(A, a_s, B, b_s, off)
        ends = off.tolist()
        for e in (0, 1, 77, 128, 254, 255):
            lo, hi = ends[e], ends[e + 1]
            if hi > lo:
                d = {"A": A[lo:hi].cpu(), "a_s": a_s[lo:hi].cpu(), "B": B[e].cpu(), "b_s": b_s[e].cpu()}
                T.assert_gemm(C[lo:hi], d, "bf16", f"{tokens} tokens, expert {e}")


# ---------------------------------------------------------------------------
# Streams, graphs, repetition
# ---------------------------------------------------------------------------
def test_another_stream_and_repetition(gpu):
    d = T.make_gemm(77, 300, 1000, seed=4, bias=True)
    s = torch.cuda.Stream()
    args = [d[k].to(DEV) for k in ("A", "a_s", "B", "b_s", "bias")]
    torch.cuda.synchronize()
    C = gpu.int8_gemm(*args, out_dtype=torch.float32, out=torch.empty(77, 300, device=DEV), stream=s)
    s.synchronize()
    T.assert_gemm(C, d, "fp32")
    again = [gpu.int8_gemm(*args, out_dtype=torch.float32) for _ in range(5)]
    assert all(torch.equal(C, x) for x in again)


def test_graph_replays(gpu):
    """The whole chain captured once and replayed over new inputs."""
    h, x = (torch.randn(40, 512, device=DEV).to(torch.bfloat16) for _ in range(2))
    w = torch.randn(512, device=DEV).to(torch.bfloat16)
    B, b_s = gpu.quantize_tokens(torch.randn(256, 512, device=DEV).to(torch.bfloat16))
    Bg, bg = torch.stack([B, B.flip(0)]), torch.stack([b_s, b_s.flip(0)])
    off = torch.tensor([0, 13, 40], dtype=torch.int32, device=DEV)

    def chain():
        r, q, s = gpu.block_norm(h, x, post_weight=w, pre_weight=w, quantize="int8")
        q2, s2 = gpu.quantize_tokens(r)
        return r, q, s, gpu.int8_gemm(q, s, B, b_s), gpu.int8_grouped_gemm(q2, s2, Bg, bg, off)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        chain()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = chain()
    for i in range(4):
        h.copy_(torch.randn(40, 512, device=DEV))
        x.copy_(torch.randn(40, 512, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        assert all(torch.equal(a, b) for a, b in zip(got, chain())), i


# ---------------------------------------------------------------------------
# Every kernel configuration, forced
# ---------------------------------------------------------------------------
CONFIGS = range(13)


@pytest.mark.parametrize("cfg", CONFIGS)
@pytest.mark.parametrize("M,N,K,out", [(1, 1, 16, "fp32"), (1, 700, 128, "bf16"), (64, 64, 240, "fp16"), (70, 300, 384, "fp32"),
                                       (257, 264, 512, "bf16"), (300, 520, 656, "fp32"), (513, 257, 2048, "bf16"),
                                       (129, 640, 144, "fp16"), (600, 40, 1008, "bf16")])
def test_forced_configuration(gpu, cfg, M, N, K, out):
    d = T.make_gemm(M, N, K, seed=cfg + M, bias=cfg % 2 == 0)
    with forced_config(cfg):
        C = _gemm(gpu, d, out)
    T.assert_gemm(C, d, out, f"configuration {cfg}, {M}x{N}x{K}")


@pytest.mark.parametrize("cfg", CONFIGS)
@pytest.mark.parametrize("name", ["decode", "ragged", "empty_ends", "big"])
def test_forced_configuration_grouped(gpu, cfg, name):
    counts = GROUPS[name]
    d = T.make_gemm(sum(counts), 200, 336, seed=cfg, experts=len(counts))
    with forced_config(cfg):
        C = _grouped(gpu, d, counts, "bf16")
    lo = 0
    for e, n in enumerate(counts):
        if n:
            T.assert_gemm(C[lo:lo + n], _expert(d, e, lo, lo + n), "bf16", f"configuration {cfg}, {name} expert {e}")
        lo += n


def test_forced_configuration_that_does_not_take_the_operands(gpu):
    d = T.make_gemm(5, 7, 9, seed=1)
    for cfg in (1, 99):
        with forced_config(cfg), pytest.raises(gpu.FP8BGError) as e:
            _gemm(gpu, d, "bf16")
        assert e.value.status == gpu.UNSUPPORTED


def test_offsets_past_32_bits(gpu):
    """C, A and B of more than 2^31 (and A's rows of 2^32) elements: the first
    and last rows and columns, with pitches that put them that far apart."""
    K, N, M, lda = 64, 24, 70000, 65536
    A = torch.zeros(M * lda // 4 + 16, dtype=torch.int32, device=DEV).view(torch.int8)[:M * lda].view(M, lda)[:, :K]
    d = T.make_gemm(64, N, K, seed=2)
    rows = torch.cat([torch.arange(32), torch.arange(M - 32, M)]).to(DEV)
    A[rows] = d["A"].to(DEV)
    a_s = torch.ones(M, device=DEV)
    a_s[rows] = d["a_s"].to(DEV)
    C = gpu.int8_gemm(A, a_s, d["B"].to(DEV), d["b_s"].to(DEV), out_dtype=torch.float32)
    T.assert_gemm(C[rows], d, "fp32", "A past 2^32 bytes")
    del A, C
    out = torch.empty(40000, 65536, device=DEV, dtype=torch.bfloat16)[:, :N]       # C past 2^31 elements
    q = torch.zeros(40000, K, dtype=torch.int8, device=DEV)
    q[-64:] = d["A"].to(DEV)
    s = torch.ones(40000, device=DEV)
    s[-64:] = d["a_s"].to(DEV)
    C = gpu.int8_gemm(q, s, d["B"].to(DEV), d["b_s"].to(DEV), out=out)
    T.assert_gemm(C[-64:], d, "bf16", "C past 2^31 elements")


@pytest.mark.parametrize("cfg", [None, *CONFIGS])
def test_arbitrary_offsets_stay_inside_the_operands(gpu, cfg):
    """Offsets in no order at all: nothing outside C is written, and no value of
    C is anything but some expert's product for its row (ranges that overlap
    may each write a part of one) or what was there."""
    E, M, N, K = 70, 300, 64, 64
    r = np.random.default_rng(11)
    d = T.make_gemm(M, N, K, seed=6, experts=E)
    off = r.integers(-50, M + 50, E + 1)
    guard = torch.full((M + 2, N), 9.0, device=DEV)
    with forced_config(cfg):
        C = _grouped(gpu, d, None, "fp32", offsets=off.tolist(), out=guard[1:M + 1])
    assert bool((guard[0] == 9).all()) and bool((guard[-1] == 9).all())
    C = C.cpu()
    fine = C == 9
    for e in range(E):
        fine |= C == T.gemm_bits({"A": d["A"], "a_s": d["a_s"], "B": d["B"][e], "b_s": d["b_s"][e]}, "fp32")
    assert bool(fine.all())


@pytest.mark.parametrize("cfg", CONFIGS)
@pytest.mark.parametrize("out", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("N,off,pitch", [(257, 1, 259), (300, 3, 307), (513, 2, 516), (67, 5, 77)])
def test_outputs_that_start_anywhere(gpu, cfg, out, N, off, pitch):
    """Rows of C at any element, every configuration: what lies around them stays."""
    M, K = 261, 272
    d = T.make_gemm(M, N, K, seed=cfg + N, bias=cfg % 2 == 1)
    buf = torch.full((M + 2, pitch), 7.0, device=DEV, dtype=T.DTYPES[out])
    with forced_config(cfg):
        C = _gemm(gpu, d, out, out=buf[1:M + 1, off:off + N])
    T.assert_gemm(C, d, out, f"configuration {cfg}, {N} columns from {off}")
    assert bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all())
    assert bool((buf[:, :off] == 7).all()) and bool((buf[:, off + N:] == 7).all())
