"""What is measured of the 8-bit-integer path: its products, the token
quantiser that feeds them, and the norms between two blocks.

  gemm      C[m,n] = a_s[m] * b_s[n] * sum_k A[m,k] * B[n,k] (+ bias[n]),
            A and B int8, one scale per token and one per output channel
  grouped   the same per expert: rows offsets[e] .. offsets[e+1]-1 of A use
            weight B[e] and scales b_s[e]
  quantize  s[m] = max(max_k |x[m,k]|, 1e-12) / 127,
            q[m,k] = round(clamp(x[m,k] / s[m], -127, 127)), ties to even
  norm      u = rms(h) * post_weight, r = residual_scale * x + gate * u,
            y = rms(r) * pre_weight, rms(v) = v / sqrt(mean(v^2) + eps);
            y in the type of x, or quantised per token (int8), or quantised
            per 128 columns (E4M3)

`run` takes the inputs that `prepare` makes through one of them: by
elementary operations in 32 bits where `own` is false, by the calls of
block_scaled_fp8_gemm_amd where it is true.  Codes are returned as the values
that they stand for, code * scale, rounded to bf16.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


def listed():
    return [
        # One token through a square projection: all of the weight is read for one row.
        {"name": "gemm_token", "op": "gemm", "M": 1, "N": 4096, "K": 4096, "out": "bf16", "bias": False, "pad": 0},
        # A decode batch of 64 through a narrow projection with a long K.
        {"name": "gemm_decode", "op": "gemm", "M": 64, "N": 512, "K": 4096, "out": "bf16", "bias": False, "pad": 0},
        # Sizes that no tile divides, rows that start off 16-byte boundaries, a bias, 32-bit outputs.
        {"name": "gemm_odd", "op": "gemm", "M": 301, "N": 1537, "K": 1000, "out": "fp32", "bias": True, "pad": 0},
        # Prefill: bound by the matrix cores.
        {"name": "gemm_prefill", "op": "gemm", "M": 16384, "N": 4096, "K": 4096, "out": "bf16", "bias": False,
         "pad": 0},
        # 64 tokens, 8 of 256 experts each: the experts' weights are what is read.
        {"name": "grouped_decode", "op": "grouped", "tokens": 64, "topk": 8, "E": 256, "N": 512, "K": 4096,
         "skew": 0.0, "out": "bf16"},
        # Few experts with uneven loads and sizes that no tile divides.
        {"name": "grouped_ragged", "op": "grouped", "tokens": 100, "topk": 2, "E": 8, "N": 515, "K": 776,
         "skew": 1.0, "out": "fp32"},
        # Prefill over the same 256 experts: 128 rows each on average.
        {"name": "grouped_prefill", "op": "grouped", "tokens": 4096, "topk": 8, "E": 256, "N": 512, "K": 4096,
         "skew": 0.0, "out": "bf16"},
        # The activations of a decode batch and of a prefill.
        {"name": "quantize_decode", "op": "quantize", "M": 64, "K": 4096, "dtype": "bf16", "pad": 0},
        {"name": "quantize_prefill", "op": "quantize", "M": 16384, "K": 4096, "dtype": "bf16", "pad": 0},
        # One token between two blocks, gated per channel.
        {"name": "norm_token", "op": "norm", "M": 1, "D": 4096, "dtype": "bf16", "gate": "channel", "post": True,
         "quant": "none", "pad": 0},
        # An odd width, one gate value per token, 32-bit activations.
        {"name": "norm_odd", "op": "norm", "M": 777, "D": 1027, "dtype": "fp32", "gate": "token", "post": True,
         "quant": "none", "pad": 0},
        # Prefill with a gate for every element, quantised for the int8 product that follows.
        {"name": "norm_prefill", "op": "norm", "M": 16384, "D": 4096, "dtype": "bf16", "gate": "full", "post": True,
         "quant": "int8", "pad": 0},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi, unit):
    """Half of the sizes are any number, the others a multiple of `unit`."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.5 else max(unit, v // unit * unit)


def draw(rng):
    op = rng.choice(["gemm", "grouped", "quantize", "norm"])
    if op == "gemm":
        M, N, K = _log(rng, 1, 16384), _size(rng, 64, 8192, 64), _size(rng, 64, 4096, 128)
        return {"op": op, "M": min(M, (16384 * 4096 * 4096) // (N * K)), "N": N, "K": K,
                "out": rng.choice(["bf16", "fp16", "fp32"]), "bias": rng.random() < 0.4,
                "pad": rng.choice([0, 0, 16, 3])}
    if op == "grouped":
        E = _log(rng, 4, 256)
        K = _size(rng, 64, 4096, 128)
        N = _size(rng, 64, max(64, min(2048, (256 * 512 * 4096) // (E * K))), 64)
        topk = rng.randint(1, min(8, E))
        tokens = min(_log(rng, 1, 4096), max(1, (4096 * 8 * 512 * 4096) // (topk * N * K)))
        return {"op": op, "tokens": tokens, "topk": topk, "E": E, "N": N, "K": K,
                "skew": round(rng.uniform(0.0, 0.6), 2), "out": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "quantize":
        K = _size(rng, 32, 16384, 128)
        return {"op": op, "M": min(_log(rng, 1, 16384), (16384 * 4096) // K), "K": K,
                "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "pad": rng.choice([0, 0, 8, 1])}
    D = _size(rng, 32, 8192, 128)
    quant = rng.choice(["none", "int8", "fp8"] if D % 128 == 0 else ["none", "int8"])
    return {"op": op, "M": min(_log(rng, 1, 16384), (16384 * 4096) // D), "D": D,
            "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]),
            "gate": rng.choice(["none", "channel", "token", "full"]), "post": rng.random() < 0.8, "quant": quant,
            "pad": rng.choice([0, 0, 8, 1])}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _codes(g, rows, cols, pad=0):
    """Int8 codes of normal values quantised per row (the largest of a row is
    about 4 deviations), in rows `pad` elements apart."""
    return _normal(g, rows, cols + pad).mul_(127.0 / 4.0).round_().clamp_(-127, 127).to(torch.int8)[:, :cols]


def _outlier_rows(g, M):
    """1% of tokens are ten times as large."""
    return 1.0 + 9.0 * (torch.rand(M, generator=g, device="cuda") < 0.01).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case, "op": op}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        s["A"] = _codes(g, M, K, case["pad"])
        s["a_s"] = _outlier_rows(g, M) * (4.0 / 127.0) * (1.0 + 0.1 * torch.rand(M, generator=g, device="cuda"))
        s["B"] = _codes(g, N, K)
        s["b_s"] = (0.02 * 4.0 / 127.0) * (1.0 + 0.1 * torch.rand(N, generator=g, device="cuda"))
        s["bias"] = 0.1 * _normal(g, N) if case["bias"] else None
        s["out"] = DTYPES[case["out"]]
    elif op == "grouped":
        E, N, K, T, topk = case["E"], case["N"], case["K"], case["tokens"], case["topk"]
        popular = case["skew"] * _normal(g, E)
        noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device="cuda").clamp_(1e-6, 1 - 1e-6)))
        picked = torch.topk(popular + noise, topk, dim=1).indices
        counts = torch.bincount(picked.reshape(-1), minlength=E)
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["most"] = int(counts.max())
        M = T * topk
        s["A"] = _codes(g, M, K)
        s["a_s"] = _outlier_rows(g, M) * (4.0 / 127.0) * (1.0 + 0.1 * torch.rand(M, generator=g, device="cuda"))
        s["B"] = _codes(g, E * N, K).view(E, N, K)
        s["b_s"] = (0.02 * 4.0 / 127.0) * (1.0 + 0.1 * torch.rand(E, N, generator=g, device="cuda"))
        s["out"] = DTYPES[case["out"]]
    elif op == "quantize":
        M, K = case["M"], case["K"]
        x = _normal(g, M, K + case["pad"]) * _outlier_rows(g, M)[:, None]
        s["x"] = x.to(DTYPES[case["dtype"]])[:, :K]
    else:
        M, D, t = case["M"], case["D"], DTYPES[case["dtype"]]
        channels = 1.0 + 4.0 * (torch.rand(D + case["pad"], generator=g, device="cuda") < 0.01).float()
        s["h"] = (0.5 * _normal(g, M, D + case["pad"]) * channels).to(t)[:, :D]
        s["x"] = (2.0 * _normal(g, M, D + case["pad"]) * _outlier_rows(g, M)[:, None]).to(t)[:, :D]
        s["post"] = (1.0 + 0.1 * _normal(g, D)).to(t) if case["post"] else None
        s["pre"] = (1.0 + 0.1 * _normal(g, D)).to(t)
        shape = {"none": None, "channel": (D,), "token": (M, 1), "full": (M, D)}[case["gate"]]
        s["gate"] = torch.sigmoid(_normal(g, *shape)).to(t) if shape else None
        s["scale"] = 0.875
    return s


# ---------------------------------------------------------------------------
# The plain forms, in 32 bits
# ---------------------------------------------------------------------------
def _plain_quantize(v):
    """Values that the int8 codes of each row stand for, and the rows' scales."""
    s = v.abs().amax(dim=1).clamp(min=1e-12) / 127.0
    return (torch.round((v / s[:, None]).clamp(-127, 127)) * s[:, None]).to(torch.bfloat16), s


def _plain_quantize_e4m3(v):
    groups = v.view(v.shape[0], -1, 128)
    s = groups.abs().amax(dim=2).clamp(min=1e-12) / 448.0
    codes = (groups / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return (codes.float() * s[..., None]).to(torch.bfloat16).view(v.shape), s


def _plain(s):
    op = s["op"]
    if op == "gemm":
        C = (s["A"].float() @ s["B"].float().t()) * (s["a_s"][:, None] * s["b_s"][None, :])
        return (C if s["bias"] is None else C + s["bias"]).to(s["out"])
    if op == "grouped":
        # Each expert's rows as columns of a matrix of its own, zeros past its last.
        E, N, K = s["B"].shape
        row = torch.arange(s["A"].shape[0], device="cuda", dtype=torch.int32)
        e = torch.searchsorted(s["offsets"][1:], row, right=True)
        at = row - s["offsets"][e]
        X = torch.zeros(E, s["most"], K, device="cuda")
        X[e, at] = s["A"].float()
        Y = torch.bmm(s["B"].float(), X.transpose(1, 2).contiguous())
        return (Y[e, :, at] * (s["a_s"][:, None] * s["b_s"][e])).to(s["out"])
    if op == "quantize":
        return _plain_quantize(s["x"].float())
    h, x, t = s["h"].float(), s["x"].float(), s["x"].dtype
    if s["post"] is not None:
        h = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS) * s["post"].float()
    if s["gate"] is not None:
        h = h * s["gate"].float()
    r = s["scale"] * x + h
    y = r * torch.rsqrt(r.square().mean(dim=1, keepdim=True) + EPS) * s["pre"].float()
    quant = s["case"]["quant"]
    if quant == "none":
        return r.to(t), y.to(t)
    return (r.to(t), *(_plain_quantize(y) if quant == "int8" else _plain_quantize_e4m3(y)))


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def _own(s):
    import block_scaled_fp8_gemm_amd as fbg

    op = s["op"]
    if op == "gemm":
        return fbg.int8_gemm(s["A"], s["a_s"], s["B"], s["b_s"], bias=s["bias"], out_dtype=s["out"])
    if op == "grouped":
        return fbg.int8_grouped_gemm(s["A"], s["a_s"], s["B"], s["b_s"], s["offsets"], out_dtype=s["out"])
    if op == "quantize":
        q, scale = fbg.quantize_tokens(s["x"])
        return torch.mul(q, scale[:, None], out=torch.empty_like(q, dtype=torch.bfloat16)), scale
    quant = s["case"]["quant"]
    got = fbg.block_norm(s["h"], s["x"], post_weight=s["post"], gate=s["gate"], pre_weight=s["pre"],
                         residual_scale=s["scale"], eps=EPS, quantize=None if quant == "none" else quant)
    if quant == "none":
        return got
    r, q, scale = got
    values = torch.empty_like(q, dtype=torch.bfloat16)
    if quant == "int8":
        torch.mul(q, scale[:, None], out=values)
    else:
        torch.mul(q.float().view(len(q), -1, 128), scale[..., None], out=values.view(len(q), -1, 128))
    return r, values, scale


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_codes(y, scale, fmt):
    """The values in `fmt` nearest to y / scale, ties to even, times scale."""
    v = y / scale
    if fmt == "int8":
        return torch.round(v.clamp(-127, 127)) * scale
    v = v.clamp(-448, 448)
    exponent = torch.frexp(v)[1].sub(1).clamp(min=-6)       # 2^exponent <= |v|, the subnormals' step below
    step = torch.ldexp(torch.ones_like(v), exponent - 3)    # three bits of fraction
    return torch.round(v / step) * step * scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gemm":
        C = torch.matmul(s["A"].double(), s["B"].double().t().contiguous())
        C = C * s["a_s"].double()[:, None] * s["b_s"].double()
        return C if s["bias"] is None else C + s["bias"].double()
    if op == "grouped":
        C = torch.empty(s["A"].shape[0], s["B"].shape[1], dtype=torch.float64, device="cuda")
        ends = s["offsets"].tolist()
        for e, (lo, hi) in enumerate(zip(ends, ends[1:])):
            if hi > lo:
                C[lo:hi] = torch.matmul(s["A"][lo:hi].double(), s["B"][e].double().t().contiguous())
                C[lo:hi] *= s["a_s"][lo:hi].double()[:, None] * s["b_s"][e].double()
        return C
    if op == "quantize":
        x = s["x"].double()
        scale = x.abs().max(dim=1).values.clamp(min=1e-12) / 127
        return _exact_codes(x, scale[:, None], "int8"), scale
    u = s["h"].double()
    D = u.shape[1]
    if s["post"] is not None:
        u = u / torch.sqrt((u * u).sum(dim=1, keepdim=True) / D + EPS) * s["post"].double()
    if s["gate"] is not None:
        u = u * s["gate"].double()
    r = s["scale"] * s["x"].double() + u
    y = r / torch.sqrt((r * r).sum(dim=1, keepdim=True) / D + EPS) * s["pre"].double()
    if case["quant"] == "none":
        return r, y
    if case["quant"] == "int8":
        scale = y.abs().max(dim=1).values.clamp(min=1e-12) / 127
        return r, _exact_codes(y, scale[:, None], "int8"), scale
    scale = y.view(len(y), -1, 128).abs().max(dim=2).values.clamp(min=1e-12) / 448
    return r, _exact_codes(y.view(len(y), -1, 128), scale[..., None], "e4m3").view(y.shape), scale


def work(case):
    """Bytes (each input read once, each output written once, the codes being
    the outputs of a quantiser) and operations of one pass."""
    op = case["op"]
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + N * K + 4 * M + 4 * N * (2 if case["bias"] else 1) + M * N * SIZES[case["out"]],
                "flops": 2 * M * N * K}
    if op == "grouped":
        E, N, K, T, topk = case["E"], case["N"], case["K"], case["tokens"], case["topk"]
        M, busy = T * topk, E * (1 - (1 - topk / E) ** T)   # experts that hold a row, picked evenly
        return {"bytes": M * K + busy * (N * K + 4 * N) + 4 * M + 4 * (E + 1) + M * N * SIZES[case["out"]],
                "flops": 2 * M * N * K}
    if op == "quantize":
        M, K = case["M"], case["K"]
        return {"bytes": M * K * SIZES[case["dtype"]] + M * K + 4 * M, "flops": 3 * M * K}
    M, D, size = case["M"], case["D"], SIZES[case["dtype"]]
    gate = {"none": 0, "channel": D, "token": M, "full": M * D}[case["gate"]]
    out = {"none": M * D * size, "int8": M * D + 4 * M, "fp8": M * D + 4 * M * (D // 128)}[case["quant"]]
    return {"bytes": (3 * M * D + gate + D * (2 if case["post"] else 1)) * size + out, "flops": 12 * M * D}
